"""ctypes view of libgdn.so: the structs and prototypes of include/libgdn.h.

Loading is lazy; a missing library raises at first use (there is no other
implementation to fall back to).
"""
from __future__ import annotations

import ctypes
import os
import threading
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libgdn.so")

GDN_OK = 0
GDN_F32, GDN_BF16, GDN_E4M3, GDN_I8 = 0, 1, 2, 3
GDN_DECAY_LOG, GDN_DECAY_GAMMA = 0, 1

STATUS_NAMES = {0: "GDN_OK", 1: "GDN_ERR_NULL", 2: "GDN_ERR_SHAPE", 3: "GDN_ERR_DTYPE",
                4: "GDN_ERR_LAYOUT", 5: "GDN_ERR_UNSUPPORTED", 6: "GDN_ERR_HIP"}

# every extern "C" symbol include/libgdn.h declares
EXPORTED = ("gdn_last_error", "gdn_version", "gdn_header_digest", "gdn_gate", "gdn_prefill", "gdn_prefill_workspace_size",
            "gdn_prefill_noalloc", "gdn_decode", "gdn_conv1d", "gdn_wait_timeouts",
            "gdn_attn_decode", "gdn_attn_decode_workspace_size", "gdn_kv_append", "gdn_kv_read", "gdn_rope",
            "gdn_pages_copy",
            "gdn_pages_workspace_size", "gdn_pages_extend", "gdn_pages_fork", "gdn_pages_free",
            "gdn_pages_compact")
NOALLOC_SCRATCH_BYTES = 32 << 20  # GDN_NOALLOC_SCRATCH_BYTES

_i32, _i64, _f32, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class PrefillArgs(ctypes.Structure):
    _fields_ = [
        ("n_seqs", _i32), ("seq_len", _i32), ("total_tokens", _i64),
        ("hq", _i32), ("hv", _i32), ("dk", _i32), ("dv", _i32),
        ("io_dtype", _i32), ("decay_kind", _i32), ("chunk_size", _i32), ("scale", _f32),
        ("q", _vp), ("q_stride_token", _i64), ("q_stride_head", _i64),
        ("k", _vp), ("k_stride_token", _i64), ("k_stride_head", _i64),
        ("v", _vp), ("v_stride_token", _i64), ("v_stride_head", _i64),
        ("out", _vp), ("out_stride_token", _i64), ("out_stride_head", _i64),
        ("decay", _vp), ("beta", _vp), ("cu_seqlens", _vp),
        ("initial_state", _vp), ("final_state", _vp),
        ("qk_l2norm", _i32), ("qk_l2norm_eps", _f32),
        ("A_log", _vp), ("dt_bias", _vp), ("gate_a", _vp), ("gate_b", _vp),
        ("update_rule", _i32),
        ("state_pool", _vp), ("pool_size", _i32),
        ("pool_slot_stride", _i64), ("pool_head_stride", _i64),
        ("read_slot", _vp), ("write_slot", _vp),
        ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
        ("decay_per_key", _i32),
    ]


class DecodeArgs(ctypes.Structure):
    _fields_ = [
        ("batch", _i32), ("T", _i32), ("n_householder", _i32),
        ("hq", _i32), ("hv", _i32), ("dk", _i32), ("dv", _i32),
        ("io_dtype", _i32), ("disable_state_update", _i32), ("scale", _f32),
        ("q", _vp), ("k", _vp), ("v", _vp), ("A_log", _vp), ("dt_bias", _vp),
        ("a", _vp), ("b", _vp),
        ("pool", _vp), ("pool_size", _i32),
        ("pool_slot_stride", _i64), ("pool_head_stride", _i64),
        ("read_idx", _vp), ("write_idx", _vp), ("scatter_idx", _vp),
        ("out", _vp),
        ("qk_l2norm", _i32), ("qk_l2norm_eps", _f32),
        ("decay_per_key", _vp),
    ]


class Conv1dArgs(ctypes.Structure):
    _fields_ = [
        ("total_tokens", _i64), ("conv_dim", _i32), ("kernel_size", _i32),
        ("n_seqs", _i32), ("io_dtype", _i32), ("write_state", _i32), ("max_slots", _i32),
        ("x", _vp), ("x_stride_token", _i64),
        ("weight", _vp), ("conv_state", _vp),
        ("slot_idx", _vp), ("row_offsets", _vp),
        ("out", _vp), ("out_stride_token", _i64),
    ]


class AttnDecodeArgs(ctypes.Structure):
    _fields_ = [
        ("batch", _i32), ("T", _i32), ("hq", _i32), ("hkv", _i32), ("d", _i32),
        ("io_dtype", _i32), ("cache_dtype", _i32), ("scale", _f32),
        ("q", _vp), ("q_stride_row", _i64), ("q_stride_token", _i64), ("q_stride_head", _i64),
        ("k_cache", _vp), ("k_stride_page", _i64), ("k_stride_token", _i64), ("k_stride_head", _i64),
        ("v_cache", _vp), ("v_stride_page", _i64), ("v_stride_token", _i64), ("v_stride_head", _i64),
        ("n_pages", _i32), ("page_size", _i32), ("max_pages", _i32),
        ("page_table", _vp), ("page_table_stride", _i64), ("lens", _vp),
        ("k_scale", _vp), ("v_scale", _vp),
        ("out", _vp), ("lse", _vp), ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
        ("scale_block", _i32), ("k_block_scale", _vp), ("v_block_scale", _vp),
    ]


class KvAppendArgs(ctypes.Structure):
    _fields_ = [
        ("total_tokens", _i64), ("batch", _i32), ("hkv", _i32), ("d", _i32),
        ("io_dtype", _i32), ("cache_dtype", _i32),
        ("k", _vp), ("k_stride_token", _i64), ("k_stride_head", _i64),
        ("v", _vp), ("v_stride_token", _i64), ("v_stride_head", _i64),
        ("cu_seqlens", _vp),
        ("k_cache", _vp), ("kc_stride_page", _i64), ("kc_stride_token", _i64), ("kc_stride_head", _i64),
        ("v_cache", _vp), ("vc_stride_page", _i64), ("vc_stride_token", _i64), ("vc_stride_head", _i64),
        ("n_pages", _i32), ("page_size", _i32), ("max_pages", _i32),
        ("page_table", _vp), ("page_table_stride", _i64), ("lens", _vp),
        ("k_scale", _vp), ("v_scale", _vp),
        ("scale_block", _i32), ("k_block_scale", _vp), ("v_block_scale", _vp),
    ]


class KvReadArgs(ctypes.Structure):
    _fields_ = KvAppendArgs._fields_ + [("zero_rest", _i32)]


class RopeArgs(ctypes.Structure):
    _fields_ = [
        ("total_tokens", _i64), ("batch", _i32), ("hq", _i32), ("hkv", _i32), ("d", _i32), ("rot", _i32),
        ("io_dtype", _i32), ("interleaved", _i32), ("factor", _f32),
        ("q", _vp), ("q_stride_token", _i64), ("q_stride_head", _i64),
        ("k", _vp), ("k_stride_token", _i64), ("k_stride_head", _i64),
        ("q_out", _vp), ("qo_stride_token", _i64), ("qo_stride_head", _i64),
        ("k_out", _vp), ("ko_stride_token", _i64), ("ko_stride_head", _i64),
        ("inv_freq", _vp), ("positions", _vp), ("positions_i64", _i32),
        ("lens", _vp), ("cu_seqlens", _vp), ("zero_rest", _i32),
    ]


class PagesArgs(ctypes.Structure):
    _fields_ = [
        ("rows", _i32), ("max_pages", _i32), ("n_pages", _i32), ("page_size", _i32),
        ("page_table", _vp), ("page_table_stride", _i64), ("lens", _vp), ("refs", _vp),
        ("page_table_out", _vp), ("page_table_out_stride", _i64), ("lens_out", _vp), ("refs_out", _vp),
        ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
    ]


_lock = threading.Lock()
_lib = None
_calls = None
_no_calls = False  # whether loading the module has failed


def load(path: str | None = None):
    """Load libgdn.so (once) and declare its prototypes."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError("libgdn.so is not built (%s); run "
                               "`python -m gated_deltanet_state_delta_amd.build`" % p)
        lib = ctypes.CDLL(p)
        lib.gdn_last_error.restype = ctypes.c_char_p
        lib.gdn_last_error.argtypes = []
        lib.gdn_version.restype = ctypes.c_char_p
        lib.gdn_version.argtypes = []
        lib.gdn_header_digest.restype = ctypes.c_char_p
        lib.gdn_header_digest.argtypes = []
        lib.gdn_gate.restype = ctypes.c_int
        lib.gdn_gate.argtypes = [_vp, _vp, _vp, _vp, _i32, _i64, _i32, _vp, _vp, _vp, _vp]
        lib.gdn_prefill_workspace_size.restype = ctypes.c_size_t
        lib.gdn_prefill_workspace_size.argtypes = [ctypes.POINTER(PrefillArgs)]
        lib.gdn_prefill.restype = ctypes.c_int
        lib.gdn_prefill.argtypes = [ctypes.POINTER(PrefillArgs), _vp]
        lib.gdn_prefill_noalloc.restype = ctypes.c_int
        lib.gdn_prefill_noalloc.argtypes = [ctypes.POINTER(PrefillArgs), _vp]
        lib.gdn_decode.restype = ctypes.c_int
        lib.gdn_decode.argtypes = [ctypes.POINTER(DecodeArgs), _vp]
        lib.gdn_wait_timeouts.restype = ctypes.c_int
        lib.gdn_wait_timeouts.argtypes = [ctypes.POINTER(ctypes.c_uint32), _i32]
        lib.gdn_conv1d.restype = ctypes.c_int
        lib.gdn_conv1d.argtypes = [ctypes.POINTER(Conv1dArgs), _vp]
        lib.gdn_attn_decode_workspace_size.restype = ctypes.c_size_t
        lib.gdn_attn_decode_workspace_size.argtypes = [ctypes.POINTER(AttnDecodeArgs)]
        lib.gdn_attn_decode.restype = ctypes.c_int
        lib.gdn_attn_decode.argtypes = [ctypes.POINTER(AttnDecodeArgs), _vp]
        lib.gdn_kv_append.restype = ctypes.c_int
        lib.gdn_kv_append.argtypes = [ctypes.POINTER(KvAppendArgs), _vp]
        lib.gdn_kv_read.restype = ctypes.c_int
        lib.gdn_kv_read.argtypes = [ctypes.POINTER(KvReadArgs), _vp]
        lib.gdn_rope.restype = ctypes.c_int
        lib.gdn_rope.argtypes = [ctypes.POINTER(RopeArgs), _vp]
        lib.gdn_pages_copy.restype = ctypes.c_int
        lib.gdn_pages_copy.argtypes = [_vp, _i64, _i64, _i32, _vp, _vp, _i64, _vp]
        lib.gdn_pages_workspace_size.restype = ctypes.c_size_t
        lib.gdn_pages_workspace_size.argtypes = [_i32, _i32]
        pages = ctypes.POINTER(PagesArgs)
        for name, argtypes in (("gdn_pages_extend", [pages, _vp, _vp, _vp]),
                               ("gdn_pages_fork", [pages, _vp, _vp, _vp, _vp]),
                               ("gdn_pages_free", [pages, _vp, _vp]),
                               ("gdn_pages_compact", [pages, _vp, _vp, _vp, _vp])):
            getattr(lib, name).restype = ctypes.c_int
            getattr(lib, name).argtypes = argtypes
        if path is None:
            _lib = lib
        return lib


def calls():
    """The module _calls (binding/calls.cpp), bound to the library.  Binding raises
    where the two were built from different headers."""
    global _calls
    if _calls is None:
        lib = load()
        if not os.path.exists(os.path.join(PKG, "_calls.so")):
            raise RuntimeError("_calls.so is not built; run `python -m gated_deltanet_state_delta_amd.build`")
        from . import _calls as module
        module.bind(*(ctypes.cast(getattr(lib, "gdn_" + name), _vp).value for name in
                      ("header_digest", "attn_decode", "attn_decode_workspace_size", "kv_append", "kv_read", "rope")))
        _calls = module
    return _calls


def short_way():
    """calls(), or None where the module is missing or does not load: the calls then
    go the general way in Python, with one warning."""
    global _no_calls
    if not _no_calls:
        load()  # without the library there is no way at all
        try:
            return calls()
        except (ImportError, RuntimeError) as e:
            _no_calls = True
            warnings.warn("calls of one token a row take 5 to 10 us longer on the host, without the module _calls: %s" % e,
                          RuntimeWarning, stacklevel=4)
    return None


class GdnError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__("%s: %s" % (STATUS_NAMES.get(status, str(status)), msg))
        self.status = status


def check(status: int):
    if status != GDN_OK:
        raise GdnError(status, load().gdn_last_error().decode(errors="replace"))
