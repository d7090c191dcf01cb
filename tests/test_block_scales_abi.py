"""Refusals of the block-scaled cache calls, of kv_read and of rope on the host
(no GPU needed), and the frequencies of long contexts."""
import ctypes
import math
import os

import pytest
import torch

import gated_deltanet_state_delta_amd as gdn
import gated_deltanet_state_delta_amd._lib as L
from test_abi import test_struct_layout_matches_the_binding as layout_test
from test_paged_abi import CACHE_ERRORS, FAKE, _append, _attn, _set


def _read(**over):
    a = L.KvReadArgs()
    for f, _ in L.KvAppendArgs._fields_:
        setattr(a, f, getattr(_append(), f))
    return _set(a, over)


CALLS = {"attn_decode": _attn, "kv_append": _append, "kv_read": _read}
BLOCKS = dict(cache_dtype=2, scale_block=8, k_block_scale=FAKE, v_block_scale=FAKE)


@pytest.mark.parametrize("cname,pycls", [("gdn_attn_decode_args", "AttnDecodeArgs"), ("gdn_kv_append_args", "KvAppendArgs"),
                                         ("gdn_kv_read_args", "KvReadArgs"), ("gdn_rope_args", "RopeArgs")])
def test_struct_layout(cname, pycls, tmp_path):
    layout_test(cname, pycls, tmp_path)


@pytest.mark.parametrize("call", sorted(CALLS))
@pytest.mark.parametrize("over,status", [
    (dict(cache_dtype=3), 1),                                      # int8 without block scales
    (dict(cache_dtype=3, k_scale=FAKE, v_scale=FAKE), 1),
    (dict(scale_block=8, k_block_scale=FAKE, v_block_scale=FAKE), 2),  # bf16 cache
    (dict(BLOCKS, scale_block=-8), 2), (dict(BLOCKS, scale_block=0), 2), (dict(BLOCKS, scale_block=5), 2),
    (dict(BLOCKS, scale_block=32), 2),                             # over the page
    (dict(BLOCKS, k_scale=FAKE), 2), (dict(BLOCKS, v_scale=FAKE), 2),
    (dict(BLOCKS, k_block_scale=None), 1), (dict(BLOCKS, v_block_scale=None), 1),
    (dict(BLOCKS, k_block_scale=FAKE + 2), 4), (dict(BLOCKS, cache_dtype=3, v_block_scale=FAKE + 1), 4),
    (dict(BLOCKS, cache_dtype=4), 3),
    (dict(BLOCKS, page_size=1 << 17, scale_block=1 << 17, max_pages=1), 5),
])
def test_block_scales_refused(call, over, status):
    lib = L.load()
    assert getattr(lib, "gdn_" + call)(ctypes.byref(CALLS[call](**over)), None) == status, lib.gdn_last_error()
    assert ("gdn_" + call).encode() in lib.gdn_last_error()


@pytest.mark.parametrize("over,status", CACHE_ERRORS + [
    (dict(total_tokens=-1), 2), (dict(total_tokens=7), 2), (dict(total_tokens=(1 << 28) + 4), 5),
    (dict(hkv=1 << 17), 5), (dict(k=None), 1), (dict(v=None), 1), (dict(k=FAKE + 2), 4),
    (dict(k_stride_token=100), 4), (dict(v_stride_head=-64), 4),
    (dict(kc_stride_token=60), 4), (dict(vc_stride_head=1 << 23), 4), (dict(kc_stride_page=2000), 4),
])
def test_kv_read_refuses(over, status):
    assert L.load().gdn_kv_read(ctypes.byref(_read(**over)), None) == status, L.load().gdn_last_error()


def test_too_many_blocks_are_refused():
    lib = L.load()
    a = _append(**dict(BLOCKS, total_tokens=4, batch=1 << 28, cu_seqlens=FAKE))
    assert lib.gdn_kv_append(ctypes.byref(a), None) == 5 and b"2 * batch" in lib.gdn_last_error()


@pytest.mark.parametrize("over", [dict(), dict(v_cache=FAKE * 2), dict(v_block_scale=FAKE * 2)])
def test_keys_and_values_have_caches_and_scales_of_their_own(over):
    lib = L.load()
    a = _append(**{**BLOCKS, "k_cache": FAKE, "v_cache": FAKE, "k_block_scale": FAKE, "v_block_scale": FAKE, **over})
    assert lib.gdn_kv_append(ctypes.byref(a), None) == 4 and b"for keys and values" in lib.gdn_last_error()


def test_nothing_to_do_needs_no_launch():
    lib = L.load()
    for over in (dict(batch=0), dict(total_tokens=0)):
        assert lib.gdn_kv_read(ctypes.byref(_read(**over)), None) == 0
        assert lib.gdn_kv_append(ctypes.byref(_append(**dict(BLOCKS, **over))), None) == 0
    assert lib.gdn_kv_append(ctypes.byref(_append(**dict(BLOCKS, n_pages=0, k_block_scale=None))), None) == 0
    assert lib.gdn_attn_decode(ctypes.byref(_attn(**dict(BLOCKS, batch=0))), None) == 0
    assert lib.gdn_kv_read(None, None) == 1 and lib.gdn_rope(None, None) == 1
    assert lib.gdn_rope(ctypes.byref(_rope(total_tokens=0)), None) == 0
    assert lib.gdn_rope(ctypes.byref(_rope(batch=0)), None) == 0


def test_workspace_of_an_int8_cache_is_that_of_any_8_bit_one():
    f = L.load().gdn_attn_decode_workspace_size
    big = dict(batch=1, max_pages=1000, page_table_stride=1000)
    sizes = [f(ctypes.byref(_attn(**big, cache_dtype=t))) for t in (2, 3)]
    assert sizes[0] == sizes[1] > 0


def _rope(**over):
    a = L.RopeArgs()
    a.total_tokens, a.batch, a.hq, a.hkv, a.d, a.rot, a.io_dtype, a.factor = 8, 4, 6, 2, 64, 32, 1, 1.0
    a.q, a.q_stride_token, a.q_stride_head = FAKE, 384, 64
    a.k, a.k_stride_token, a.k_stride_head = FAKE * 2, 128, 64
    a.q_out, a.qo_stride_token, a.qo_stride_head = FAKE * 3, 384, 64
    a.k_out, a.ko_stride_token, a.ko_stride_head = FAKE * 4, 128, 64
    a.inv_freq, a.lens = FAKE * 5, FAKE * 6
    return _set(a, over)


@pytest.mark.parametrize("over,status", [
    (dict(io_dtype=2), 3), (dict(io_dtype=3), 3), (dict(total_tokens=-1), 2), (dict(total_tokens=7), 2), (dict(batch=-1), 2),
    (dict(hq=0), 2), (dict(hkv=-1), 2), (dict(d=0), 2), (dict(rot=0), 2), (dict(rot=31), 2), (dict(rot=66), 2),
    (dict(d=1026), 5), (dict(hq=1 << 16), 5), (dict(total_tokens=(1 << 24) + 4), 5),
    (dict(q=None), 1), (dict(q_out=None), 1), (dict(inv_freq=None), 1), (dict(lens=None), 1), (dict(k=None), 1),
    (dict(k_out=None), 1), (dict(hkv=0), 1), (dict(hkv=0, k=None), 1),
    (dict(q=FAKE + 1), 4), (dict(k_out=FAKE * 4 + 1), 4), (dict(inv_freq=FAKE + 4), 4), (dict(positions=FAKE + 2), 4),
    (dict(positions=FAKE + 4, positions_i64=1), 4),
    (dict(q_stride_token=-384), 4), (dict(qo_stride_head=-1), 4), (dict(k_stride_token=1 << 40), 4),
    (dict(q_out=FAKE, qo_stride_token=400), 4), (dict(k_out=FAKE * 2, ko_stride_head=32), 4),  # in place, other strides
    (dict(q_out=FAKE + 64), 4), (dict(k_out=FAKE * 2 + 512), 4),                                # partly over the input
    (dict(q_out=FAKE * 2), 4), (dict(k_out=FAKE), 4), (dict(k_out=FAKE * 3), 4),                # over the other's
])
def test_rope_refuses(over, status):
    assert L.load().gdn_rope(ctypes.byref(_rope(**over)), None) == status, L.load().gdn_last_error()
    assert b"gdn_rope" in L.load().gdn_last_error()


# ------------------------------------------------------------------ binding --

E4, I8 = torch.zeros(10, 16, 2, 64, dtype=torch.float8_e4m3fn), torch.zeros(10, 16, 2, 64, dtype=torch.int8)
S = torch.ones(10, 2, 4)


def _attn_in(**over):
    kw = dict(q=torch.zeros(2, 1, 4, 64).bfloat16(), k_cache=I8, v_cache=I8, page_table=torch.zeros(2, 4, dtype=torch.int32),
              lens=torch.zeros(2, dtype=torch.int32), k_scale=S, v_scale=S)
    return dict(kw, **over)


def _append_in(**over):
    kw = dict(_attn_in(**over), k=torch.zeros(2, 1, 2, 64).bfloat16(), v=torch.zeros(2, 1, 2, 64).bfloat16())
    kw.pop("q")
    return kw


def _read_in(**over):
    kw = _attn_in(**over)
    kw.pop("q")
    return dict(dict(kw, tokens=3), **{k: v for k, v in over.items() if k == "tokens"})


BAD_SCALES = [
    dict(k_scale=None), dict(v_scale=None), dict(k_scale=None, v_scale=None),
    dict(k_scale=torch.ones(2), v_scale=torch.ones(2)),                     # a factor a head for int8
    dict(k_cache=E4, v_cache=E4, k_scale=torch.ones(2)),                    # one of each kind
    dict(k_scale=torch.ones(10, 2, 3), v_scale=torch.ones(10, 2, 3)),       # 3 does not divide 16
    dict(k_scale=torch.ones(10, 2, 0), v_scale=torch.ones(10, 2, 0)),
    dict(k_scale=torch.ones(9, 2, 4)), dict(v_scale=torch.ones(10, 4, 2)), dict(v_scale=torch.ones(10, 2, 2)),
    dict(k_scale=S.double()), dict(k_scale=S.bfloat16()), dict(k_scale=torch.ones(10, 4, 2).transpose(1, 2)),
    dict(k_cache=I8.bfloat16(), v_cache=I8.bfloat16()), dict(v_cache=E4), dict(k_cache=I8.to(torch.uint8), v_cache=I8.to(torch.uint8)),
]


@pytest.mark.parametrize("over", BAD_SCALES)
def test_binding_refuses_scales(over):
    for f, make in ((gdn.attn_decode_args, _attn_in), (gdn.kv_append_args, _append_in), (gdn.kv_read_args, _read_in)):
        with pytest.raises(ValueError):
            f(**make(**over))


def test_binding_passes_block_scales():
    for cache, code in ((I8, 3), (E4, 2)):
        for f, make in ((gdn.attn_decode_args, _attn_in), (gdn.kv_append_args, _append_in), (gdn.kv_read_args, _read_in)):
            a = f(**make(k_cache=cache, v_cache=cache))[0]
            assert (a.cache_dtype, a.scale_block, a.k_scale, a.k_block_scale) == (code, 4, None, S.data_ptr())
    a = gdn.attn_decode_args(**_attn_in(k_cache=E4, v_cache=E4, k_scale=torch.ones(2), v_scale=torch.ones(2)))[0]
    assert a.scale_block == 0 and a.k_scale and not a.k_block_scale


@pytest.mark.parametrize("over", [
    dict(tokens=-1), dict(tokens=1.5), dict(dtype=torch.float16), dict(lens=torch.zeros(2, 1)), dict(lens=torch.zeros(2)),
    dict(cu_seqlens=torch.zeros(2, dtype=torch.int32)), dict(k_cache=I8[0]), dict(page_table=torch.zeros(3, 4, dtype=torch.int32)),
    dict(out=(torch.zeros(2, 3, 2, 64), torch.zeros(2, 3, 2, 32))), dict(out=(torch.zeros(2, 2, 3, 64).transpose(1, 2),) * 2),
    dict(out=(torch.zeros(2, 3, 2, 64), torch.zeros(2, 3, 2, 64).bfloat16())), dict(out=(torch.zeros(2, 3, 2, 64),)),
    dict(out=(torch.zeros(2, 3, 2, 64),) * 2), dict(out=()),
])
def test_kv_read_args_refuse(over):
    kw = dict(k_cache=I8, v_cache=I8, page_table=torch.zeros(2, 4, dtype=torch.int32), lens=torch.zeros(2, dtype=torch.int32),
              tokens=3, k_scale=S, v_scale=S)
    with pytest.raises(ValueError):
        gdn.kv_read_args(**dict(kw, **over))


def test_kv_read_args_shapes():
    kw = dict(_attn_in())
    kw.pop("q")
    a, _, out = gdn.kv_read_args(tokens=3, **kw)
    assert a.total_tokens == 6 and out[0].shape == (2, 3, 2, 64) and out[0].dtype == torch.bfloat16 and a.zero_rest
    a, _, out = gdn.kv_read_args(tokens=5, cu_seqlens=torch.tensor([0, 2, 5]), dtype=torch.float32, **kw)
    assert a.total_tokens == 5 and out[1].shape == (5, 2, 64) and out[1].dtype == torch.float32 and a.cu_seqlens
    given = tuple(torch.zeros(5, 2, 64) for _ in range(2))
    a, _, out = gdn.kv_read_args(tokens=5, cu_seqlens=torch.tensor([0, 2, 5]), out=given, **kw)
    assert out[0] is given[0] and not a.zero_rest


def test_batches_of_no_rows_read_and_turn_to_zeros():
    none, cu = torch.zeros(0, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    _, _, out = gdn.kv_read_args(I8, I8, torch.zeros(0, 4, dtype=torch.int32), none, 5, cu_seqlens=cu, k_scale=S, v_scale=S)
    assert all(t.shape == (5, 2, 64) and (t == 0).all() for t in out)
    _, _, out = gdn.rope_args(torch.ones(5, 2, 64), None, F, lens=none, cu_seqlens=cu)
    assert (out[0] == 0).all()
    # one output given, one new: the new one's tokens of no row are zeros
    q, k = torch.ones(5, 2, 64), torch.ones(5, 1, 64)
    a, _, out = gdn.rope_args(q, k, F, lens=none[:0].new_zeros(1), cu_seqlens=torch.tensor([0, 2]), out=(q, None))
    assert out[0] is q and (out[1] == 0).all() and not a.zero_rest


Q, K, F = torch.zeros(2, 3, 4, 64), torch.zeros(2, 3, 2, 64), torch.ones(16, dtype=torch.float64)
LENS = torch.zeros(2, dtype=torch.int32)


@pytest.mark.parametrize("over", [
    dict(q=Q.half(), k=K.half()), dict(q=Q[0, 0]), dict(k=K.bfloat16()), dict(k=K[0]), dict(k=K[:, :2]), dict(k=torch.zeros(2, 3, 2, 32)),
    dict(inv_freq=torch.ones(0).double()), dict(inv_freq=torch.ones(33).double()), dict(inv_freq=F.half()), dict(inv_freq=F[None]),
    dict(lens=None), dict(positions=torch.zeros(2, 3, dtype=torch.int32)), dict(lens=LENS[:1]), dict(lens=LENS.float()),
    dict(lens=LENS[None]), dict(lens=None, positions=torch.zeros(6, dtype=torch.int32)), dict(lens=None, positions=torch.zeros(2, 3)),
    dict(cu_seqlens=torch.zeros(3, dtype=torch.int32)), dict(q=Q[0], k=K[0]),
    dict(lens=None, positions=torch.zeros(2, 3, dtype=torch.int64), cu_seqlens=torch.zeros(3, dtype=torch.int32)),
    dict(out=(Q[:1], K)), dict(out=(Q.bfloat16(), K)), dict(out=(torch.zeros(1, 3, 4, 64).expand(2, 3, 4, 64), K)),
    dict(out=(torch.zeros(2, 3, 64, 4).transpose(2, 3), K)), dict(out=(Q,)), dict(out=()),
])
def test_rope_args_refuse(over):
    with pytest.raises(ValueError):
        gdn.rope_args(**dict(dict(q=Q, k=K, inv_freq=F, lens=LENS), **over))


def test_rope_args_layouts():
    a, _, (q, k) = gdn.rope_args(Q, K, F, lens=LENS)
    assert (a.total_tokens, a.batch, a.hq, a.hkv, a.d, a.rot, a.q_stride_token, a.k_stride_head) == (6, 2, 4, 2, 64, 32, 256, 64)
    fused = torch.zeros(6, 8 * 64)
    q, k = fused[:, :256].view(6, 4, 64), fused[:, 256:384].view(6, 2, 64)
    a, _, out = gdn.rope_args(q, k, F, lens=LENS, cu_seqlens=torch.tensor([0, 4, 6]), out=(q, k))
    assert a.q == a.q_out == fused.data_ptr() and a.q_stride_token == a.qo_stride_token == 512 and not a.zero_rest
    a, _, out = gdn.rope_args(q, None, F.float(), positions=torch.zeros(6, dtype=torch.int64))
    assert out[1] is None and a.hkv == 0 and not a.k and a.positions_i64 == 1 and a.rot == 32 and a.zero_rest
    # a step of a sequence-first buffer: tokens of the rows one stride apart
    step = torch.zeros(3, 5, 4, 64)[1][:, None]
    assert gdn.rope_args(step, None, F, lens=torch.zeros(5, dtype=torch.int32))[0].q_stride_token == 256
    # rows that are not one stride apart are copied, and refused in place
    cut = torch.zeros(2, 5, 4, 64)[:, :3]
    a, keep, _ = gdn.rope_args(cut, None, F, lens=LENS)
    assert a.q != cut.data_ptr() and a.q_stride_token == 256
    with pytest.raises(ValueError):
        gdn.rope_args(cut, None, F, lens=LENS, out=(cut, None))


def test_cpu_tensors_are_refused():
    for call in (lambda: gdn.rope(Q, K, F, lens=LENS), lambda: gdn.kv_read(tokens=3, **{k: v for k, v in _attn_in().items() if k != "q"}),
                 lambda: gdn.kv_append(**_append_in())):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_frequencies():
    f, m = gdn.rope_frequencies(64)
    assert f.dtype == torch.float64 and m == 1.0 and f[0] == 1.0
    assert all(abs(float(f[i]) - 10000.0 ** (-2 * i / 64)) < 1e-15 for i in range(32))
    g, m = gdn.rope_frequencies(64, scaling="linear", scale=4)
    assert m == 1.0 and torch.equal(g, f / 4)
    g, m = gdn.rope_frequencies(64, scaling="base", scale=4)  # the fastest as before, the slowest a quarter
    assert m == 1.0 and g[0] == 1.0 and abs(float(g[-1] / f[-1]) - 0.25) < 1e-12
    g, m = gdn.rope_frequencies(64, scaling="parts", scale=8, trained=4096, slow=1, fast=32)
    assert abs(m - (0.1 * math.log(8) + 1)) < 1e-15
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(g[turns >= 32], f[turns >= 32]) and torch.allclose(g[turns <= 1], f[turns <= 1] / 8, rtol=1e-15)
    mid = (turns > 1) & (turns < 32)
    keep = (turns[mid] - 1) / 31
    assert mid.any() and torch.allclose(g[mid], f[mid] * keep + f[mid] / 8 * (1 - keep), rtol=1e-14)
    assert torch.equal(gdn.rope_frequencies(64, scaling="parts", scale=1, trained=4096)[0], f)
    assert gdn.rope_frequencies(2, scaling="base", scale=4)[0].tolist() == [1.0]
    for bad in (dict(rot=3), dict(rot=0), dict(rot=64, base=0), dict(rot=64, scaling="parts", scale=2), dict(rot=64, scaling="x"),
                dict(rot=64, scale=0), dict(rot=64, scaling="parts", trained=10, slow=2, fast=2)):
        with pytest.raises(ValueError):
            gdn.rope_frequencies(**bad)


def test_the_short_way_has_no_thread_locals():
    """One in a library that is loaded late slows every other library's thread-locals down."""
    import subprocess
    path = os.path.join(os.path.dirname(L.__file__), "_calls.so")
    out = subprocess.run(["readelf", "-lW", path], check=True, capture_output=True, text=True).stdout
    assert " TLS " not in out and "LOAD" in out
    assert L.calls().rope
