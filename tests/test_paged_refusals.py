"""More refusals of the paged-cache calls and of rope on the host (no GPU needed)."""
import ctypes

import pytest

import gated_deltanet_state_delta_amd._lib as L
from test_block_scales_abi import BLOCKS, _read, _rope
from test_paged_abi import FAKE, _attn

LONG = dict(batch=1, max_pages=1000, page_table_stride=1000)


@pytest.mark.parametrize("over", [
    dict(scale_block=-8), dict(scale_block=5), dict(scale_block=32), dict(cache_dtype=1), dict(cache_dtype=1, scale_block=-1),
    dict(page_size=1 << 17, scale_block=1 << 17),
])
def test_the_workspace_of_a_scale_block_that_the_call_refuses_is_0(over):
    lib = L.load()
    assert lib.gdn_attn_decode_workspace_size(ctypes.byref(_attn(**{**LONG, **BLOCKS}))) > 0
    a = _attn(**{**LONG, **BLOCKS, **over})
    assert lib.gdn_attn_decode(ctypes.byref(a), None) in (2, 5)
    assert lib.gdn_attn_decode_workspace_size(ctypes.byref(a)) == 0


@pytest.mark.parametrize("over", [
    dict(qo_stride_token=64), dict(qo_stride_token=383), dict(qo_stride_token=0), dict(qo_stride_head=0), dict(qo_stride_head=63),
    dict(ko_stride_token=0), dict(ko_stride_head=32, ko_stride_token=96), dict(ko_stride_head=511, ko_stride_token=64),
    dict(total_tokens=1, batch=1, qo_stride_head=8),
    dict(q_out=FAKE, q_stride_token=0, qo_stride_token=0), dict(k_out=FAKE * 2, k_stride_head=0, ko_stride_head=0),  # in place
])
def test_rope_refuses_outputs_whose_rows_overlap(over):
    """Threads would write one place with different values."""
    lib = L.load()
    assert lib.gdn_rope(ctypes.byref(_rope(**over)), None) == 4, lib.gdn_last_error()
    assert b"overlap" in lib.gdn_last_error()


@pytest.mark.parametrize("at,stride", [(300, 768), (383, 768), (385, 768), (400, 700), (768 + 300, 768), (-300, 768), (384, 767)])
def test_rope_refuses_slices_that_overlap(at, stride):
    """Queries of 6 heads of 64 in rows of `stride`, their output `at` elements behind them."""
    a = _rope(q_stride_token=stride, qo_stride_token=stride, q_out=FAKE + 2 * at)
    assert L.load().gdn_rope(ctypes.byref(a), None) == 4 and b"overlap" in L.load().gdn_last_error()


@pytest.mark.parametrize("over", [
    dict(k_stride_token=0), dict(v_stride_token=0), dict(k_stride_head=0), dict(v_stride_head=32), dict(k_stride_token=64),
    dict(v_stride_token=64, v_stride_head=192), dict(total_tokens=1, batch=1, v_stride_head=56),
])
def test_kv_read_refuses_outputs_whose_rows_overlap(over):
    lib = L.load()
    assert lib.gdn_kv_read(ctypes.byref(_read(**over)), None) == 4, lib.gdn_last_error()
    assert b"overlap" in lib.gdn_last_error()
