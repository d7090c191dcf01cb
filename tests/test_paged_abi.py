"""Refusals of the paged-cache calls on the host (no GPU needed): the C ABI's
argument checks and the binding's shape checks, before anything is launched."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import gated_deltanet_state_delta_amd as gdn
import gated_deltanet_state_delta_amd._lib as L

FAKE = 0x10000
HERE = os.path.dirname(os.path.abspath(__file__))


def _set(a, over):
    for k, v in over.items():
        setattr(a, k, v)
    return a


def _attn(**over):
    a = L.AttnDecodeArgs()
    a.batch, a.T, a.hq, a.hkv, a.d, a.io_dtype, a.cache_dtype, a.scale = 4, 2, 8, 2, 64, 1, 1, 0.125
    a.q, a.q_stride_row, a.q_stride_token, a.q_stride_head = FAKE, 1024, 512, 64
    a.k_cache, a.k_stride_page, a.k_stride_token, a.k_stride_head = FAKE * 2, 2048, 128, 64
    a.v_cache, a.v_stride_page, a.v_stride_token, a.v_stride_head = FAKE * 3, 2048, 128, 64
    a.n_pages, a.page_size, a.max_pages, a.page_table_stride = 10, 16, 4, 4
    a.page_table, a.lens, a.out = FAKE * 4, FAKE * 5, FAKE * 6
    return _set(a, over)


def _append(**over):
    a = L.KvAppendArgs()
    a.total_tokens, a.batch, a.hkv, a.d, a.io_dtype, a.cache_dtype = 8, 4, 2, 64, 1, 1
    a.k, a.k_stride_token, a.k_stride_head = FAKE, 128, 64
    a.v, a.v_stride_token, a.v_stride_head = FAKE * 7, 128, 64
    a.k_cache, a.kc_stride_page, a.kc_stride_token, a.kc_stride_head = FAKE * 2, 2048, 128, 64
    a.v_cache, a.vc_stride_page, a.vc_stride_token, a.vc_stride_head = FAKE * 3, 2048, 128, 64
    a.n_pages, a.page_size, a.max_pages, a.page_table_stride = 10, 16, 4, 4
    a.page_table, a.lens = FAKE * 4, FAKE * 5
    return _set(a, over)


CACHE_ERRORS = [
    (dict(io_dtype=2), 3), (dict(io_dtype=7), 3), (dict(cache_dtype=0), 3), (dict(cache_dtype=5), 3),
    (dict(cache_dtype=2), 1),                                   # e4m3 without scales
    (dict(cache_dtype=2, k_scale=FAKE), 1),
    (dict(k_scale=FAKE, v_scale=FAKE), 2),                      # scales without e4m3
    (dict(batch=-1), 2), (dict(hkv=0), 2), (dict(n_pages=-1), 2), (dict(page_size=0), 2), (dict(max_pages=-1), 2),
    (dict(d=48), 5), (dict(d=16), 5), (dict(d=512), 5),
    (dict(max_pages=1 << 20, page_table_stride=1 << 20, page_size=1025), 5),
    (dict(page_table_stride=3), 4),
    (dict(page_table=None), 1), (dict(lens=None), 1), (dict(k_cache=None), 1), (dict(v_cache=None), 1),
    (dict(k_cache=FAKE + 8), 4), (dict(v_cache=FAKE + 2), 4),
]


@pytest.mark.parametrize("over,status", CACHE_ERRORS + [
    (dict(T=0), 2), (dict(T=65), 5), (dict(hq=0), 2), (dict(hq=7), 2), (dict(hq=1 << 17), 5),
    (dict(batch=1 << 20, hq=1 << 12), 5), (dict(batch=1 << 23, hkv=8), 5),
    (dict(q=None), 1), (dict(out=None), 1), (dict(q=FAKE + 4), 4), (dict(out=FAKE + 8), 4),
    (dict(q_stride_token=516), 4), (dict(q_stride_row=-8), 4),
    (dict(k_stride_token=60), 4), (dict(k_stride_token=132), 4), (dict(k_stride_token=1 << 23), 4),
    (dict(k_stride_head=32), 4), (dict(k_stride_token=64, k_stride_head=128), 4),  # overlapping rows
    (dict(v_stride_page=1024), 4), (dict(v_stride_page=2052), 4), (dict(k_stride_page=-2048), 4),
    (dict(workspace=FAKE + 16, workspace_bytes=1 << 30), 4),
    (dict(out=FAKE), 4), (dict(out=FAKE + 1024), 4),                              # over q
    (dict(batch=1 << 17, max_pages=1 << 26, page_table_stride=1 << 26), 5),       # positions of all rows
])
def test_attn_decode_refuses(over, status):
    assert L.load().gdn_attn_decode(ctypes.byref(_attn(**over)), None) == status, L.load().gdn_last_error()
    assert b"gdn_attn_decode" in L.load().gdn_last_error()


@pytest.mark.parametrize("over,status", CACHE_ERRORS + [
    (dict(total_tokens=-1), 2), (dict(total_tokens=7), 2), (dict(total_tokens=(1 << 28) + 4), 5),
    (dict(hkv=1 << 17), 5), (dict(k=None), 1), (dict(v=None), 1), (dict(k=FAKE + 2), 4),
    (dict(k_stride_token=100), 4), (dict(v_stride_head=-64), 4),
    (dict(kc_stride_token=60), 4), (dict(vc_stride_head=1 << 23), 4), (dict(kc_stride_page=2000), 4),
])
def test_kv_append_refuses(over, status):
    assert L.load().gdn_kv_append(ctypes.byref(_append(**over)), None) == status, L.load().gdn_last_error()
    assert b"gdn_kv_append" in L.load().gdn_last_error()


def test_calls_with_nothing_to_do_return_without_a_launch():
    lib = L.load()
    assert lib.gdn_attn_decode(ctypes.byref(_attn(batch=0)), None) == 0
    for over in (dict(batch=0), dict(total_tokens=0), dict(n_pages=0), dict(max_pages=0)):
        assert lib.gdn_kv_append(ctypes.byref(_append(**over)), None) == 0
    assert lib.gdn_pages_copy(None, 64, 64, 4, None, None, 0, None) == 0
    assert lib.gdn_pages_copy(None, 0, 0, 4, None, None, 3, None) == 0
    for name in ("gdn_attn_decode", "gdn_kv_append"):
        assert getattr(lib, name)(None, None) == 1


def test_workspace_depends_on_sizes_alone():
    f = L.load().gdn_attn_decode_workspace_size
    one = f(ctypes.byref(_attn(batch=1, max_pages=1000, page_table_stride=1000)))
    assert one > 0 and one % 4 == 0
    assert f(ctypes.byref(_attn(batch=1, max_pages=1000, page_table_stride=1000, lens=None, q=None))) == one
    assert f(ctypes.byref(_attn(batch=4096))) == 0  # tables of one step
    assert f(ctypes.byref(_attn(batch=1, max_pages=1))) == 0  # one short range
    assert f(None) == 0 and f(ctypes.byref(_attn(batch=0))) == 0


def test_pages_copy_refuses():
    f = L.load().gdn_pages_copy
    assert f(FAKE, -1, 64, 4, FAKE, FAKE, 1, None) == 2
    assert f(FAKE, 64, 64, -4, FAKE, FAKE, 1, None) == 2
    assert f(FAKE, 64, 64, 4, FAKE, FAKE, -1, None) == 2
    assert f(FAKE, 64, 63, 4, FAKE, FAKE, 1, None) == 4
    assert f(FAKE, 64, 64, 4, FAKE, FAKE, 1 << 31, None) == 5
    assert f(FAKE, 1 << 40, 1 << 40, 4, FAKE, FAKE, 1, None) == 5
    for args in ((None, FAKE, FAKE), (FAKE, None, FAKE), (FAKE, FAKE, None)):
        assert f(args[0], 64, 64, 4, args[1], args[2], 1, None) == 1


def _pages(**over):
    a = L.PagesArgs()
    a.rows, a.max_pages, a.n_pages, a.page_size = 4, 5, 20, 16
    a.page_table, a.page_table_stride, a.lens, a.refs = FAKE, 5, FAKE * 2, FAKE * 3
    a.page_table_out, a.page_table_out_stride, a.lens_out, a.refs_out = FAKE * 4, 5, FAKE * 5, FAKE * 6
    a.workspace, a.workspace_bytes = FAKE * 7, L.load().gdn_pages_workspace_size(4, 20)
    return _set(a, over)


PAGES_CALLS = {"extend": (FAKE * 8, FAKE * 9), "fork": (FAKE * 8, FAKE * 9, FAKE * 10), "free": (FAKE * 8,),
               "compact": (FAKE * 8, FAKE * 9, FAKE * 10)}


@pytest.mark.parametrize("call", sorted(PAGES_CALLS))
def test_page_table_calls_refuse(call):
    lib = L.load()
    f, args = getattr(lib, "gdn_pages_" + call), PAGES_CALLS[call]
    errors = [(dict(rows=-1), 2), (dict(max_pages=0), 2), (dict(n_pages=0), 2), (dict(page_size=0), 2),
              (dict(n_pages=(1 << 24) + 1), 5), (dict(rows=(1 << 20) + 1), 5), (dict(page_size=1 << 29), 5),
              (dict(page_table_stride=4), 4), (dict(page_table_out_stride=4), 4), (dict(refs=None), 1),
              (dict(refs_out=None), 1), (dict(page_table=None), 1), (dict(page_table_out=None), 1),
              (dict(page_table_out=FAKE, page_table_out_stride=6), 4)]
    if call != "compact":
        errors += [(dict(lens=None), 1), (dict(lens_out=None), 1)]
    if call != "free":
        errors += [(dict(workspace=None), 1), (dict(workspace=FAKE + 4), 4), (dict(workspace_bytes=100), 2)]
    if call == "fork":
        errors += [(dict(page_table_out=FAKE), 4), (dict(page_table_out=FAKE + 40), 4), (dict(lens_out=FAKE * 2), 4)]
    for over, status in errors:
        assert f(ctypes.byref(_pages(**over)), *args, None) == status, (over, lib.gdn_last_error())
        assert ("gdn_pages_" + call).encode() in lib.gdn_last_error()
    for i in range(len(args)):
        assert f(ctypes.byref(_pages()), *(None if j == i else x for j, x in enumerate(args)), None) == 1
    assert f(None, *args, None) == 1


# ------------------------------------------------------------ the binding --


def _inputs(**over):
    x = dict(q=torch.zeros(2, 1, 4, 64), k_cache=torch.zeros(3, 16, 2, 64), v_cache=torch.zeros(3, 16, 2, 64),
             page_table=torch.zeros(2, 5, dtype=torch.int32), lens=torch.zeros(2, dtype=torch.int32))
    x.update(over)
    return x


E4 = torch.zeros(3, 16, 2, 64).to(torch.float8_e4m3fn)


@pytest.mark.parametrize("over", [
    dict(q=torch.zeros(2, 4, 64)), dict(q=torch.zeros(2, 1, 4, 64).half()), dict(q=torch.zeros(2, 1, 4, 32)),
    dict(k_cache=torch.zeros(3, 16, 64)), dict(v_cache=torch.zeros(3, 8, 2, 64)), dict(k_cache=torch.zeros(3, 16, 2, 64).bfloat16()),
    dict(v_cache=torch.zeros(3, 16, 2, 64).bfloat16()), dict(k_cache=torch.zeros(3, 0, 2, 64), v_cache=torch.zeros(3, 0, 2, 64)),
    dict(page_table=torch.zeros(3, 5, dtype=torch.int32)), dict(page_table=torch.zeros(2, 5)), dict(lens=torch.zeros(3, dtype=torch.int32)),
    dict(lens=torch.zeros(2)), dict(k_scale=torch.ones(2), v_scale=torch.ones(2)), dict(k_cache=E4, v_cache=E4),
    dict(k_cache=E4, v_cache=E4, k_scale=torch.ones(2), v_scale=torch.ones(3)),
    dict(k_cache=E4, v_cache=E4, k_scale=torch.ones(2).double(), v_scale=torch.ones(2)),
    dict(out=torch.zeros(2, 1, 4, 32)), dict(out=torch.zeros(2, 1, 4, 64).bfloat16()), dict(out=torch.zeros(2, 1, 4, 128)[..., :64]),
    dict(lse=torch.zeros(2, 4)), dict(k_cache=torch.zeros(3, 16, 64, 2).transpose(2, 3), v_cache=torch.zeros(3, 16, 2, 64)),
])
def test_attn_decode_args_refuse(over):
    with pytest.raises(ValueError):
        gdn.attn_decode_args(**_inputs(**over))


def test_attn_decode_args_layouts():
    """Strides as given, copies only where the kernel cannot read in place."""
    a, keep, out = gdn.attn_decode_args(**_inputs())
    assert (a.k_stride_page, a.k_stride_token, a.k_stride_head, a.hkv, a.page_size) == (2048, 128, 64, 2, 16)
    assert out.shape == (2, 1, 4, 64) and abs(a.scale - 0.125) < 1e-9
    hf = torch.zeros(3, 2, 16, 64).transpose(1, 2)
    a, keep, _ = gdn.attn_decode_args(**_inputs(k_cache=hf))
    assert (a.k_stride_token, a.k_stride_head, a.k_cache) == (64, 1024, hf.data_ptr())
    wide = torch.zeros(2, 1, 9, 64)[:, :, :4]
    a, keep, _ = gdn.attn_decode_args(**_inputs(q=wide))
    assert a.q == wide.data_ptr() and a.q_stride_row == 576
    odd = torch.zeros(2, 1, 4 * 65)[..., :260].view(2, 1, 4, 65)[..., :64]
    a, keep, _ = gdn.attn_decode_args(**_inputs(q=odd))
    assert a.q != odd.data_ptr() and a.q_stride_head == 64
    t = torch.zeros(2, 9, dtype=torch.int32)[:, :5]
    a, keep, _ = gdn.attn_decode_args(**_inputs(page_table=t))
    assert a.page_table == t.data_ptr() and a.page_table_stride == 9


@pytest.mark.parametrize("over", [
    dict(k=torch.zeros(2, 64), v=torch.zeros(2, 64)), dict(k=torch.zeros(3, 1, 2, 64), v=torch.zeros(3, 1, 2, 64)),
    dict(v=torch.zeros(2, 1, 2, 32)), dict(v=torch.zeros(2, 1, 2, 64).bfloat16()), dict(k=torch.zeros(2, 1, 2, 64).half(), v=torch.zeros(2, 1, 2, 64).half()),
    dict(cu_seqlens=torch.zeros(3, dtype=torch.int32)), dict(k=torch.zeros(4, 2, 64), v=torch.zeros(4, 2, 64), cu_seqlens=torch.zeros(2, dtype=torch.int32)),
    dict(k=torch.zeros(2, 1, 3, 64), v=torch.zeros(2, 1, 3, 64)), dict(lens=torch.zeros(2, 1, dtype=torch.int32)),
])
def test_kv_append_args_refuse(over):
    x = _inputs(k=torch.zeros(2, 1, 2, 64), v=torch.zeros(2, 1, 2, 64))
    x.pop("q")
    x.update(over)
    with pytest.raises(ValueError):
        gdn.kv_append_args(**x)


def test_pages_args_refuse():
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    t, n, f = i32(4, 5), i32(4), i32(9)
    for bad in ((i32(4), n, f), (i32(4, 0), n, f), (t, i32(3), f), (t, n, i32(0)), (t, n, i32(3, 3)), (t.float(), n, f),
                (t, n.float(), f)):
        with pytest.raises(ValueError):
            gdn.pages_args(*bad, 16)
    for out in ((i32(4, 6), i32(4), i32(9)), (i32(4, 5), i32(4), f.long()), (i32(5, 4).t(), i32(4), i32(9)),
                (i32(1, 5).expand(4, 5), i32(4), i32(9))):
        with pytest.raises(ValueError):
            gdn.pages_args(t, n, f, 16, out)
    gdn.pages_args(t, n, f, 16, (t, n, f))
    with pytest.raises(ValueError):
        gdn.pages_args(t, n, f, 16, (t, n, f), apart=True)
    gdn.pages_args(t, n, f, 16, (i32(4, 5), i32(4), f), apart=True)
    big = i32(30)
    with pytest.raises(ValueError):  # shifted by one entry
        gdn.pages_args(big[:20].view(4, 5), n, f, 16, (big[1:21].view(4, 5), i32(4), i32(9)))


def test_cpu_tensors_are_refused():
    x = _inputs()
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    kv = torch.zeros(2, 1, 2, 64)
    for call in (lambda: gdn.attn_decode(**x),
                 lambda: gdn.kv_append(kv, kv, x["k_cache"], x["v_cache"], x["page_table"], x["lens"]),
                 lambda: gdn.pages_copy(x["k_cache"], i32(1), i32(1)),
                 lambda: gdn.pages_extend(i32(2, 3), i32(2), i32(5), i32(2), 16),
                 lambda: gdn.pages_fork(i32(2, 3), i32(2), i32(5), i32(2), 16),
                 lambda: gdn.pages_free(i32(2, 3), i32(2), i32(5), i32(2).bool(), 16),
                 lambda: gdn.pages_compact(i32(2, 3), i32(5))):
        with pytest.raises(ValueError):
            call()


def _with_strides(t, *strides):
    """t's values with the strides of its dimensions of one entry replaced
    (None: as they are); still contiguous to torch."""
    t = torch.as_strided(t, t.shape, [s if n == 1 and s is not None else st for n, s, st in zip(t.shape, strides, t.stride())])
    assert t.is_contiguous()
    return t


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("rows,hkv", [(64, 4), (1, 4), (5, 1), (1, 1)])
def test_kv_append_args_read_the_tokens_where_they_are(rows, hkv, packed):
    """Dimensions of one entry carry any stride, also in a contiguous tensor: a
    step of a sequence-first buffer is one, and its token stride is the rows'."""
    d, dense = 64, (hkv * 64, 64)
    steps = torch.zeros(3, rows, hkv, d)
    if packed:
        inputs = [torch.zeros(rows, hkv, d), _with_strides(torch.zeros(rows, hkv, d), 7, 13, 1)]
    else:
        inputs = [torch.zeros(rows, 1, hkv, d), steps[:1].transpose(0, 1), steps[1:2].transpose(0, 1),
                  torch.zeros(1, rows, hkv, d).transpose(0, 1), _with_strides(torch.zeros(rows, 1, hkv, d), 7, 7, 13, 1)]
    cache = torch.zeros(9, 16, hkv, d)
    x = dict(k_cache=cache, v_cache=cache.clone(), page_table=torch.zeros(rows, 4, dtype=torch.int32),
             lens=torch.zeros(rows, dtype=torch.int32), cu_seqlens=torch.arange(rows + 1, dtype=torch.int32) if packed else None)
    for k in inputs:
        for v in inputs:
            a, keep = gdn.kv_append_args(k, v, **x)
            assert (a.k, a.v, a.total_tokens) == (k.data_ptr(), v.data_ptr(), rows)
            assert (a.k_stride_token, a.k_stride_head) == dense and (a.v_stride_token, a.v_stride_head) == dense


def _alone(code):
    """Runs code, which prints one number, in a process of its own: a call
    that never returns or ends its process fails this test alone."""
    head = "import ctypes, sys; sys.path[:0] = %r\nimport gated_deltanet_state_delta_amd._lib as L\n" \
           "from test_paged_abi import _append, _attn\nlib = L.load()\n" % [HERE, os.path.dirname(HERE)]
    res = subprocess.run([sys.executable, "-c", head + code], capture_output=True, text=True, timeout=100,
                         env=dict(os.environ, HIP_VISIBLE_DEVICES=""))
    assert res.returncode == 0, (res.returncode, res.stderr[-500:])
    return [int(x) for x in res.stdout.split()]


@pytest.mark.parametrize("page_size", [(1 << 30) + 1, (1 << 31) - 1])
def test_page_sizes_past_their_limit_are_refused(page_size):
    """Also where a table of no entries holds no positions."""
    code = "for f, make in ((lib.gdn_attn_decode, _attn), (lib.gdn_kv_append, _append)):\n" \
           "    for over in (dict(max_pages=0), dict(max_pages=0, n_pages=0), dict()):\n" \
           "        print(f(ctypes.byref(make(page_size=%d, **over)), None))" % page_size
    assert _alone(code) == [5] * 6


def test_workspace_size_of_refused_sizes_is_zero():
    """Sizes that gdn_attn_decode refuses need no workspace, and asking for one
    ends no process."""
    sizes = [dict(d=1 << 30, io_dtype=0, cache_dtype=0), dict(d=1 << 30), dict(d=1 << 28), dict(d=48), dict(d=(1 << 31) - 1),
             dict(T=65536, hq=65536, hkv=1), dict(T=1 << 30), dict(T=65), dict(hq=1 << 30, T=4, hkv=1), dict(hq=7),
             dict(page_size=(1 << 31) - 1, max_pages=(1 << 31) - 1, batch=(1 << 31) - 1), dict(batch=1 << 23, hq=512, hkv=2)]
    code = "for over in %r:\n" \
           "    a = _attn(**dict(dict(max_pages=9999, page_table_stride=9999), **over))\n" \
           "    print(lib.gdn_attn_decode_workspace_size(ctypes.byref(a)), lib.gdn_attn_decode(ctypes.byref(a), None), flush=True)"
    got = _alone(code % sizes)
    assert got[::2] == [0] * len(sizes) and set(got[1::2]) <= {2, 5}


def test_attn_decode_args_read_queries_where_they_are():
    """A contiguous query is read with its dense strides, whatever its
    dimensions of one entry carry; others with their own."""
    lone, step = torch.zeros(1, 1, 4, 64), torch.zeros(3, 2, 4, 64)[1:2].transpose(0, 1)
    cases = [(_with_strides(lone, 7, 7, None, None), (256, 256, 64)), (step, (256, 256, 64)),
             (_with_strides(torch.zeros(2, 1, 1, 64), None, 7, 13, None), (64, 64, 64)),
             (torch.zeros(1, 2, 4, 64).transpose(1, 2).contiguous().transpose(1, 2), (512, 64, 128)),
             (_with_strides(torch.zeros(1, 5, 4, 64), 3, None, None, None), (1280, 256, 64)),
             (torch.zeros(1, 1, 9, 64)[:, :, 2:6], (256, 256, 64))]
    for q, want in cases:
        x = _inputs(q=q, page_table=torch.zeros(q.shape[0], 5, dtype=torch.int32), lens=torch.zeros(q.shape[0], dtype=torch.int32))
        if q.shape[2] == 1:
            x.update(k_cache=torch.zeros(3, 16, 1, 64), v_cache=torch.zeros(3, 16, 1, 64))
        a, keep, out = gdn.attn_decode_args(**x)
        got = (a.q_stride_row, a.q_stride_token, a.q_stride_head)
        assert a.q == q.data_ptr() and out.shape == q.shape and out.is_contiguous()
        # strides of dimensions of one entry are not used, but the library checks them
        assert all(s % 8 == 0 for s in got) and all(s == w for s, w, n in zip(got, want, q.shape) if n > 1)
        # the library takes them: the workspace, checked last, is what it refuses
        a.k_cache, a.v_cache, a.q, a.out, a.page_table, a.lens = (FAKE * 2, FAKE * 4, FAKE * 32, FAKE * 64, FAKE * 96, FAKE * 97)
        a.workspace, a.workspace_bytes = FAKE + 16, 1 << 20
        assert L.load().gdn_attn_decode(ctypes.byref(a), None) == 4
        assert b"workspace must be" in L.load().gdn_last_error()


def test_head_strides_have_room():
    """Only token strides have to stay below 2^23 elements: a heads-first page
    of 65536 tokens with heads of 128 steps 2^23 elements from head to head.
    The value cache, whose rows overlap, is what is refused."""
    lib = L.load()
    for head in (1 << 23, 1 << 33, (1 << 40) - 64):
        cache = dict(d=64, n_pages=2, page_size=16)
        attn = _attn(k_stride_token=64, k_stride_head=head, k_stride_page=2 * head, v_stride_token=64, v_stride_head=128, **cache)
        append = _append(kc_stride_token=64, kc_stride_head=head, kc_stride_page=2 * head, vc_stride_token=64, vc_stride_head=128, **cache)
        for f, a in ((lib.gdn_attn_decode, attn), (lib.gdn_kv_append, append)):
            assert f(ctypes.byref(a), None) == 4 and b"rows overlap" in lib.gdn_last_error(), lib.gdn_last_error()
    for over in (dict(k_stride_head=1 << 40, k_stride_page=1 << 42), dict(k_stride_head=(1 << 63) - 64, k_stride_page=(1 << 63) - 64)):
        assert lib.gdn_attn_decode(ctypes.byref(_attn(k_stride_token=64, **over)), None) == 4
        assert b"strides must be" in lib.gdn_last_error()
    one = torch.empty_strided((4, 1, 3, 64), (1 << 25, 1, 1 << 23, 1), device="meta")  # pages of one token
    x = _inputs(q=torch.zeros(2, 1, 3, 64), k_cache=one, v_cache=one)
    a, keep, _ = gdn.attn_decode_args(**x)
    assert (a.k_stride_page, a.k_stride_head) == (1 << 25, 1 << 23) and a.k_stride_token < 1 << 23


def test_page_sizes_that_no_int32_holds_are_refused():
    """They would reach the library as other numbers."""
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    for page_size in ((1 << 32) + 16, -(1 << 32) + 16, 1 << 31, 16.5):
        with pytest.raises(ValueError):
            gdn.pages_args(i32(4, 5), i32(4), i32(9), page_size)
    a, keep, _ = gdn.pages_args(i32(4, 5), i32(4), i32(9), torch.tensor(16))
    assert a.page_size == 16
