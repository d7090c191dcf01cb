"""gdn_attn_decode on the GPU against the 64-bit reference: every type, head
size and kind of page; ragged, empty and over-long rows; groups and several
new tokens; layouts; values that must not be seen; splits; streams, graphs."""
import ctypes

import pytest
import torch

import gated_deltanet_state_delta_amd as gdn
from gated_deltanet_state_delta_amd import _lib
from gpu_util import require_gpu
from paged_ref import DT, attn_bound, attn_ref, caches, paged, poison_unheld

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _scales(cache, hkv, seed=5):
    if cache != "e4m3":
        return None, None
    g = torch.Generator().manual_seed(seed)
    return torch.rand(hkv, generator=g) * 0.01 + 0.005, torch.rand(hkv, generator=g) * 0.01 + 0.005


def _dev(c):
    """A CPU tensor on the GPU with the same strides (a permuted view stays one)."""
    if c is None:
        return None
    order = sorted(range(c.dim()), key=lambda i: -c.stride(i))
    back = [order.index(i) for i in range(c.dim())]
    return c.permute(order).contiguous().cuda().permute(back)


def _check(q, kc, vc, table, lens, io, ks=None, vs=None, scale=None, ref=None, **kw):
    d = q.shape[-1]
    s = d ** -0.5 if scale is None else scale
    out, lse = gdn.attn_decode(q.cuda(), _dev(kc), _dev(vc), table.cuda(), lens.cuda(), scale=scale, k_scale=_dev(ks),
                               v_scale=_dev(vs), return_lse=True, **kw)
    want, want_lse, mean, size = ref or attn_ref(q, kc, vc, table, lens, s, ks, vs)
    got = out.double().cpu()
    bound = attn_bound(want, mean, size, lens, d, io)
    bad = ((got - want).abs() > bound) | got.isnan()
    assert not bad.any(), "%d values off, worst by %.2f bounds" % (bad.sum(), ((got - want).abs() / bound).max())
    lse = lse.double().cpu()
    none = want_lse == -float("inf")
    assert torch.equal(lse == -float("inf"), none)
    # the score's error, the sum's, log2 and the scaling: a few roundings of values up to |lse| + log n
    tol = 2.0 ** -24 * ((d + 16) * size[..., 0] + 32 * (want_lse.abs() + 16))
    assert ((lse - want_lse).abs()[~none] <= tol[~none]).all()
    return out


LENS = [1, 0, 2, 15, 16, 17, 63, 64, 65, 130, 257, -3]


@pytest.mark.parametrize("page", [16, 64, 1, 5, 24])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("io,cache", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "e4m3"), ("f32", "e4m3")])
def test_types_head_sizes_and_pages(io, cache, d, page):
    lens = torch.tensor(LENS, dtype=torch.int32)
    table, n_pages = paged(LENS, page, seed=d + page)
    kc, vc = caches(n_pages, page, 2, d, cache, seed=d * 7 + page)
    kc, vc = (poison_unheld(c, table, lens, page, float("nan")) for c in (kc, vc))
    q = torch.randn(len(LENS), 1, 6, d, generator=torch.Generator().manual_seed(d)).to(DT[io])
    _check(q, kc, vc, table, lens, io, *_scales(cache, 2))


@pytest.mark.parametrize("page", [16, 7])
@pytest.mark.parametrize("T,group", [(1, 1), (1, 16), (1, 20), (2, 3), (4, 8), (5, 5), (64, 1), (7, 6)])
def test_new_tokens_and_groups(T, group, page):
    lens = torch.tensor([0, 1, T - 1, T, T + 1, 40, 100, 3 * T + 50], dtype=torch.int32)
    table, n_pages = paged(lens, page, seed=T)
    kc, vc = caches(n_pages, page, 3, 64, "bf16", seed=T * 100 + group)
    kc, vc = (poison_unheld(c, table, lens, page, float("nan")) for c in (kc, vc))
    q = torch.randn(8, T, 3 * group, 64, generator=torch.Generator().manual_seed(T)).bfloat16()
    _check(q, kc, vc, table, lens, "bf16")


@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("T,group", [(1, 17), (4, 8), (3, 11), (8, 8), (16, 6), (40, 5)])
@pytest.mark.parametrize("io,cache,d", [("bf16", "bf16", 128), ("bf16", "bf16", 256), ("f32", "f32", 256),
                                        ("f32", "f32", 64), ("bf16", "e4m3", 256), ("f32", "e4m3", 128)])
def test_row_tiles(io, cache, d, T, group, page):
    """17 to 200 query rows of a key-value head: one to seven row tiles of one
    or two times 16, alone in a workgroup's waves and several to a unit."""
    lens = torch.tensor([T, 0, 30, 210], dtype=torch.int32)
    table, n_pages = paged(lens, page, seed=T)
    kc, vc = caches(n_pages, page, 2, d, cache, seed=T * 100 + group)
    kc, vc = (poison_unheld(c, table, lens, page, float("nan")) for c in (kc, vc))
    q = torch.randn(4, T, 2 * group, d, generator=torch.Generator().manual_seed(T)).to(DT[io])
    _check(q, kc, vc, table, lens, io, *_scales(cache, 2))


@pytest.mark.parametrize("page", [32, 6])
@pytest.mark.parametrize("io,cache", [("bf16", "bf16"), ("f32", "f32"), ("f32", "e4m3")])
def test_values_that_a_token_does_not_see(io, cache, page):
    """Infinite and NaN values at the later of several new tokens reach that
    token's result only."""
    lens = torch.tensor([5, 37, 130], dtype=torch.int32)
    table, n_pages = paged(lens, page)
    kc, vc = caches(n_pages, page, 2, 64, cache, seed=11)
    ks, vs = _scales(cache, 2)
    q = torch.randn(3, 4, 4, 64, generator=torch.Generator().manual_seed(3)).to(DT[io])
    clean = attn_ref(q, kc, vc, table, lens, 0.125, ks, vs)
    wide = attn_ref(q.repeat_interleave(10, 2), kc, vc, table, lens, 0.125, ks, vs)  # 80 rows of a head
    kw, vw = kc.float(), vc.float()
    for b in range(3):
        j = int(lens[b]) - 1  # the newest token: seen by token 3 alone
        e, at = int(table[b, j // page]), j % page
        vw[e, at] = float("nan") if cache == "e4m3" else float("inf")
        kw[e, at, 1] = float("nan")
    kc, vc = kw.to(kc.dtype), vw.to(vc.dtype)
    for x, ref in ((q, clean), (q.repeat_interleave(10, 2), wide)):
        out = gdn.attn_decode(x.cuda(), kc.cuda(), vc.cuda(), table.cuda(), lens.cuda(), k_scale=_dev(ks), v_scale=_dev(vs))
        got = out.double().cpu()
        bound = attn_bound(ref[0], ref[2], ref[3], lens, 64, io)
        assert ((got - ref[0]).abs() <= bound)[:, :3].all()
        assert not got[:, 3].isfinite().any()


@pytest.mark.parametrize("page", [16, 3])
def test_entries_outside_the_cache_hold_nothing(page):
    lens = torch.tensor([100, 100, 40], dtype=torch.int32)
    table, n_pages = paged(lens, page, spare=0)
    kc, vc = caches(n_pages, page, 2, 128, "bf16", seed=2)
    table[0, 1], table[0, 3], table[1] = -1, n_pages, 1 << 30
    table[2, -1] = -(1 << 31)
    q = torch.randn(3, 2, 4, 128, generator=torch.Generator().manual_seed(4)).bfloat16()
    out = _check(q, kc, vc, table, lens, "bf16")
    assert (out[1] == 0).all()


def test_lengths_past_the_table_are_clamped_and_int64_tables_do_not_wrap():
    lens = torch.tensor([1 << 30, 70], dtype=torch.int64)
    table, n_pages = paged([64, 64], 16, width=4)
    kc, vc = caches(n_pages, 16, 1, 64, "f32", seed=9)
    table = table.long()
    table[1, 0] = (1 << 32) + int(table[1, 0])  # not a page
    q = torch.randn(2, 1, 2, 64, generator=torch.Generator().manual_seed(8))
    ref = table.clone()
    ref[1, 0] = -1
    want = attn_ref(q, kc, vc, ref, torch.tensor([64, 64]), 0.125)
    out = gdn.attn_decode(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), lens.cuda())
    assert ((out.double().cpu() - want[0]).abs() <= attn_bound(want[0], want[2], want[3], [64], 64, "f32")).all()


@pytest.mark.parametrize("layout", ["heads_first", "interleaved", "slice", "strided_q"])
@pytest.mark.parametrize("page", [16, 5])
def test_layouts(layout, page):
    lens = torch.tensor([33, 7, 90], dtype=torch.int32)
    table, n_pages = paged(lens, page)
    q = torch.randn(3, 2, 6, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
    kc, vc = caches(n_pages, page, 3, 64, "bf16", seed=21, heads_first=layout == "heads_first")
    want = attn_ref(q, kc, vc, table, lens, 0.125)
    if layout == "interleaved":  # keys and values of a page in one block
        both = torch.stack([kc, vc], 1).cuda()
        k, v = both[:, 0], both[:, 1]
    elif layout == "slice":  # heads of a wider cache
        wide = torch.full((n_pages, page, 8, 64), float("nan"), dtype=torch.bfloat16)
        wide[:, :, 2:5] = kc
        k, v = wide.cuda()[:, :, 2:5], _dev(vc)
    else:
        k, v = _dev(kc), _dev(vc)
    qd = q.cuda()
    if layout == "strided_q":  # the query part of a fused projection
        qd = torch.cat([q, q[:, :, :3]], 2).cuda()[:, :, :6]
        assert not qd.is_contiguous()
    out = gdn.attn_decode(qd, k, v, table.cuda(), lens.cuda())
    assert ((out.double().cpu() - want[0]).abs() <= attn_bound(want[0], want[2], want[3], lens, 64, "bf16")).all()


@pytest.mark.parametrize("n_pages,page,hkv,heads_first", [(1, 64, 2, False), (1, 64, 1, True), (40, 1, 3, True),
                                                          (40, 1, 1, False), (5, 16, 1, True), (1, 1, 1, False)])
def test_dimensions_of_one_entry(n_pages, page, hkv, heads_first):
    """Strides of dimensions of one entry mean nothing."""
    n = n_pages * page - n_pages * page // 5
    lens = torch.tensor([n, max(n - 3, 0)], dtype=torch.int32)
    table = torch.randperm(n_pages, generator=torch.Generator().manual_seed(1)).to(torch.int32).repeat(2, 1)
    kc, vc = caches(n_pages, page, hkv, 64, "bf16", seed=3, heads_first=heads_first)
    q = torch.randn(2, 1, 2 * hkv, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
    want = attn_ref(q, kc, vc, table, lens, 0.125)
    odd = lambda c: torch.as_strided(c, c.shape, [7 if sz == 1 else st for sz, st in zip(c.shape[:3], c.stride())] + [1])
    for k, v in ((_dev(kc), _dev(vc)), (odd(_dev(kc)), odd(_dev(vc)))):
        out = gdn.attn_decode(q.cuda(), k, v, table.cuda(), lens.cuda())
        assert ((out.double().cpu() - want[0]).abs() <= attn_bound(want[0], want[2], want[3], lens, 64, "bf16")).all()


@pytest.mark.parametrize("page,d,hkv", [(16, 128, 1), (64, 64, 2), (5, 128, 1), (1, 256, 1)])
@pytest.mark.parametrize("io,cache", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "e4m3")])
def test_split_rows(io, cache, page, d, hkv):
    """Few rows: the length is split and joined; without a workspace one
    workgroup walks each row.  Both match, and the split is repeatable."""
    lens = torch.tensor([3001, 1, 0, 129, 1024], dtype=torch.int32)
    table, n_pages = paged(lens, page, seed=3)
    kc, vc = caches(n_pages, page, hkv, d, cache, seed=5)
    ks, vs = _scales(cache, hkv)
    q = torch.randn(5, 1, 4 * hkv, d, generator=torch.Generator().manual_seed(2)).to(DT[io])
    ref = attn_ref(q, kc, vc, table, lens, d ** -0.5, ks, vs)
    assert gdn.attn_decode_workspace_size(q, kc, vc, table, lens, k_scale=ks, v_scale=vs) > 0
    out = _check(q, kc, vc, table, lens, io, ks, vs, ref=ref)
    again = _check(q, kc, vc, table, lens, io, ks, vs, ref=ref)
    assert torch.equal(out, again)
    a, keep, one = gdn.attn_decode_args(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), lens.cuda(), k_scale=_dev(ks),
                                        v_scale=_dev(vs))
    _lib.check(_lib.load().gdn_attn_decode(ctypes.byref(a), torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    bound = attn_bound(ref[0], ref[2], ref[3], lens, d, io)
    assert ((one.double().cpu() - ref[0]).abs() <= bound).all()


@pytest.mark.parametrize("page", [16, 9])
@pytest.mark.parametrize("T,rows,hkv,most", [(1, 70, 64, 200), (3, 131, 32, 150), (1, 3, 64, 2500)])
def test_shares_of_many_rows(T, rows, hkv, most, page):
    """Many heads leave few shares: one ends a row, takes whole ones (empty
    ones among them) and begins another, and long rows lie in several."""
    r = torch.Generator().manual_seed(rows)
    lens = torch.randint(0, most, (rows,), generator=r).to(torch.int32)
    lens[rows // 2] = 0
    table, n_pages = paged(lens, page, seed=rows)
    kc, vc = caches(n_pages, page, hkv, 32, "f32", seed=rows)
    q = torch.randn(rows, T, hkv, 32, generator=r)
    _check(q, kc, vc, table, lens, "f32")


@pytest.mark.parametrize("rows", [4096, 4097])
def test_batches_of_thousands(rows):
    """The largest batch that is dealt out in shares, and one more."""
    r = torch.Generator().manual_seed(rows)
    lens = torch.randint(0, 140, (rows,), generator=r).to(torch.int32)
    lens[5] = 3000
    table, n_pages = paged(lens, 16, seed=rows)
    kc, vc = caches(n_pages, 16, 1, 32, "bf16", seed=1)
    q = torch.randn(rows, 1, 2, 32, generator=r).bfloat16()
    _check(q, kc, vc, table, lens, "bf16")


def test_two_calls_at_once():
    """Two streams, each call with a workspace of its own."""
    lens = [3000, 900, 4000]
    table, n_pages = paged(lens, 16)
    kc, vc = (c.cuda() for c in caches(n_pages, 16, 4, 128, "bf16", seed=4))
    table, n = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    qs = [torch.randn(3, 1, 8, 128, generator=torch.Generator().manual_seed(i)).bfloat16().cuda() for i in range(2)]
    want = [gdn.attn_decode(q, kc, vc, table, n) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(gdn.attn_decode(qs[i], kc, vc, table, n, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


def test_a_given_workspace_is_used_and_checked():
    lens = torch.tensor([1500], dtype=torch.int32)
    table, n_pages = paged(lens, 16)
    kc, vc = (c.cuda() for c in caches(n_pages, 16, 2, 64, "bf16", seed=4))
    q = torch.randn(1, 1, 4, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    a = (q, kc, vc, table.cuda(), lens.cuda())
    need = gdn.attn_decode_workspace_size(*a)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8).cuda()  # NaN where nothing is written
    assert torch.equal(gdn.attn_decode(*a, workspace=ws), gdn.attn_decode(*a))
    assert (ws[need:] == 255).all() and not (ws[:need] == 255).all()
    with pytest.raises(ValueError):
        gdn.attn_decode(*a, workspace=ws[:need - 4])


def test_out_over_q_is_refused():
    kc, vc = (c.cuda() for c in caches(4, 16, 2, 64, "bf16", seed=4))
    q = torch.randn(1, 1, 4, 64).bfloat16().cuda()
    with pytest.raises(gdn.GdnError):
        gdn.attn_decode(q, kc, vc, torch.zeros(1, 2, dtype=torch.int32).cuda(), torch.ones(1, dtype=torch.int32).cuda(), out=q)


def test_scores_far_apart_and_infinite():
    """Scores of +-10^4 (one key takes all the weight) and a key of -inf score."""
    lens = torch.tensor([300], dtype=torch.int32)
    table, n_pages = paged(lens, 16)
    kc, vc = caches(n_pages, 16, 1, 64, "f32", seed=2)
    kc *= 1000
    q = torch.full((1, 1, 1, 64), 10.0)
    e, at = int(table[0, 6]), 3
    kc[e, at] = 0
    kc[e, at, 0, 0] = -float("inf")
    want = attn_ref(q, kc, vc, table, lens, 0.125)
    out = gdn.attn_decode(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), lens.cuda())
    top = want[0]
    # one key holds the weight (the next is e^-100 or less): its value, within one rounding
    s = (kc[table[0].long()].reshape(-1, 64)[:300] * 10).sum(-1) * 0.125
    assert float(s.topk(2).values.diff()) < -100
    assert ((out.double().cpu() - top).abs() <= 2.0 ** -22 * top.abs()).all()


@pytest.mark.parametrize("cache", ["f32", "e4m3"])
def test_the_largest_queries(cache):
    """The largest finite fp32 query keeps its sign and size; an infinite one
    gives no number, as its scores' differences are none."""
    lens = torch.tensor([40], dtype=torch.int32)
    table, n_pages = paged(lens, 16)
    kc, vc = caches(n_pages, 16, 1, 64, cache, seed=2)
    kw = torch.zeros(kc.shape)
    kw[..., 5] = 2.0 ** -9
    kw[int(table[0, 1]), 7, 0, 5] = 2.0 ** -8
    kc = kw.to(DT[cache])
    one = torch.ones(1).cuda() if cache == "e4m3" else None
    q = torch.zeros(1, 1, 3, 64)
    q[0, 0, 0, 5], q[0, 0, 1, 5], q[0, 0, 2, 5] = 3.4028234e38, 3.3961e38, float("inf")
    out = gdn.attn_decode(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), lens.cuda(), k_scale=one, v_scale=one).cpu()
    want = vc[int(table[0, 1]), 7, 0].float()
    # the weight is one key's: its value, within the division's and sum's roundings
    assert ((out[0, 0, :2] - want).abs() <= 2.0 ** -22 * want.abs()).all()
    assert out[0, 0, 2].isnan().all()


def test_offsets_past_32_bits():
    """Pages whose element offset needs more than 32 bits."""
    n_pages, page, hkv, d = (1 << 21) + 64, 16, 1, 64  # 2^31 elements and some
    kc = torch.empty((n_pages, page, hkv, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    table = torch.arange(n_pages - 8, n_pages, dtype=torch.int32).flip(0)[None]
    lens = torch.tensor([120], dtype=torch.int32)
    k8, v8 = caches(8, page, hkv, d, "bf16", seed=1)
    kc[n_pages - 8:], vc[n_pages - 8:] = k8.cuda(), v8.cuda()
    q = torch.randn(1, 1, 4, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    want = attn_ref(q, k8, v8, table - (n_pages - 8), lens, 0.125)
    bound = attn_bound(want[0], want[2], want[3], lens, d, "bf16")
    out = gdn.attn_decode(q.cuda(), kc, vc, table.cuda(), lens.cuda())
    assert ((out.double().cpu() - want[0]).abs() <= bound).all()
    # the same rows as 3-token pages (looked up key by key)
    k3, v3 = (c.view(-1, 1, hkv, d) for c in (kc, vc))
    t3 = (table[0, :, None] * 16 + torch.arange(16, dtype=torch.int32)).reshape(1, -1)
    out = gdn.attn_decode(q.cuda(), k3, v3, t3.cuda(), lens.cuda())
    assert ((out.double().cpu() - want[0]).abs() <= bound).all()


def test_shared_pages_and_joining_by_lse():
    """Rows that share pages; and attention over two halves of a row joined by
    their lse equals the whole."""
    page = 16
    table = torch.tensor([[4, 2, 7, 1], [4, 2, 0, 3]], dtype=torch.int32)
    lens = torch.tensor([64, 50], dtype=torch.int32)
    kc, vc = caches(8, page, 2, 64, "f32", seed=6)
    q = torch.randn(2, 1, 4, 64, generator=torch.Generator().manual_seed(5))
    whole = _check(q, kc, vc, table, lens, "f32")
    halves = [gdn.attn_decode(q.cuda(), kc.cuda(), vc.cuda(), t.contiguous().cuda(), n.cuda(), return_lse=True)
              for t, n in ((table[:, :2], torch.tensor([32, 32])), (table[:, 2:], lens - 32))]
    w = torch.softmax(torch.stack([x[1] for x in halves]), 0)[..., None]
    both = sum(w[i] * halves[i][0] for i in range(2))
    # two results, each within some tens of roundings of values up to 4
    assert (both - whole).abs().max() <= 64 * 4 * 2.0 ** -24


def test_given_outputs_empty_batch_and_empty_cache():
    kc, vc = (c.cuda() for c in caches(4, 16, 2, 64, "bf16", seed=1))
    q = torch.randn(0, 1, 4, 64).bfloat16().cuda()
    assert gdn.attn_decode(q, kc, vc, torch.zeros(0, 4, dtype=torch.int32).cuda(),
                           torch.zeros(0, dtype=torch.int32).cuda()).shape == q.shape
    q = torch.randn(2, 1, 4, 64).bfloat16().cuda()
    out = torch.full_like(q, 7.0)
    table, lens = torch.zeros(2, 4, dtype=torch.int32).cuda(), torch.tensor([64, 3], dtype=torch.int32).cuda()
    got = gdn.attn_decode(q, kc[:0], vc[:0], table, lens, out=out)
    assert got is out and (out == 0).all()
    out.fill_(7.0)
    assert (gdn.attn_decode(q, kc, vc, table[:, :0], lens, out=out) == 0).all()


def test_other_stream_and_captured_graphs():
    """A call on a stream of its own, and two graphs (each with its own
    workspace) replayed in turn with eager work between."""
    lens = [2000, 700]
    table, n_pages = paged(lens, 16)
    kc, vc = (c.cuda() for c in caches(n_pages, 16, 2, 128, "bf16", seed=4))
    table, n = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    qs = [torch.randn(2, 1, 8, 128, generator=torch.Generator().manual_seed(i)).bfloat16().cuda() for i in range(2)]
    want = [gdn.attn_decode(q, kc, vc, table, n) for q in qs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gdn.attn_decode(qs[0], kc, vc, table, n, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want[0])
    graphs, outs = [], []
    for q in qs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(gdn.attn_decode(q, kc, vc, table, n))
        graphs.append(graph)
    for i in (0, 1, 0, 0, 1):
        outs[i].zero_()
        graphs[i].replay()
        eager = gdn.attn_decode(qs[1 - i], kc, vc, table, n)
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want[i]) and torch.equal(eager, want[1 - i])
    n.fill_(100)  # lengths are read by the kernel: a replay follows them
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], gdn.attn_decode(qs[0], kc, vc, table, n))


# T, query heads a key-value head: one row of a head, several tokens, two row tiles, more
ROWS = [(1, 2), (3, 2), (3, 8), (5, 9)]


@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("T,group", ROWS)
@pytest.mark.parametrize("io,cache", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "e4m3"), ("f32", "e4m3")])
def test_a_nan_query_gives_nan(io, cache, T, group, page):
    """NaN in the query of one head of one token of each row: that head's
    result and lse are NaN, every other as without it.  Rows walked whole and
    rows that are split and joined, the last one seeing nothing."""
    lens = torch.tensor([T + 20, 700, 0], dtype=torch.int32)
    table, n_pages = paged(lens, page, seed=T)
    kc, vc = caches(n_pages, page, 2, 64, cache, seed=T + group)
    ks, vs = _scales(cache, 2)
    q = torch.randn(3, T, 2 * group, 64, generator=torch.Generator().manual_seed(T)).to(DT[io])
    want, want_lse, mean, size = attn_ref(q, kc, vc, table, lens, 0.125, ks, vs)
    odd = torch.zeros(3, T, 2 * group, dtype=torch.bool)
    for b, (t, h) in enumerate([(0, 1), (T - 1, 2 * group - 1), (0, 0)]):
        q[b, t, h, (b * 31 + 5) % 64] = float("nan")
        odd[b, t, h] = b < 2
    bound = attn_bound(want, mean, size, lens, 64, io)
    tol = 2.0 ** -24 * ((64 + 16) * size[..., 0] + 32 * (want_lse.abs() + 16))
    args = (q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), lens.cuda())
    for split in (True, False):
        if split:
            assert gdn.attn_decode_workspace_size(*args, k_scale=_dev(ks), v_scale=_dev(vs)) > 0
            out, lse = gdn.attn_decode(*args, k_scale=_dev(ks), v_scale=_dev(vs), return_lse=True)
        else:  # without a workspace one wave walks each row and head
            lse = torch.empty(3, T, 2 * group, device="cuda")
            a, keep, out = gdn.attn_decode_args(*args, k_scale=_dev(ks), v_scale=_dev(vs), lse=lse)
            _lib.check(_lib.load().gdn_attn_decode(ctypes.byref(a), torch.cuda.current_stream().cuda_stream))
        out, lse = out.double().cpu(), lse.double().cpu()
        assert torch.equal(out.isnan(), odd[..., None].expand_as(out)) and torch.equal(lse.isnan(), odd)
        assert ((out - want).abs() <= bound)[~odd].all()
        assert torch.equal(lse == -float("inf"), (want_lse == -float("inf")) & ~odd)
        seen = ~odd & (want_lse > -float("inf"))
        assert ((lse - want_lse).abs() <= tol)[seen].all()


@pytest.mark.parametrize("page", [16, 3])
@pytest.mark.parametrize("T", [1, 2])
@pytest.mark.parametrize("io,cache", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "e4m3"), ("f32", "e4m3")])
def test_keys_of_nan_and_scores_of_minus_infinity(io, cache, T, page):
    """Rows whose only visible keys are NaN give NaN; rows whose scores are all
    -inf give zeros and lse -inf; one NaN key among others gives NaN."""
    lens = torch.tensor([1, 300, 300, 300], dtype=torch.int32)
    table, n_pages = paged(lens, page, seed=1)
    kc, vc = caches(n_pages, page, 1, 64, cache, seed=3)
    kw = kc.float()

    def put(b, at, value):
        for j in at:
            kw[int(table[b, j // page]), j % page] = value
    put(0, [0], float("nan"))
    put(1, range(300), float("nan"))
    if cache == "e4m3":  # no infinities: the query's are the scores'
        put(2, range(300), 2.0)
    else:
        put(2, range(300), -float("inf"))
    put(3, [170], float("nan"))
    q = torch.rand(4, T, 2, 64, generator=torch.Generator().manual_seed(2)) + 0.5
    if cache == "e4m3":
        q[2] = -float("inf")
    q, kc = q.to(DT[io]), kw.to(kc.dtype)
    one = torch.ones(1).cuda() if cache == "e4m3" else None
    out, lse = gdn.attn_decode(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), lens.cuda(), k_scale=one, v_scale=one,
                               return_lse=True)
    out, lse = out.cpu(), lse.cpu()
    # row 0 holds one token: the first of two new ones stands before it and sees nothing
    if T == 2:
        assert (out[0, 0] == 0).all() and (lse[0, 0] == -float("inf")).all()
    assert out[0, -1].isnan().all() and lse[0, -1].isnan().all()
    assert out[1].isnan().all() and lse[1].isnan().all()
    assert (out[2] == 0).all() and (lse[2] == -float("inf")).all()
    assert out[3].isnan().all() and lse[3].isnan().all()


@pytest.mark.parametrize("page", [65536, 65536 + 3])
def test_heads_far_apart(page):
    """Heads-first pages so long that a head begins 2^23 elements behind the
    one before it: appended to and attended over."""
    hkv, d, lens = 3, 128, torch.tensor([200, 33], dtype=torch.int32)
    kc, vc = (torch.zeros(3, hkv, page, d, dtype=torch.bfloat16, device="cuda").transpose(1, 2) for _ in range(2))
    assert kc.stride(2) >= 1 << 23
    table = torch.tensor([[2], [0]], dtype=torch.int32)
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(233, hkv, d, generator=g).bfloat16() for _ in range(2))
    cu = torch.tensor([0, 200, 233], dtype=torch.int32)
    gdn.kv_append(k.cuda(), v.cuda(), kc, vc, table.cuda(), lens.cuda(), cu_seqlens=cu.cuda())
    for c, x in ((kc, k), (vc, v)):
        assert torch.equal(c[2, :200].cpu(), x[:200]) and torch.equal(c[0, :33].cpu(), x[200:])
        assert not c[1].any() and not c[2, 200:].any() and not c[0, 33:].any()
    q = torch.randn(2, 1, 6, d, generator=g).bfloat16()
    small = [torch.zeros(3, 256, hkv, d).bfloat16() for _ in range(2)]
    for c, x in zip(small, (k, v)):
        c[2, :200], c[0, :33] = x[:200], x[200:]
    want = attn_ref(q, *small, table, lens, d ** -0.5)
    out = gdn.attn_decode(q.cuda(), kc, vc, table.cuda(), lens.cuda())
    assert ((out.double().cpu() - want[0]).abs() <= attn_bound(want[0], want[2], want[3], lens, d, "bf16")).all()


@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("T,group", [(3, 4), (3, 8), (5, 9)])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("io,cache", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "e4m3"), ("f32", "e4m3")])
def test_several_new_tokens_of_every_type_and_head_size(io, cache, d, T, group, page):
    """12, 24 and 45 query rows of a key-value head: the walks of one row tile,
    of two and of more, each over pages that tiles do and do not divide.  Rows
    shorter than the new tokens, an empty one, one of several tiles; unheld
    slots are NaN, and so is the newest token's value in the longest row, which
    the tokens before it do not see."""
    lens = torch.tensor([T + 1, 0, 2, 30, 210], dtype=torch.int32)
    table, n_pages = paged(lens, page, seed=T)
    kc, vc = caches(n_pages, page, 2, d, cache, seed=T * 100 + d)
    kc, vc = (poison_unheld(c, table, lens, page, float("nan")) for c in (kc, vc))
    ks, vs = _scales(cache, 2)
    q = torch.randn(5, T, 2 * group, d, generator=torch.Generator().manual_seed(d + T)).to(DT[io])
    ref = attn_ref(q, kc, vc, table, lens, d ** -0.5, ks, vs)
    _check(q, kc, vc, table, lens, io, ks, vs, ref=ref)
    w = vc.float()
    w[int(table[4, 209 // page]), 209 % page] = float("nan")
    out = gdn.attn_decode(q.cuda(), kc.cuda(), w.to(vc.dtype).cuda(), table.cuda(), lens.cuda(), k_scale=_dev(ks),
                          v_scale=_dev(vs)).double().cpu()
    assert out[4, -1].isnan().all()
    keep = torch.ones(5, T, dtype=torch.bool)
    keep[4, -1] = False
    assert ((out - ref[0]).abs() <= attn_bound(ref[0], ref[2], ref[3], lens, d, io))[keep].all()
