"""Block-scaled 8-bit caches on the GPU: kv_append bit for bit against a block by
block reference, kv_read bit for bit, attn_decode against 64 bits, and the calls
together as a server uses them."""
import random

import pytest
import torch

import gated_deltanet_state_delta_amd as gdn
from blocks_ref import (CODE, append_ref, attn_blocks_bound, attn_blocks_ref, blocks_cache, codes, need_scale, read_ref,
                        rope_bound, rope_ref, values)
from gpu_util import require_gpu
from paged_ref import DT, paged

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _dev(c):
    """A CPU tensor on the GPU with the same strides (a permuted view stays one)."""
    order = sorted(range(c.dim()), key=lambda i: -c.stride(i))
    back = [order.index(i) for i in range(c.dim())]
    return c.permute(order).contiguous().cuda().permute(back)


def _bits(t):
    """The bits of a tensor, every NaN as one."""
    t = t.cpu().float()
    return torch.where(t.isnan(), torch.full_like(t, 12345.0), t)


def _offsets(counts):
    return torch.tensor([sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32)


def _append(counts, lens, page, block, hkv, d, io, cache, packed=True, seed=0, heads_first=False, table=None, width=None,
            n_pages=None, x=None, cu=None, state=None):
    g = torch.Generator().manual_seed(seed)
    if table is None:
        table, n_pages = paged(lens, page, seed=seed, width=width)
    kc, vc, ks, vs = state or blocks_cache(n_pages, page, hkv, d, block, cache, seed, heads_first)
    k, v = x or (torch.randn(sum(counts), hkv, d, generator=g).mul_(2).to(DT[io]) for _ in range(2))
    lens = torch.tensor(lens, dtype=torch.int32)
    want = [append_ref(c, s, y, counts, table, lens, cache) for c, s, y in ((kc, ks, k), (vc, vs, v))]
    if packed:
        cu = (_offsets(counts) if cu is None else cu).cuda()
    else:
        k, v = (y.view(len(counts), counts[0], hkv, d) for y in (k, v))
    dev = [_dev(t) for t in (kc, vc, ks, vs)]
    got = gdn.kv_append(k.cuda(), v.cuda(), dev[0], dev[1], table.cuda(), lens.cuda(), cu_seqlens=cu, k_scale=dev[2], v_scale=dev[3])
    assert got[0] is dev[0] and got[1] is dev[1]
    for i in range(2):
        assert torch.equal(_bits(dev[2 + i]), _bits(want[i][1])), "scales"
        assert torch.equal(_bits(dev[i]), _bits(want[i][0])), "codes"
    return dev, table, lens


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("cache", ["e4m3", "int8"])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_one_token_a_row(io, cache, d):
    """Blocks begun, continued with and without growth; a row with no room."""
    _append([1] * 7, [1, 16, 17, 40, 0, 33, 24], 16, 8, 3, d, io, cache, packed=False, seed=d)


@pytest.mark.parametrize("page,block", [(16, 16), (16, 1), (16, 4), (5, 5), (5, 1), (12, 3), (64, 64), (1, 1), (24, 2)])
@pytest.mark.parametrize("cache", ["e4m3", "int8"])
@pytest.mark.parametrize("io,d", [("bf16", 64), ("f32", 128)])
def test_packed_prompts(io, d, cache, page, block):
    """Ragged rows, empty ones among them, some continuing a longer row; one
    whose new tokens begin before its start (not written)."""
    _append([0, 70, 1, 0, 33, 5, 0], [9, 70, 30, 0, 50, 3, 2], page, block, 2, d, io, cache, seed=page + block)


@pytest.mark.parametrize("page,block,d", [(128, 128, 64), (256, 256, 128), (300, 150, 256), (1024, 1024, 256), (640, 640, 32)])
@pytest.mark.parametrize("io,cache", [("bf16", "e4m3"), ("f32", "int8"), ("bf16", "int8"), ("f32", "e4m3")])
def test_blocks_that_one_wave_does_not_hold(io, cache, page, block, d):
    """Blocks taken by a whole workgroup, in one part and in several."""
    _append([block + 17, 3, 0, block // 2, 2 * block], [block + 17, 40, 0, block, 2 * block + 9], page, block, 2, d, io, cache,
            seed=page + d)


@pytest.mark.parametrize("T", [2, 5, 40])
@pytest.mark.parametrize("cache", ["e4m3", "int8"])
def test_several_tokens_of_every_row(cache, T):
    _append([T] * 5, [T, T + 3, 100, T - 1, T + 16], 16, 16, 2, 64, "bf16", cache, packed=False, seed=T)


def test_many_blocks_of_a_workgroup():
    """More blocks than there are workgroups at one block each."""
    _append([1500, 900, 2000], [1500, 1000, 2001], 16, 1, 1, 32, "bf16", "int8", seed=3)
    _append([1] * 1300, [1 + 7 * i % 40 for i in range(1300)], 16, 4, 1, 32, "bf16", "e4m3", packed=False, seed=4)


@pytest.mark.parametrize("cache", ["e4m3", "int8"])
def test_layouts(cache):
    _append([20, 3], [40, 3], 16, 4, 3, 64, "bf16", cache, seed=1, heads_first=True)
    # keys and values as slices of one projection, and a step of a sequence-first buffer
    g = torch.Generator().manual_seed(2)
    table, n_pages = paged([40, 3], 16, seed=2)
    kc, vc, ks, vs = blocks_cache(n_pages, 16, 2, 64, 4, cache, 2)
    fused = torch.randn(23, 6, 64, generator=g).bfloat16()
    lens = torch.tensor([40, 3], dtype=torch.int64)
    want = [append_ref(c, s, y, [20, 3], table, lens, cache) for c, s, y in ((kc, ks, fused[:, 2:4]), (vc, vs, fused[:, 4:]))]
    dev, f = [t.cuda() for t in (kc, vc, ks, vs)], fused.cuda()
    gdn.kv_append(f[:, 2:4], f[:, 4:], dev[0], dev[1], table.cuda(), lens.cuda(), cu_seqlens=_offsets([20, 3]).cuda(),
                  k_scale=dev[2], v_scale=dev[3])
    for i in range(2):
        assert torch.equal(_bits(dev[i]), _bits(want[i][0])) and torch.equal(dev[2 + i].cpu(), want[i][1])
    steps = torch.randn(3, 2, 2, 64, generator=g).bfloat16()  # [step, row, head, d]
    want = append_ref(kc, ks, steps[1], [1, 1], table, lens, cache)
    dev = [t.cuda() for t in (kc, vc, ks, vs)]
    x = steps.cuda()[1][:, None]
    gdn.kv_append(x, x, dev[0], dev[1], table.cuda(), lens.cuda(), k_scale=dev[2], v_scale=dev[3])
    assert torch.equal(_bits(dev[0]), _bits(want[0])) and torch.equal(dev[2].cpu(), want[1])


@pytest.mark.parametrize("cache", ["e4m3", "int8"])
def test_positions_and_entries_that_hold_nothing(cache):
    """Entries outside the cache, positions past the table, more tokens than positions."""
    table, n_pages = paged([64, 64, 64], 16, width=4, spare=0)
    table[0, 1], table[1, 0], table[2, 3] = -1, n_pages, 1 << 30
    _append([60, 20, 90], [64, 64, 80], 16, 8, 2, 64, "bf16", cache, seed=5, table=table, n_pages=n_pages)
    _append([4, 4, 4], [-5, 1 << 30, 2], 16, 8, 2, 64, "bf16", cache, seed=6, table=table, n_pages=n_pages)


@pytest.mark.parametrize("cache", ["e4m3", "int8"])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_values_that_are_not_numbers_and_extreme_ones(io, cache):
    inf, nan = float("inf"), float("nan")
    g = torch.Generator().manual_seed(7)
    x = torch.randn(40, 2, 64, generator=g)
    x[0, 0, :3] = torch.tensor([inf, -inf, 2.0])
    x[5, 1, 7] = nan
    x[8:16, 0] = 0.0                     # a block of zeros
    x[16:24, 0] = -0.0
    x[16, 0, 5] = 1e-45                  # smaller than any scale
    x[24, 1, 9] = 3.3e38
    x[32:, 0] = inf                      # nothing finite
    x[33, 1, :] = 448.0 * 2.0 ** -20     # on the border between two powers of two
    x = x.to(DT[io])
    _append([40], [40], 8, 8, 2, 64, io, cache, x=(x, x.flip(0).contiguous()), seed=8)
    # the same into blocks whose older tokens and scales are anything
    table, n_pages = paged([44], 8, seed=9)
    state = blocks_cache(n_pages, 8, 2, 64, 8, cache, 9)
    first = int(table[0, 0])
    for scale in (nan, inf, 0.0, 1e-40, 2.0 ** -126, 3e38, 0.37, 2.0 ** 100):
        state[2][first], state[3][first] = scale, scale
        _append([40], [44], 8, 8, 2, 64, io, cache, x=(x, x.flip(0).contiguous()), table=table, n_pages=n_pages, state=state)


def test_every_quotient_rounds_as_the_division_does():
    """int8: quotients next to the middle between two codes; e4m3: all codes'
    values, midpoints and their neighbours, under scales that are no power of two."""
    k = torch.arange(-127, 127, dtype=torch.float32) + 0.5
    for s_old in (0.031, 0.37, 1.0, 3.1e-5):
        mid = k * s_old
        x = torch.cat([mid, torch.nextafter(mid, mid + 1), torch.nextafter(mid, mid - 1), torch.arange(-127, 128) * s_old])
        x = torch.cat([x, torch.zeros(-x.numel() % 64)]).reshape(-1, 1, 64)
        n = x.shape[0]
        table, n_pages = paged([n + 1], 32, seed=1)
        state = blocks_cache(n_pages, 32, 1, 64, 32, "int8", 1)
        for s in state[2:]:
            s.fill_(s_old)
        _append([n], [n + 1], 32, 32, 1, 64, "f32", "int8", x=(x, -x), table=table, n_pages=n_pages, state=state)
    c = torch.arange(0, 0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    for s_old in (0.37, 1.1, 2.0 ** -30, 5.0):
        mid = (c[1:] + c[:-1]) / 2 * s_old
        x = torch.cat([c * s_old, mid, torch.nextafter(mid, mid + 1), torch.nextafter(mid, mid * 0)])
        x = torch.cat([x, torch.zeros(-x.numel() % 64)]).reshape(-1, 1, 64)
        n = x.shape[0]
        table, n_pages = paged([n + 1], 32, seed=1)
        state = blocks_cache(n_pages, 32, 1, 64, 32, "e4m3", 1)
        for s in state[2:]:
            s.fill_(s_old)
        _append([n], [n + 1], 32, 32, 1, 64, "f32", "e4m3", x=(x, -x), table=table, n_pages=n_pages, state=state)


@pytest.mark.parametrize("cache", ["e4m3", "int8"])
def test_offsets_that_decrease_write_nothing_astray(cache):
    """What lies in a row's range may be left out, but nothing else changes."""
    table, n_pages = paged([30, 30, 30], 16, seed=4)
    kc, vc, ks, vs = blocks_cache(n_pages, 16, 2, 64, 4, cache, 4)
    x = torch.randn(30, 2, 64).bfloat16()
    lens = torch.tensor([30, 30, 30], dtype=torch.int32)
    for cu in ([0, 20, 10, 30], [-5, 12, 50, 30], [30, 20, 10, 0], [0, 40, 40, 40], [5, 9, 9, 20]):
        dev = [t.cuda() for t in (kc, vc, ks, vs)]
        gdn.kv_append(x.cuda(), x.cuda(), dev[0], dev[1], table.cuda(), lens.cuda(), k_scale=dev[2], v_scale=dev[3],
                      cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
        at = [min(max(i, 0), 30) for i in cu]
        may = [append_ref(kc, ks, x[at[b]:max(at[b], at[b + 1])],
                          [max(0, at[b + 1] - at[b]) if i == b else 0 for i in range(3)], table, lens, cache) for b in range(3)]
        got = _bits(dev[0])
        ok = got == _bits(kc)
        for c, _ in may:
            ok |= got == _bits(c)
        assert ok.all(), cu
        if at == sorted(at):  # ordinary offsets: all of it
            want = append_ref(kc, ks, x[at[0]:], [at[b + 1] - at[b] for b in range(3)], table, lens, cache)
            assert torch.equal(got, _bits(want[0])) and torch.equal(dev[2].cpu(), want[1])


def test_pages_past_2_31_codes():
    """A page whose codes lie beyond 2^31 elements of the cache."""
    n_pages, page, hkv, d = (1 << 31) // (64 * 8 * 256) + 3, 64, 8, 256
    kc, vc = (torch.zeros(n_pages, page, hkv, d, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(n_pages, hkv, 4, device="cuda") for _ in range(2))
    table = torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32)
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(100, hkv, d, generator=g).bfloat16() for _ in range(2))
    lens, cu = torch.tensor([100], dtype=torch.int32).cuda(), torch.tensor([0, 100], dtype=torch.int32).cuda()
    gdn.kv_append(k.cuda(), v.cuda(), kc, vc, table.cuda(), lens, cu_seqlens=cu, k_scale=ks, v_scale=vs)
    small = torch.zeros(2, page, hkv, d, dtype=torch.int8), torch.zeros(2, hkv, 4)
    for x, c, s in ((k, kc, ks), (v, vc, vs)):
        want = append_ref(*small, x, [100], table - (n_pages - 2), torch.tensor([100]), "int8")
        assert torch.equal(c[-2:].cpu(), want[0]) and torch.equal(s[-2:].cpu(), want[1])
    got = gdn.kv_read(kc, vc, table.cuda(), lens, 100, cu_seqlens=cu, dtype=torch.float32, k_scale=ks, v_scale=vs)
    q = torch.randn(1, 1, 16, d, generator=g).bfloat16()
    out = gdn.attn_decode(q.cuda(), kc, vc, table.cuda(), lens, k_scale=ks, v_scale=vs).double().cpu()
    held = [(c[-2:].cpu(), s[-2:].cpu()) for c, s in ((kc, ks), (vc, vs))]
    for (c, s), t in zip(held, got):
        assert torch.equal(t.cpu(), read_ref(c, s, [100], table - (n_pages - 2), torch.tensor([100]), torch.float32))
    want, _, mean, size = attn_blocks_ref(q, held[0][0], held[1][0], held[0][1], held[1][1], table - (n_pages - 2),
                                          torch.tensor([100]), d ** -0.5)
    assert ((out - want).abs() <= attn_blocks_bound(want, mean, size, [100], d, "bf16")).all()


# --------------------------------------------------------------------- read --


@pytest.mark.parametrize("page,block", [(16, 16), (16, 4), (5, 1), (24, 8)])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("cache", ["e4m3", "int8"])
def test_read_blocks(cache, io, d, page, block):
    counts, lens = [0, 70, 1, 0, 33, 5, 0], torch.tensor([9, 70, 30, 0, 50, 3, 2], dtype=torch.int32)
    table, n_pages = paged(lens, page, seed=d)
    state = blocks_cache(n_pages, page, 2, d, block, cache, d)
    kc, vc, ks, vs = (t.cuda() for t in state)
    got = gdn.kv_read(kc, vc, table.cuda(), lens.cuda(), sum(counts), cu_seqlens=_offsets(counts).cuda(), dtype=DT[io],
                      k_scale=ks, v_scale=vs)
    for y, c, s in zip(got, state[:2], state[2:]):
        assert torch.equal(y.cpu(), read_ref(c, s, counts, table, lens, DT[io]))


@pytest.mark.parametrize("cache", ["bf16", "f32", "e4m3"])
def test_read_other_caches(cache):
    """Caches without block scales; every row, heads first; rows that hold less than is read."""
    lens = torch.tensor([40, 3, 0, 64, 200], dtype=torch.int64)
    table, n_pages = paged([40, 3, 0, 64, 64], 16, width=4, spare=0, seed=1)
    table[3, 1] = n_pages
    g = torch.Generator().manual_seed(1)
    kc, vc = (torch.randn(n_pages, 3, 16, 64, generator=g).to(DT[cache]).transpose(1, 2) for _ in range(2))
    ks = vs = None
    if cache == "e4m3":
        ks, vs = torch.rand(3, generator=g), torch.rand(3, generator=g)
    dev = [None if t is None else _dev(t) for t in (kc, vc, ks, vs)]
    for io in ("bf16", "f32") if cache == "e4m3" else (cache,):
        got = gdn.kv_read(dev[0], dev[1], table.cuda(), lens.cuda(), 7, k_scale=dev[2], v_scale=dev[3], dtype=DT[io])
        for y, c, s in zip(got, (kc, vc), (ks, vs)):
            full = None if s is None else s[None, :, None].expand(n_pages, 3, 1)
            want = read_ref(c, full, [7] * 5, table, lens, DT[io]).view(5, 7, 3, 64)
            assert torch.equal(y.cpu(), want)
    assert (got[0][2] == 0).all() and (got[0][4] == 0).all() and (got[0][1, :4] == 0).all()


def test_read_leaves_tokens_of_no_row():
    lens, cu = torch.tensor([20, 30], dtype=torch.int32), torch.tensor([3, 8, 12], dtype=torch.int32)
    table, n_pages = paged(lens, 16)
    state = blocks_cache(n_pages, 16, 2, 64, 16, "int8", 0)
    dev = [t.cuda() for t in state]
    given = tuple(torch.full((20, 2, 64), 7.0, dtype=torch.bfloat16).cuda() for _ in range(2))
    args = (dev[0], dev[1], table.cuda(), lens.cuda(), 20)
    out = gdn.kv_read(*args, cu_seqlens=cu.cuda(), k_scale=dev[2], v_scale=dev[3], out=given)
    new = gdn.kv_read(*args, cu_seqlens=cu.cuda(), k_scale=dev[2], v_scale=dev[3])
    want = read_ref(state[0], state[2], [5, 4], table, lens, torch.bfloat16)
    assert out[0] is given[0]
    for y, rest in ((out[0], 7.0), (new[0], 0.0)):
        assert torch.equal(y[3:12].cpu(), want) and (y[:3] == rest).all() and (y[12:] == rest).all()


def test_what_is_appended_is_read_back_as_near_as_the_codes_are():
    """Half a step of e4m3 (2^-4 of the value, or of its smallest normal number 2^-6 scale) and of int8 (half a
    scale), however the tokens came: growth by a power of two keeps e4m3's values but for their smallest, and
    int8's are rounded once more each time the scale grows."""
    g = torch.Generator().manual_seed(3)
    n, page, d = 48, 16, 64
    x = torch.randn(n, 2, d, generator=g) * torch.exp(torch.randn(n, 1, 1, generator=g))
    table, n_pages = paged([n], page)
    for cache in ("e4m3", "int8"):
        for step in (1, 5, n):
            c = [torch.zeros(n_pages, page, 2, d, dtype=CODE[cache]).cuda() for _ in range(2)]
            s = [torch.full((n_pages, 2, 1), float("nan")).cuda() for _ in range(2)]
            grew = torch.zeros(n, 2)
            for at in range(0, n, step):
                to = min(n, at + step)
                before = s[0].clone()
                lens = torch.tensor([to], dtype=torch.int32).cuda()
                y = x[None, at:to].cuda()
                gdn.kv_append(y, y, *c, table.cuda(), lens, k_scale=s[0], v_scale=s[1])
                changed = (s[0] != before).cpu()[table[0].long(), :, 0]  # [page of the row, head]
                grew[:at] += changed.repeat_interleave(page, 0)[:at].float()
            got = gdn.kv_read(*c, table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(), n, dtype=torch.float32,
                              k_scale=s[0], v_scale=s[1])[0].cpu()[0]
            scale = s[0].cpu()[table[0].long(), :, 0].repeat_interleave(page, 0)[:n, :, None]
            if cache == "int8":
                bound = (0.5 + 0.5 * grew[..., None]) * scale * (1 + 2.0 ** -20)
            else:
                bound = torch.maximum(x.abs() * 2.0 ** -4, (1 + grew[..., None]) * scale * 2.0 ** -10)
            assert ((got - x).abs() <= bound).all(), (cache, step)
            assert step == 1 or (grew == 0).any()


# ---------------------------------------------------------------- attention --

LENS = [1, 0, 2, 15, 16, 17, 63, 64, 65, 130, 257, -3]


def _attend(q, state, table, lens, io, ref=None, **kw):
    d = q.shape[-1]
    out, lse = gdn.attn_decode(q.cuda(), _dev(state[0]), _dev(state[1]), table.cuda(), lens.cuda(), k_scale=state[2].cuda(),
                               v_scale=state[3].cuda(), return_lse=True, **kw)
    want, want_lse, mean, size = ref or attn_blocks_ref(q, *state, table, lens, d ** -0.5)
    got, bound = out.double().cpu(), attn_blocks_bound(want, mean, size, lens, d, io)
    bad = ((got - want).abs() > bound) | got.isnan()
    assert not bad.any(), "%d values off, worst by %.2f bounds" % (bad.sum(), ((got - want).abs() / bound).max())
    lse, none = lse.double().cpu(), want_lse == -float("inf")
    assert torch.equal(lse == -float("inf"), none)
    tol = 2.0 ** -24 * ((d + 18) * size[..., 0] + 32 * (want_lse.abs() + 16))
    assert ((lse - want_lse).abs()[~none] <= tol[~none]).all()
    return out


def _poison(state, table, lens, page):
    """Scales of blocks that no row holds are NaN, and e4m3 codes of slots that no row holds."""
    kc, vc, ks, vs = (t.clone() for t in state)
    block = page // ks.shape[2]
    held = torch.zeros(kc.shape[0], page, dtype=torch.bool)
    for b in range(table.shape[0]):
        for j in range(min(max(int(lens[b]), 0), table.shape[1] * page)):
            e = int(table[b, j // page])
            if 0 <= e < kc.shape[0]:
                held[e, j % page] = True
    any_held = held.view(kc.shape[0], -1, block).any(-1)
    for s in (ks, vs):
        s.masked_fill_(~any_held[:, None], float("nan"))
    if kc.dtype != torch.int8:
        kc, vc = (torch.where(held[..., None, None], c.float(), float("nan")).to(c.dtype) for c in (kc, vc))
    return [kc, vc, ks, vs]


# blocks of a multiple of 16, of 8, 4 and 1 token in pages of a multiple of 16; others
@pytest.mark.parametrize("page,block", [(16, 16), (64, 4), (1, 1), (5, 5), (24, 8), (32, 1), (16, 8), (48, 48), (48, 3), (32, 2)])
@pytest.mark.parametrize("room", [0, 600])  # tokens that the table has room for beyond: teams of waves, or shares
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("cache", ["e4m3", "int8"])
def test_types_head_sizes_pages_and_blocks(cache, io, d, room, page, block):
    lens = torch.tensor(LENS, dtype=torch.int32)
    table, n_pages = paged(LENS, page, seed=d + page, width=-(-(max(LENS) + room) // page))
    state = _poison(blocks_cache(n_pages, page, 2, d, block, cache, d * 7 + page), table, lens, page)
    q = torch.randn(len(LENS), 1, 6, d, generator=torch.Generator().manual_seed(d)).to(DT[io])
    _attend(q, state, table, lens, io)


@pytest.mark.parametrize("page,block", [(16, 16), (16, 1), (6, 3)])
@pytest.mark.parametrize("room", [0, 600])
@pytest.mark.parametrize("T,group", [(1, 16), (1, 20), (2, 3), (4, 8), (64, 1), (16, 6)])
@pytest.mark.parametrize("io,cache,d", [("bf16", "e4m3", 128), ("bf16", "int8", 256), ("f32", "int8", 64), ("f32", "e4m3", 256),
                                        ("bf16", "int8", 32), ("f32", "int8", 128), ("bf16", "e4m3", 64)])
def test_new_tokens_and_groups(io, cache, d, T, group, room, page, block):
    lens = torch.tensor([0, 1, T - 1, T, 40, 100, 3 * T + 50], dtype=torch.int32)
    table, n_pages = paged(lens, page, seed=T, width=-(-(int(lens.max()) + room) // page))
    state = _poison(blocks_cache(n_pages, page, 2, d, block, cache, T * 100 + group), table, lens, page)
    q = torch.randn(7, T, 2 * group, d, generator=torch.Generator().manual_seed(T)).to(DT[io])
    _attend(q, state, table, lens, io)


@pytest.mark.parametrize("room", [0, 600])
@pytest.mark.parametrize("io,cache,page,block", [(io, cache, page, block) for io in ("bf16", "f32") for cache in ("e4m3", "int8")
                                                 for page, block in ((32, 1), (6, 1), (16, 16)) if cache == "e4m3" or block == 1])
def test_values_that_a_token_does_not_see(io, cache, page, block, room):
    """The newest of several tokens has scales of NaN (its own block's, or where blocks are
    longer, e4m3 codes of NaN; int8 has none): the tokens before it do not see them."""
    lens = torch.tensor([5, 37, 130], dtype=torch.int32)
    table, n_pages = paged(lens, page, width=-(-(130 + room) // page))
    state = blocks_cache(n_pages, page, 2, 64, block, cache, 11)
    q = torch.randn(3, 4, 4, 64, generator=torch.Generator().manual_seed(3)).to(DT[io])
    refs = [(y, attn_blocks_ref(y, *state, table, lens, 0.125)) for y in (q, q.repeat_interleave(10, 2))]
    state = [t.clone() for t in state]
    for b in range(3):
        j = int(lens[b]) - 1
        e, at = int(table[b, j // page]), j % page
        for i in (0, 1) if block > 1 else (2, 3):
            if block > 1:
                w = state[i].float()
                w[e, at] = float("nan")
                state[i] = w.to(state[i].dtype)
            else:
                state[i][e, :, at] = float("nan") if b else float("inf")
    for y, ref in refs:
        out = gdn.attn_decode(y.cuda(), state[0].cuda(), state[1].cuda(), table.cuda(), lens.cuda(), k_scale=state[2].cuda(),
                              v_scale=state[3].cuda())
        got = out.double().cpu()
        bound = attn_blocks_bound(ref[0], ref[2], ref[3], lens, 64, io)
        assert ((got - ref[0]).abs() <= bound)[:, :3].all()
        assert got[1:, 3].isnan().all()


@pytest.mark.parametrize("cache", ["e4m3", "int8"])
@pytest.mark.parametrize("page,block", [(16, 16), (16, 1), (7, 7)])
def test_split_rows(cache, page, block):
    """Long rows joined from many parts, repeatable, like one wave's walk; entries outside the cache."""
    lens = torch.tensor([5000, 70, 0, 3001], dtype=torch.int32)
    table, n_pages = paged(lens, page, spare=0)
    table[0, 9], table[3, 3] = -1, n_pages
    state = blocks_cache(n_pages, page, 2, 128, block, cache, 2)
    q = torch.randn(4, 2, 8, 128, generator=torch.Generator().manual_seed(4)).bfloat16()
    out = _attend(q, state, table, lens, "bf16")
    again = _attend(q, state, table, lens, "bf16")
    assert torch.equal(out, again)
    dev = [t.cuda() for t in (q, state[0], state[1], table, lens, state[2], state[3])]
    assert gdn.attn_decode_workspace_size(*dev[:5], k_scale=dev[5], v_scale=dev[6]) > 0


@pytest.mark.parametrize("cache", ["e4m3", "int8"])
@pytest.mark.parametrize("page,block", [(16, 16), (32, 1), (7, 7)])
@pytest.mark.parametrize("lens", [[512, 500, 1, 0, 300], [65, 128, 3, 96, 127], [64, 33, 7, 0, 2], [512] * 70])
def test_short_tables(lens, page, block, cache):
    """Teams at their longest and shortest, one wave alone, and as many rows as teams take (140 heads); entries
    outside the cache at a wave's first and last tile."""
    hkv = 2 if len(lens) < 50 else 14
    table, n_pages = paged(lens, page, spare=0, width=-(-max(lens) // page))
    table[0, 0], table[0, table.shape[1] // 4], table[1, -1] = -1, n_pages, 1 << 30
    state = blocks_cache(n_pages, page, hkv, 64, block, cache, 3)
    q = torch.randn(len(lens), 2, 2 * hkv, 64, generator=torch.Generator().manual_seed(4)).bfloat16()
    lens = torch.tensor(lens, dtype=torch.int32)
    some = list(range(len(lens)))[:5]
    out = gdn.attn_decode(q.cuda(), *(t.cuda() for t in state[:2]), table.cuda(), lens.cuda(), k_scale=state[2].cuda(),
                          v_scale=state[3].cuda())
    few = _attend(q[some], state, table[some], lens[some], "bf16")
    bound = 2 * 2.0 ** -8 * out[some].abs().double() + 1e-4  # the same sums in another order, rounded to bf16
    assert ((out[some].double() - few.double()).abs() <= bound).all()
    assert torch.equal(out, gdn.attn_decode(q.cuda(), *(t.cuda() for t in state[:2]), table.cuda(), lens.cuda(),
                                            k_scale=state[2].cuda(), v_scale=state[3].cuda()))


def test_scales_of_a_block_size_that_is_its_page_agree_with_factors_a_head():
    """The same factor everywhere: the two forms of an e4m3 cache differ by roundings only."""
    lens = torch.tensor([300, 17], dtype=torch.int32)
    table, n_pages = paged(lens, 16)
    kc, vc, ks, vs = blocks_cache(n_pages, 16, 2, 128, 16, "e4m3", 5)
    f = torch.tensor([0.01, 0.02])
    ks, vs = (f[None, :, None].expand(n_pages, 2, 1).contiguous() for _ in range(2))
    q = torch.randn(2, 1, 4, 128, generator=torch.Generator().manual_seed(1))
    a = _attend(q, [kc, vc, ks, vs], table, lens, "f32")
    b = gdn.attn_decode(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), lens.cuda(), k_scale=f.cuda(), v_scale=f.cuda())
    assert torch.allclose(a, b, rtol=1e-4, atol=1e-6)


def test_thousands_of_rows():
    """More rows than are dealt into shares, with tables longer than teams take."""
    rows, g = 5000, torch.Generator().manual_seed(1)
    lens = torch.randint(0, 40, (rows,), generator=g).to(torch.int32)
    lens[17] = 530
    need = (lens + 15) // 16
    n_pages, table, at = int(need.sum()), torch.full((rows, 40), -1, dtype=torch.int32), 0
    for b, n in enumerate(need.tolist()):
        table[b, :n], at = torch.arange(at, at + n), at + n
    state = blocks_cache(n_pages, 16, 1, 32, 16, "int8", 1)
    q = torch.randn(rows, 1, 2, 32, generator=g).bfloat16()
    out = gdn.attn_decode(q.cuda(), state[0].cuda(), state[1].cuda(), table.cuda(), lens.cuda(), k_scale=state[2].cuda(),
                          v_scale=state[3].cuda()).double().cpu()
    some = [0, 17, 18, 999, 4097, 4999] + torch.randint(0, rows, (40,), generator=g).tolist()
    want, _, mean, size = attn_blocks_ref(q[some], *state, table[some], lens[some], 32 ** -0.5)
    assert ((out[some] - want).abs() <= attn_blocks_bound(want, mean, size, lens[some], 32, "bf16")).all()
    # and one token appended to each
    lens = lens + 1
    fresh = (lens - 1) % 16 == 0
    extra = torch.arange(n_pages, n_pages + int(fresh.sum()), dtype=torch.int32)
    table[fresh, ((lens - 1) // 16)[fresh].long()] = extra
    state = blocks_cache(n_pages + len(extra), 16, 1, 32, 16, "int8", 2)
    x = torch.randn(rows, 1, 1, 32, generator=g).bfloat16()
    dev = [t.cuda() for t in state]
    gdn.kv_append(x.cuda(), x.cuda(), dev[0], dev[1], table.cuda(), lens.cuda(), k_scale=dev[2], v_scale=dev[3])
    want = append_ref(state[0], state[2], x[:, 0], [1] * rows, table, lens, "int8")
    assert torch.equal(dev[0].cpu(), want[0]) and torch.equal(dev[2].cpu(), want[1])


def test_no_pages_no_rows_no_tokens():
    """Caches of no pages, tables of no entries, batches of no rows, rows of no tokens."""
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32).cuda()
    for n_pages, width, rows in ((0, 4, 3), (2, 0, 3), (2, 4, 0), (0, 0, 3)):
        c = [torch.zeros(n_pages, 16, 2, 64, dtype=torch.int8).cuda() for _ in range(2)]
        s = [torch.ones(n_pages, 2, 4).cuda() for _ in range(2)]
        kw, table, lens = dict(k_scale=s[0], v_scale=s[1]), i32(rows, width), i32(rows) + 20
        q = torch.ones(rows, 1, 4, 64).bfloat16().cuda()
        out = gdn.attn_decode(q, *c, table, lens, **kw)
        assert out.shape == q.shape and (out == 0).all()
        gdn.kv_append(q[:, :, :2], q[:, :, :2], *c, table, lens, **kw)
        for got in (gdn.kv_read(*c, table, lens, 3, **kw), gdn.kv_read(*c, table, lens, 7, cu_seqlens=i32(rows + 1), **kw)):
            assert all((t == 0).all() for t in got)
        assert all((t == 0).all() for t in gdn.kv_read(*c, table, lens, 0, **kw))


# ----------------------------------------------------------- all of it at once --


@pytest.mark.parametrize("cache,page,block", [("e4m3", 16, 16), ("int8", 12, 4)])
def test_a_batch_lives_through_prompts_forks_and_compaction(cache, page, block):
    """rope, kv_append, attn_decode and kv_read over pages that grow, fork, are
    freed and compacted, the scales copied beside the codes: codes and scales
    against a plain history of each row, results against 64 bits over them."""
    rows, width, hkv, hq, d, n_pages = 5, 10, 2, 6, 64, 80
    r, gen = random.Random(page), torch.Generator().manual_seed(page)
    c = [torch.zeros(n_pages, page, hkv, d, dtype=CODE[cache]).cuda() for _ in range(2)]
    s = [torch.full((n_pages, hkv, page // block), float("nan")).cuda() for _ in range(2)]
    table = torch.full((rows, width), -1, dtype=torch.int32).cuda()
    lens, refs = torch.zeros(rows, dtype=torch.int32).cuda(), torch.zeros(n_pages, dtype=torch.int32).cuda()
    f, factor = gdn.rope_frequencies(32, scaling="parts", scale=4, trained=64)
    nblk = width * page // block
    # each row's own history as pages of one block
    hist = [[torch.zeros(nblk, block, hkv, d).to(CODE[cache]), torch.zeros(nblk, block, hkv, d).to(CODE[cache]),
             torch.zeros(nblk, hkv, 1), torch.zeros(nblk, hkv, 1), 0] for _ in range(rows)]
    plain = torch.arange(nblk, dtype=torch.int32)[None]

    def turn(x, counts, ends, heads):
        pos = torch.cat([torch.arange(e - n, e) for e, n in zip(ends, counts)])
        y, size = rope_ref(x, pos, f, False, factor)
        return y, rope_bound(y, size, pos, f, "bf16")

    def step(counts):
        """Every row's new tokens: rotated, appended, attended (T = 1) and read back."""
        nonlocal table, lens, refs
        table, lens, refs, ok = gdn.pages_extend(table, lens, refs, torch.tensor(counts, dtype=torch.int32).cuda(), page)
        fits = [h[4] + n <= width * page for h, n in zip(hist, counts)]
        assert ok.tolist() == fits
        counts = [n if o else 0 for n, o in zip(counts, fits)]
        total, cu = sum(counts), _offsets(counts)
        ends = [h[4] + n for h, n in zip(hist, counts)]
        q, k, v = (torch.randn(total, h, d, generator=gen).bfloat16() for h in (hq, hkv, hkv))
        kw = dict(lens=lens, cu_seqlens=cu.cuda(), factor=factor)
        qr, kr = gdn.rope(q.cuda(), k.cuda(), f.cuda(), **kw)
        for x, y, h in ((q, qr, hq), (k, kr, hkv)):
            want, bound = turn(x, counts, ends, h)
            assert ((y.cpu().double() - want).abs() <= bound).all()
        gdn.kv_append(kr, v.cuda(), *c, table, lens, cu_seqlens=cu.cuda(), k_scale=s[0], v_scale=s[1])
        kr = kr.cpu()
        for b in range(rows):
            h, mine = hist[b], slice(int(cu[b]), int(cu[b + 1]))
            for i, x in ((0, kr), (1, v)):
                h[i], h[i + 2] = append_ref(h[i], h[i + 2], x[mine], [counts[b]], plain, torch.tensor([ends[b]]), cache)
            h[4] = ends[b]
        assert lens.tolist() == ends
        got = gdn.kv_read(*c, table, lens, total, cu_seqlens=cu.cuda(), dtype=torch.float32, k_scale=s[0], v_scale=s[1])
        for i in range(2):
            want = torch.cat([read_ref(h[i], h[i + 2], [n], plain, torch.tensor([h[4]]), torch.float32)
                              for h, n in zip(hist, counts)])
            assert torch.equal(got[i].cpu(), want)
        if counts == [counts[0]] * rows and counts[0]:
            attend(qr.view(rows, counts[0], hq, d))
        return qr

    def attend(q):
        got = gdn.attn_decode(q, *c, table, lens, k_scale=s[0], v_scale=s[1]).double().cpu()
        q = q.cpu()
        for b in range(rows):
            h, n = hist[b], torch.tensor([hist[b][4]])
            want, _, mean, size = attn_blocks_ref(q[b:b + 1], *h[:4], plain, n, d ** -0.5)
            assert ((got[b:b + 1] - want).abs() <= attn_blocks_bound(want, mean, size, n, d, "bf16")).all(), b

    step([40, 0, 17, 3, 50])
    for i in range(8):
        kind = i % 4
        if kind in (0, 2):
            step([r.choice([1, 3])] * rows)
        elif kind == 1:
            parent = [r.choice([b, r.randrange(rows)]) for b in range(rows)]
            table, lens, refs, src, dst = gdn.pages_fork(table, lens, refs, torch.tensor(parent, dtype=torch.int32).cuda(), page)
            for pool in c + s:
                gdn.pages_copy(pool, src, dst)
            hist = [list(hist[b]) for b in parent]
            step([1] * rows)
        else:
            drop = torch.tensor([r.random() < 0.3 for _ in range(rows)])
            table, lens, refs = gdn.pages_free(table, lens, refs, drop.cuda(), page)
            for b in range(rows):
                if drop[b]:
                    hist[b][4] = 0
            table, refs, src, dst, _ = gdn.pages_compact(table, refs)
            for pool in c + s:
                gdn.pages_copy(pool, src, dst)
            step([2] * rows)


@pytest.mark.parametrize("cache", ["e4m3", "int8"])
def test_a_decode_step_captured_once_and_replayed(cache):
    """Grow, rotate, append, attend and read back in one graph, in place: every
    replay is one more token of each row, checked against eager calls on copies."""
    rows, width, page, block, hkv, hq, d, n_pages = 4, 8, 16, 8, 2, 8, 128, 40
    gen = torch.Generator().manual_seed(1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    draw = lambda h, n=rows: torch.randn(n, 1, h, d, generator=gen).bfloat16().cuda()
    c = [torch.zeros(n_pages, page, hkv, d, dtype=CODE[cache]).cuda() for _ in range(2)]
    s = [torch.zeros(n_pages, hkv, page // block).cuda() for _ in range(2)]
    table, lens, refs = torch.full((rows, width), -1, dtype=torch.int32).cuda(), i32([0] * rows), i32([0] * n_pages)
    one, start = i32([1] * rows), [14, 0, 31, 60]
    f = gdn.rope_frequencies(d)[0].cuda()
    gdn.pages_extend(table, lens, refs, i32(start), page, out=(table, lens, refs))
    k, v = (torch.randn(sum(start), hkv, d, generator=gen).bfloat16().cuda() for _ in range(2))
    gdn.kv_append(k, v, *c, table, lens, cu_seqlens=_offsets(start).cuda(), k_scale=s[0], v_scale=s[1])
    q1, k1, v1 = draw(hq), draw(hkv), draw(hkv)

    def step(table, lens, refs, c, s, q, k, v):
        gdn.pages_extend(table, lens, refs, one, page, out=(table, lens, refs))
        qr, kr = gdn.rope(q, k, f, lens=lens)
        gdn.kv_append(kr, v, *c, table, lens, k_scale=s[0], v_scale=s[1])
        out = gdn.attn_decode(qr, *c, table, lens, k_scale=s[0], v_scale=s[1])
        return out, *gdn.kv_read(*c, table, lens, 1, k_scale=s[0], v_scale=s[1])

    copy = lambda: ([t.clone() for t in (table, lens, refs)] + [[t.clone() for t in c], [t.clone() for t in s]])
    step(*copy(), q1, k1, v1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(table, lens, refs, c, s, q1, k1, v1)
    for _ in range(6):
        for t, h in ((q1, hq), (k1, hkv), (v1, hkv)):
            t.copy_(draw(h))
        other = copy()
        graph.replay()
        want = step(*other, q1, k1, v1)  # eager work between the replays
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        for a, b in zip([table, lens, refs] + c + s, other[:3] + other[3] + other[4]):
            assert torch.equal(_bits(a), _bits(b))
    assert lens.tolist() == [n + 6 for n in start]


def test_two_streams_and_another_current_stream():
    """The calls on streams of their own, at once, on separate caches."""
    state = [blocks_cache(40, 16, 2, 64, 4, "int8", i) for i in range(2)]
    lens = torch.tensor([200, 100], dtype=torch.int32)
    table, _ = paged(lens, 16)
    x = [torch.randn(2, 30, 2, 64, generator=torch.Generator().manual_seed(i)).bfloat16() for i in range(2)]
    streams, results = [torch.cuda.Stream() for _ in range(2)], []
    dev = [[t.cuda() for t in st] for st in state]
    xs, tb, ln = [y.cuda() for y in x], table.cuda(), lens.cuda()
    f = gdn.rope_frequencies(64)[0].cuda()
    torch.cuda.synchronize()
    for i in range(2):
        kw = dict(stream=streams[i])
        _, kr = gdn.rope(xs[i], xs[i], f, lens=ln, **kw)
        gdn.kv_append(kr, xs[i], dev[i][0], dev[i][1], tb, ln, k_scale=dev[i][2], v_scale=dev[i][3], **kw)
        results.append((kr, gdn.kv_read(dev[i][0], dev[i][1], tb, ln, 30, k_scale=dev[i][2], v_scale=dev[i][3], **kw)))
    torch.cuda.synchronize()
    for i in range(2):
        kr = results[i][0].cpu().view(-1, 2, 64)
        for y, (n, m) in zip((kr, x[i].view(-1, 2, 64)), ((0, 2), (1, 3))):
            want = append_ref(state[i][n], state[i][m], y, [30, 30], table, lens, "int8")
            assert torch.equal(dev[i][n].cpu(), want[0]) and torch.equal(dev[i][m].cpu(), want[1])
            assert torch.equal(results[i][1][n].cpu().view(-1, 2, 64), read_ref(*want, [30, 30], table, lens, torch.bfloat16))
