"""gdn_kv_append on the GPU: every written element equals the input (or its
e4m3 rounding by the division's definition), and nothing else changes."""
import pytest
import torch

import gated_deltanet_state_delta_amd as gdn
from gpu_util import require_gpu
from paged_ref import DT, caches, paged

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _bits(t):
    """The bits of a tensor, every NaN as one."""
    t = t.cpu()
    return torch.where(t.isnan(), torch.full_like(t.float(), 12345.0), t.float())


def _want(cache, x, counts, table, lens, page, scale):
    """The cache after the append, one token at a time."""
    c = cache.float().clone()
    at = 0
    for b, n in enumerate(counts):
        for i in range(n):
            pos = int(lens[b]) - n + i
            if 0 <= pos < table.shape[1] * page and 0 <= int(table[b, pos // page]) < c.shape[0]:
                y = x[at].float()
                if scale is not None:
                    y = (y / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).float()
                c[int(table[b, pos // page]), pos % page] = y
            at += 1
    return c


def _run(counts, lens, page, hkv, d, io, cache, packed, seed=0, heads_first=False, table=None, width=None):
    g = torch.Generator().manual_seed(seed)
    if table is None:
        table, n_pages = paged(lens, page, seed=seed, width=width)
    else:
        n_pages = 16
    kc, vc = caches(n_pages, page, hkv, d, cache, seed, heads_first=heads_first)
    total = sum(counts)
    k, v = (torch.randn(total, hkv, d, generator=g).to(DT[io]) for _ in range(2))
    ks = vs = None
    if cache == "e4m3":
        ks, vs = torch.rand(hkv, generator=g) * 0.02 + 0.001, torch.rand(hkv, generator=g) * 0.02 + 0.001
        k.view(-1)[:7] = torch.tensor([float("inf"), -float("inf"), float("nan"), 0.0, -0.0, 1e-6, 3e4])
    lens_t = torch.tensor(lens, dtype=torch.int32)
    want = [_want(c, x, counts, table, lens_t, page, s) for c, x, s in ((kc, k, ks), (vc, v, vs))]
    cu = None
    if packed:
        cu = torch.tensor([0] + [sum(counts[:i + 1]) for i in range(len(counts))], dtype=torch.int32).cuda()
    else:
        k, v = (x.view(len(counts), counts[0], hkv, d) for x in (k, v))
    dev = lambda c: c.transpose(1, 2).contiguous().cuda().transpose(1, 2) if heads_first else c.cuda()
    kd, vd = dev(kc), dev(vc)
    got = gdn.kv_append(k.cuda(), v.cuda(), kd, vd, table.cuda(), lens_t.cuda(), cu_seqlens=cu,
                        k_scale=None if ks is None else ks.cuda(), v_scale=None if vs is None else vs.cuda())
    assert got[0] is kd and got[1] is vd
    for a, b in zip(got, want):
        assert torch.equal(_bits(a), _bits(b))


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("io,cache", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "e4m3"), ("f32", "e4m3")])
def test_one_token_a_row(io, cache, d):
    _run([1] * 5, [1, 16, 17, 40, 0], 16, 3, d, io, cache, packed=False, seed=d)


@pytest.mark.parametrize("page", [1, 5, 16, 64])
@pytest.mark.parametrize("io,cache", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "e4m3")])
def test_packed_prompts(io, cache, page):
    """Ragged rows, empty ones among them, some continuing a longer row; one
    whose new tokens begin before its start (not written)."""
    _run([0, 70, 1, 0, 33, 5, 0], [9, 70, 30, 0, 50, 3, 2], page, 2, 64, io, cache, packed=True, seed=page)


def test_many_tokens_and_several_runs_a_workgroup():
    counts = [1500, 0, 2049, 700]
    _run(counts, [1500, 5, 2100, 700], 16, 1, 32, "bf16", "bf16", packed=True, seed=1)


def test_several_tokens_heads_first_and_table_limits():
    _run([3] * 4, [3, 20, 40, 2], 8, 2, 64, "bf16", "bf16", packed=False, seed=2, heads_first=True)
    # entries outside the cache, and positions past the table, are skipped
    table = torch.tensor([[-1, 3], [4, 16], [5, 6]], dtype=torch.int32)
    _run([12] * 3, [12, 14, 30], 8, 2, 64, "f32", "f32", packed=False, seed=3, table=table)


def test_every_e4m3_value_and_the_ties_between_them():
    """Each stored value, the middle of each pair of neighbours (ties to even)
    and the values next to it, at scale 1."""
    v = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    mid = (v[1:] + v[:-1]) / 2
    x = torch.cat([v, mid, torch.nextafter(mid, torch.tensor(0.0)), torch.nextafter(mid, torch.tensor(1e9))])
    x = torch.cat([x, -x, torch.tensor([448.0, 464.0, 465.0, 1e9])])
    x = torch.nn.functional.pad(x, (0, -x.numel() % 32)).view(-1, 1, 32)
    n = x.shape[0]
    kc = torch.zeros(1, n, 1, 32).to(torch.float8_e4m3fn).cuda()
    vc = kc.clone()
    one = torch.ones(1).cuda()
    gdn.kv_append(x[None].cuda(), x[None].cuda(), kc, vc, torch.zeros(1, 1, dtype=torch.int32).cuda(),
                  torch.tensor([n], dtype=torch.int32).cuda(), k_scale=one, v_scale=one)
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).float()
    assert torch.equal(kc.cpu().float().view(-1), want.view(-1)) and torch.equal(vc.cpu().float(), kc.cpu().float())


def test_offsets_clamped_and_strided_input():
    """cu_seqlens outside [0, tokens] are clamped, a decreasing pair is empty,
    tokens of no row are not written; k and v may be parts of one projection."""
    table, n_pages = paged([8, 8, 8], 8)
    kc, vc = caches(n_pages, 8, 2, 64, "bf16", 3)
    qkv = torch.randn(10, 6, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
    k, v = qkv[:, 2:4], qkv[:, 4:]
    cu = torch.tensor([3, 2, 6, 99], dtype=torch.int64)  # rows: none, 2..5, 6..9
    lens = torch.tensor([8, 8, 4], dtype=torch.int32)
    want = [c.float().clone() for c in (kc, vc)]
    for w, x in zip(want, (k, v)):
        for i in range(4):
            w[int(table[1, 0]), 4 + i] = x[2 + i].float()
            w[int(table[2, 0]), i] = x[6 + i].float()
    dq = qkv.cuda()
    got = gdn.kv_append(dq[:, 2:4], dq[:, 4:], kc.cuda(), vc.cuda(), table.cuda(), lens.cuda(), cu_seqlens=cu.cuda())
    for a, b in zip(got, want):
        assert torch.equal(a.float().cpu(), b)


def test_parts_of_a_projection_and_a_given_stream():
    """[B, T, hkv, d] slices of one projection, on a stream of their own."""
    table, n_pages = paged([9, 20], 8)
    kc, vc = caches(n_pages, 8, 2, 64, "f32", 3)
    qkv = torch.randn(2, 3, 8, 64, generator=torch.Generator().manual_seed(1))
    lens = torch.tensor([9, 20], dtype=torch.int32)
    want = [_want(c, qkv[:, :, i:i + 2].reshape(6, 2, 64), [3, 3], table, lens, 8, None) for c, i in ((kc, 4), (vc, 6))]
    dq, k, v, t, n = (x.cuda() for x in (qkv, kc, vc, table, lens))
    free = min(set(range(n_pages)) - set(table.flatten().tolist()))
    want[0][free] = want[0][int(table[0, 0])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gdn.kv_append(dq[:, :, 4:6], dq[:, :, 6:8], k, v, t, n, stream=side)
    gdn.pages_copy(k, t[0, :1], torch.tensor([free], dtype=torch.int32).cuda(), stream=side)
    side.synchronize()
    assert torch.equal(k.cpu(), want[0]) and torch.equal(v.cpu(), want[1])


def test_nothing_to_write():
    kc, vc = (c.cuda() for c in caches(2, 16, 2, 64, "bf16", 3))
    before = kc.clone()
    k = torch.randn(0, 2, 64).bfloat16().cuda()
    gdn.kv_append(k, k, kc, vc, torch.zeros(1, 1, dtype=torch.int32).cuda(), torch.ones(1, dtype=torch.int32).cuda(),
                  cu_seqlens=torch.zeros(2, dtype=torch.int32).cuda())
    assert torch.equal(kc, before)


@pytest.mark.parametrize("rows,hkv", [(64, 4), (3, 1), (1, 2)])
@pytest.mark.parametrize("io,cache", [("bf16", "bf16"), ("f32", "f32"), ("f32", "e4m3")])
def test_steps_of_a_sequence_first_buffer(io, cache, rows, hkv):
    """[B, 1, hkv, d] views of [steps, B, hkv, d]: contiguous to torch, with the
    steps' stride in the dimension of one token."""
    lens = [b % 30 + 1 for b in range(rows)]
    table, n_pages = paged(lens, 16, seed=rows)
    kc, vc = caches(n_pages, 16, hkv, 64, cache, seed=rows)
    g = torch.Generator().manual_seed(rows)
    k, v = (torch.randn(3, rows, hkv, 64, generator=g).to(DT[io]) for _ in range(2))
    s = torch.rand(hkv, generator=g) * 0.02 + 0.001 if cache == "e4m3" else None
    sd = None if s is None else s.cuda()
    lens = torch.tensor(lens, dtype=torch.int32)
    for i in range(3):
        want = [_want(c, x[i], [1] * rows, table, lens, 16, s) for c, x in ((kc, k), (vc, v))]
        step = [x.cuda()[i:i + 1].transpose(0, 1) for x in (k, v)]
        got = gdn.kv_append(*step, kc.cuda(), vc.cuda(), table.cuda(), lens.cuda(), k_scale=sd, v_scale=sd)
        for a, b in zip(got, want):
            assert torch.equal(_bits(a), b)


@pytest.mark.parametrize("cu", [[5, 10, 0, 3], [0, 10, 5, 20], [20, 15, 10, 0], [0, 20, 20, 7, 7, 30, -4, 12], [9, 9, 2, 18, 1, 4]])
def test_offsets_that_decrease_write_nothing_astray(cu):
    """Tokens may be left out, but each that is written lies where its row has
    it, and no other slot changes."""
    rows, total, page = len(cu) - 1, 20, 8
    lens = [20 - 3 * (b % 3) for b in range(rows)]
    table, n_pages = paged(lens, page, seed=7)
    kc, vc = caches(n_pages, page, 2, 32, "f32", 3)
    k, v = (torch.randn(total, 2, 32, generator=torch.Generator().manual_seed(i)) for i in range(2))
    got = gdn.kv_append(k.cuda(), v.cuda(), kc.cuda(), vc.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                        cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    at = [min(max(x, 0), total) for x in cu]
    for old, x, new in ((kc, k, got[0].cpu()), (vc, v, got[1].cpu())):
        for b in range(rows):
            n = max(0, at[b + 1] - at[b])
            for i in range(n):
                pos = lens[b] - n + i
                if pos < 0:
                    continue
                slot = new[int(table[b, pos // page]), pos % page]
                if torch.equal(slot, x[at[b] + i]):
                    slot.copy_(old[int(table[b, pos // page]), pos % page])
        assert torch.equal(new, old)
