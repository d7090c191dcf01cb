"""gdn_rope on the GPU against 64 bits: layouts of pairs, sizes and strides,
positions near and far, in place, tokens of no row."""
import pytest
import torch

import gated_deltanet_state_delta_amd as gdn
from blocks_ref import rope_bound, rope_ref
from gpu_util import require_gpu
from paged_ref import DT

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _draw(shape, io, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(DT[io])


def _check(got, x, pos, f, interleaved, factor, io):
    want, size = rope_ref(x.reshape(-1, *x.shape[-2:]), pos, f, interleaved, factor)
    got = got.double().cpu().reshape(want.shape)
    bound = rope_bound(want, size, pos, f, io)
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), "%d values off, worst by %.2f bounds" % (bad.sum(), ((got - want).abs() / bound).max())
    rot = 2 * f.shape[0]
    assert torch.equal(got[..., rot:], want[..., rot:])  # copied


@pytest.mark.parametrize("d,rot", [(64, 64), (128, 64), (128, 128), (256, 128), (96, 24), (80, 20), (80, 80), (30, 14), (7, 2), (7, 6),
                                   (192, 64), (1024, 1024), (16, 4), (8, 8), (2, 2)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_sizes(io, interleaved, d, rot):
    f, _ = gdn.rope_frequencies(rot)
    q, k = _draw((3, 2, 5, d), io, d), _draw((3, 2, 3, d), io, rot)
    lens = torch.tensor([2, 1, 70000], dtype=torch.int32)  # the second row's first token is at -1
    pos = torch.tensor([0, 1, -1, 0, 69998, 69999])
    got = gdn.rope(q.cuda(), k.cuda(), f.cuda(), lens=lens.cuda(), interleaved=interleaved, factor=1.25)
    for x, y in zip((q, k), got):
        assert y.shape == x.shape and y.dtype == x.dtype
        _check(y, x, pos, f, interleaved, 1.25, io)


@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_given_positions_near_and_far(io, kind):
    far = (1 << 31) - 1 if kind == torch.int32 else 1 << 40
    pos = torch.tensor([0, 1, 17, 4095, 131071, (1 << 20) + 7, -3, far], dtype=kind)
    f, _ = gdn.rope_frequencies(64, base=5e5)
    q = _draw((8, 4, 128), io, 1)
    y, none = gdn.rope(q.cuda(), None, f.cuda(), positions=pos.cuda())
    assert none is None
    _check(y, q, pos, f, False, 1.0, io)
    y, _ = gdn.rope(q.cuda().view(2, 4, 4, 128), None, f.cuda(), positions=pos.cuda().view(2, 4))
    _check(y, q, pos, f, False, 1.0, io)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("counts", [[1], [0, 3, 0, 1, 40, 0], [700, 2, 900], [1] * 300, [5000]])
def test_packed_rows(counts, interleaved):
    ends = [n + 11 * i for i, n in enumerate(counts)]
    pos = torch.cat([torch.arange(e - n, e) for e, n in zip(ends, counts)])
    cu = torch.tensor([sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int64)
    f, m = gdn.rope_frequencies(32, scaling="parts", scale=16, trained=128)
    q, k = _draw((sum(counts), 2, 64), "bf16", 1), _draw((sum(counts), 1, 64), "bf16", 2)
    got = gdn.rope(q.cuda(), k.cuda(), f.cuda(), lens=torch.tensor(ends).cuda(), cu_seqlens=cu.cuda(), interleaved=interleaved, factor=m)
    for x, y in zip((q, k), got):
        _check(y, x, pos, f, interleaved, m, "bf16")


@pytest.mark.parametrize("pad", [0, 8, 3])
@pytest.mark.parametrize("interleaved", [False, True])
def test_slices_of_one_projection_in_place_and_apart(interleaved, pad):
    """Queries and keys inside [tokens, (hq + 2 hkv) d + pad], whose values stay."""
    hq, hkv, d, n = 4, 2, 64, 37
    fused = _draw((n, (hq + 2 * hkv) * d + pad), "bf16", pad)
    cut = lambda t: (t[:, :hq * d].unflatten(1, (hq, d)), t[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)))
    pos, f = torch.arange(100, 100 + n), gdn.rope_frequencies(48)[0]
    dev = fused.cuda()
    apart = gdn.rope(*cut(dev), f.cuda(), positions=pos.cuda(), interleaved=interleaved)
    assert torch.equal(dev.cpu(), fused)
    q, k = cut(dev)
    same = gdn.rope(q, k, f.cuda(), positions=pos.cuda(), interleaved=interleaved, out=(q, k))
    assert same[0] is q and same[1] is k
    for x, a, b in zip(cut(fused), apart, same):
        _check(a, x, pos, f, interleaved, 1.0, "bf16")
        assert torch.equal(a.cpu(), b.cpu())
    assert torch.equal(dev[:, (hq + hkv) * d:].cpu(), fused[:, (hq + hkv) * d:])
    # one of them in place, and an output with heads before tokens
    to = torch.zeros(hkv, n, d, dtype=torch.bfloat16).cuda().transpose(0, 1)
    dev = fused.cuda()
    q, k = cut(dev)
    gdn.rope(q, k, f.cuda(), positions=pos.cuda(), interleaved=interleaved, out=(q, to))
    assert torch.equal(q, apart[0]) and torch.equal(to, apart[1]) and torch.equal(k.cpu(), cut(fused)[1])


def test_rows_that_are_not_one_stride_apart_and_misaligned_ones():
    f, lens = gdn.rope_frequencies(64)[0], torch.tensor([9, 30], dtype=torch.int32)
    pos = torch.tensor([6, 7, 8, 27, 28, 29])
    base = _draw((2, 5, 4, 64), "f32", 1)
    y, _ = gdn.rope(base.cuda()[:, 1:4], None, f.cuda(), lens=lens.cuda())
    _check(y, base[:, 1:4], pos, f, False, 1.0, "f32")
    flat = torch.zeros(2 * 3 * 4 * 64 + 1, dtype=torch.bfloat16).cuda()
    x = flat[1:].view(2, 3, 4, 64)
    x.copy_(base[:, 1:4])
    y, _ = gdn.rope(x, None, f.float().cuda(), lens=lens.cuda())
    _check(y, x.cpu(), pos, f.float().double(), False, 1.0, "bf16")


def test_tokens_of_no_row():
    """Left as they were in given outputs, zeros in new ones; offsets that decrease leave tokens out."""
    f, lens = gdn.rope_frequencies(64)[0].cuda(), torch.tensor([20, 30], dtype=torch.int32)
    q, k = _draw((20, 2, 64), "bf16", 1), _draw((20, 1, 64), "bf16", 2)
    pos = torch.cat([torch.arange(15, 20), torch.arange(26, 30)])
    cu = torch.tensor([3, 8, 12], dtype=torch.int32)
    given = tuple(torch.full_like(x, 7.0).cuda() for x in (q, k))
    kept = gdn.rope(q.cuda(), k.cuda(), f, lens=lens.cuda(), cu_seqlens=cu.cuda(), out=given)
    new = gdn.rope(q.cuda(), k.cuda(), f, lens=lens.cuda(), cu_seqlens=cu.cuda())
    for out, rest in ((kept, 7.0), (new, 0.0)):
        for x, y in zip((q, k), out):
            _check(y[3:12], x[3:12], pos, f.cpu(), False, 1.0, "bf16")
            assert (y[:3] == rest).all() and (y[12:] == rest).all()
    y, _ = gdn.rope(q.cuda(), None, f, lens=lens.cuda(), cu_seqlens=torch.tensor([12, 3, 8], dtype=torch.int32).cuda())
    _check(y[3:8], q[3:8], torch.arange(25, 30), f.cpu(), False, 1.0, "bf16")
    assert (y[:3] == 0).all() and (y[8:] == 0).all()


def test_values_that_are_not_numbers_stay_in_their_pair():
    f, q = gdn.rope_frequencies(32)[0], _draw((1, 2, 64), "f32", 1)
    clean = gdn.rope(q.cuda(), None, f.cuda(), positions=torch.tensor([5]).cuda())[0].cpu()
    q[0, 0, 3], q[0, 0, 40], q[0, 1, 20] = float("nan"), float("nan"), float("inf")
    y = gdn.rope(q.cuda(), None, f.cuda(), positions=torch.tensor([5]).cuda())[0].cpu()
    odd = torch.zeros(1, 2, 64, dtype=torch.bool)
    odd[0, 0, [3, 19, 40]] = odd[0, 1, [4, 20]] = True
    assert torch.equal(y[~odd], clean[~odd]) and not y[odd].isfinite().any()


def test_no_tokens():
    f = gdn.rope_frequencies(32)[0].cuda()
    y, z = gdn.rope(torch.zeros(0, 2, 64).cuda(), torch.zeros(0, 1, 64).cuda(), f, positions=torch.zeros(0, dtype=torch.int64).cuda())
    assert y.shape == (0, 2, 64) and z.shape == (0, 1, 64)
    y, _ = gdn.rope(torch.zeros(0, 1, 2, 64).cuda(), None, f, lens=torch.zeros(0, dtype=torch.int32).cuda())
    assert y.shape == (0, 1, 2, 64)
