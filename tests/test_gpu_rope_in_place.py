"""gdn_rope in place and inside one buffer."""
import ctypes

import pytest
import torch

import gated_deltanet_state_delta_amd as gdn
import gated_deltanet_state_delta_amd._lib as L
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 48), (80, 20), (7, 2)])
def test_tokens_of_no_row_become_zeros(d, rot, interleaved):
    """All of their head, the dimensions behind rot among them; those of tokens of a row stay.  The binding asks for
    zeros in new outputs only: by the C ABI."""
    require_gpu()
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k = (torch.randn(20, h, d, generator=g, device="cuda").bfloat16() for h in (3, 1))
    f = gdn.rope_frequencies(rot)[0].cuda()
    where = dict(lens=torch.tensor([20, 30], dtype=torch.int32).cuda(), cu_seqlens=torch.tensor([3, 8, 12], dtype=torch.int32).cuda())
    want = gdn.rope(q, k, f, interleaved=interleaved, **where)
    assert all((y[:3] == 0).all() and (y[12:] == 0).all() for y in want)
    a, keep, _ = gdn.rope_args(q, k, f, interleaved=interleaved, out=(q, k), **where)
    a.zero_rest = 1
    assert L.load().gdn_rope(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


@pytest.mark.parametrize("order", [(0, 1, 2, 3), (2, 3, 0, 1), (3, 1, 0, 2)])
@pytest.mark.parametrize("pad", [0, 3])
def test_outputs_beside_the_inputs_in_one_buffer(order, pad):
    """q, k and their outputs as slices of [tokens, sum of their widths + pad], in each order; the rest stays."""
    require_gpu()
    n, d, heads = 37, 64, (4, 2, 4, 2)
    g = torch.Generator(device="cuda").manual_seed(2)
    buf = torch.randn(n, 12 * d + pad, generator=g, device="cuda").bfloat16()
    cut, at = [None] * 4, 0
    for i in order:
        cut[i] = buf[:, at:at + heads[i] * d].unflatten(1, (heads[i], d))
        at += heads[i] * d
    f, pos = gdn.rope_frequencies(48)[0].cuda(), torch.arange(100, 100 + n).cuda()
    q, k = (t.clone() for t in cut[:2])
    want = gdn.rope(q, k, f, positions=pos)
    rest = buf[:, at:].clone()
    got = gdn.rope(cut[0], cut[1], f, positions=pos, out=(cut[2], cut[3]))
    assert got[0] is cut[2] and torch.equal(cut[2], want[0]) and torch.equal(cut[3], want[1])
    assert torch.equal(cut[0], q) and torch.equal(cut[1], k) and torch.equal(buf[:, at:], rest)
