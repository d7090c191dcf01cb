"""gdn_rope in place with zero_rest, which the binding does not ask for: by the C ABI."""
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
    """All of their head, the dimensions behind rot among them; those of tokens of a row stay."""
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
