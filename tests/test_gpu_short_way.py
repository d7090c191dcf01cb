"""The short way into libgdn (binding/calls.cpp) on the GPU: what a program keeps without it."""
import pytest
import torch

import gated_deltanet_state_delta_amd as gdn
import gated_deltanet_state_delta_amd._lib as L
from blocks_ref import blocks_cache
from gated_deltanet_state_delta_amd.paged import _short
from gpu_util import require_gpu
from paged_ref import paged

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _state(lens=(40, 3, 0, 100), page=16, hkv=2, d=64, cache="int8", block=16):
    lens = torch.tensor(lens, dtype=I32)
    table, n_pages = paged(lens, page, seed=1)
    kc, vc, ks, vs = (t.cuda() for t in blocks_cache(n_pages, page, hkv, d, block, cache, 1))
    return (kc, vc, table.cuda(), lens.cuda()), dict(k_scale=ks, v_scale=vs)


def test_every_call_works_without_the_module(monkeypatch):
    args, scales = _state()
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(4, 1, h, 64, generator=g, device="cuda").bfloat16() for h in (6, 2, 2))
    f = gdn.rope_frequencies(64)[0].cuda()

    def run():
        c = [t.clone() for t in args[:2]]
        s = {n: t.clone() for n, t in scales.items()}
        gdn.kv_append(k, v, *c, *args[2:], **s)
        return [gdn.attn_decode(q, *args, **scales), *gdn.kv_read(*args, 3, **scales), *gdn.rope(q, k, f, lens=args[3]), *c, *s.values()]

    want = run()
    monkeypatch.setattr(L, "_calls", None)
    monkeypatch.setattr(L, "_no_calls", True)
    assert _short("rope", q, k, f, args[3], None, None, False, 1.0) is None
    assert all(torch.equal(a, b) for a, b in zip(want, run()))
