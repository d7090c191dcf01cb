"""The short way into libgdn (binding/calls.cpp) on the GPU: what a program keeps without it."""
import ctypes
import threading

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


def _entries(lib):
    return [ctypes.cast(getattr(lib, "gdn_" + n), ctypes.c_void_p).value
            for n in ("header_digest", "attn_decode", "attn_decode_workspace_size", "kv_append", "kv_read", "rope")]


def test_other_threads_run_while_libgdn_does():
    """With the interpreter's own check of its lock in the place of libgdn's entries (nothing is launched): 0, as
    GDN_OK, where the calling thread does not hold it."""
    args, scales = _state()
    q, k = torch.randn(4, 1, 6, 64).bfloat16().cuda(), torch.randn(4, 1, 2, 64).bfloat16().cuda()
    f = gdn.rope_frequencies(64)[0].cuda()
    ks, vs = scales.values()
    module, entries = L.calls(), _entries(L.load())
    check = ctypes.cast(ctypes.pythonapi.PyGILState_Check, ctypes.c_void_p).value
    try:
        module.bind(entries[0], *[check] * 5)
        got = [_short("attn_decode", q, *args, None, ks, vs), _short("kv_append", k, k, *args, None, ks, vs),
               _short("kv_read", *args, 3, None, 1, ks, vs), _short("rope", q, k, f, args[3], None, None, False, 1.0)]
    finally:
        module.bind(*entries)
    assert all(x is not None for x in got)


def test_calls_of_several_threads():
    args, scales = _state((3000, 40, 700, 1))
    g = torch.Generator(device="cuda").manual_seed(1)
    q = [torch.randn(4, 1, 6, 64, generator=g, device="cuda").bfloat16() for _ in range(4)]
    f = gdn.rope_frequencies(64)[0].cuda()
    call = lambda x: [gdn.attn_decode(x, *args, **scales), *gdn.kv_read(*args, 30, **scales), gdn.rope(x, None, f, lens=args[3])[0]]
    want = [call(x) for x in q]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                got = call(q[i])
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
