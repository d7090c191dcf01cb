"""attn_decode over tables that are split: the workspace of a call on streams at once, in captured graphs, and by
the short way, which allocates it for itself."""
import pytest
import torch

import gated_deltanet_state_delta_amd as gdn
from blocks_ref import CODE, attn_blocks_bound, attn_blocks_ref, blocks_cache
from gated_deltanet_state_delta_amd.paged import _short
from gpu_util import require_gpu
from paged_ref import caches, paged

pytestmark = pytest.mark.gpu
I32 = torch.int32
CASES = [("int8", 16, 16), ("e4m3", 16, 1), ("int8", 12, 4), ("bf16", 16, None)]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _state(cache, page, block, lens, d, hkv=2, seed=1):
    """Caches, page table and scales on the GPU; the table is as long as the longest row."""
    table, n_pages = paged(lens, page, seed=seed)
    if block is None:
        state, scales = caches(n_pages, page, hkv, d, cache, seed), (None, None)
    else:
        *state, ks, vs = blocks_cache(n_pages, page, hkv, d, block, cache, seed)
        scales = (ks.cuda(), vs.cuda())
    return [t.cuda() for t in state] + [table.cuda()], dict(k_scale=scales[0], v_scale=scales[1])


def _split(q, kc, vc, table, lens, **scales):
    """Whether a call is split (its rows' parts go through a workspace), by the short way."""
    assert _short("attn_decode", q, kc, vc, table, lens, None, *scales.values()) is not None
    return gdn.attn_decode_workspace_size(q, kc, vc, table, lens, **scales) > 0


@pytest.mark.parametrize("cache,page,block", CASES)
def test_two_streams_at_once(cache, page, block):
    lens = torch.tensor([3000, 40, 0, 1700], dtype=I32)
    (kc, vc, table), scales = _state(cache, page, block, lens, 128)
    lens = lens.cuda()
    g = torch.Generator(device="cuda").manual_seed(1)
    q = [torch.randn(4, 1, 8, 128, generator=g, device="cuda").bfloat16() for _ in range(2)]
    assert _split(q[0], kc, vc, table, lens, **scales)
    want = [gdn.attn_decode(x, kc, vc, table, lens, **scales) for x in q]
    torch.cuda.synchronize()
    assert not torch.equal(*want)
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(60):
        with torch.cuda.stream(streams[i % 2]):
            got.append(gdn.attn_decode(q[i % 2], kc, vc, table, lens, **scales))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i % 2]) for i, y in enumerate(got))


@pytest.mark.parametrize("cache,page,block", CASES)
def test_two_graphs_replayed_in_turn_and_at_once(cache, page, block):
    """Attention with its join in two graphs of one memory pool each, lengths and queries changing between replays,
    eager calls among them; then both on streams of their own."""
    rows, room = 3, [3100, 64, 2000]
    (kc, vc, table), scales = _state(cache, page, block, torch.tensor(room), 64)
    g = torch.Generator(device="cuda").manual_seed(2)
    draw = lambda: torch.randn(rows, 2, 6, 64, generator=g, device="cuda").bfloat16()
    lens = [torch.tensor(room, dtype=I32).cuda() for _ in range(2)]
    q = [draw(), draw()]
    assert _split(q[0], kc, vc, table, lens[0], **scales)
    graphs, outs = [], []
    for i in range(2):
        gdn.attn_decode(q[i], kc, vc, table, lens[i], **scales)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            outs.append(gdn.attn_decode(q[i], kc, vc, table, lens[i], **scales))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for step in range(8):
        for i in range(2):
            q[i].copy_(draw())
            lens[i].copy_(torch.tensor([[3100, 64, 2000], [1, 0, 1999], [2999, 3, 17], [700 * step % 3100, 64, 100 * step]][(step + i) % 4]))
        want = [gdn.attn_decode(q[i], kc, vc, table, lens[i], **scales) for i in range(2)]
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i] if step % 2 else torch.cuda.current_stream()):
                graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), step


@pytest.mark.parametrize("cache", ["e4m3", "int8"])
def test_a_growing_batch_captured_with_its_join(cache):
    """Append and attend in one graph over rows long enough to be split: every replay is one more token of each
    row, its bits those of eager calls on copies, and within bounds of 64 bits."""
    page, block, hkv, hq, d, room = 16, 8, 2, 4, 64, 1500
    start = [1400, 5, 700]
    (kc, vc, table), scales = _state(cache, page, block, torch.tensor([room] * 3), d, hkv, 3)
    lens = torch.tensor(start, dtype=I32).cuda()
    g = torch.Generator(device="cuda").manual_seed(3)
    draw = lambda h: torch.randn(3, 1, h, d, generator=g, device="cuda").bfloat16()
    q, k, v = draw(hq), draw(hkv), draw(hkv)
    assert _split(q, kc, vc, table, lens, **scales) and kc.dtype == CODE[cache]

    def step(kc, vc, lens, k_scale, v_scale):
        lens.add_(1)
        gdn.kv_append(k, v, kc, vc, table, lens, k_scale=k_scale, v_scale=v_scale)
        return gdn.attn_decode(q, kc, vc, table, lens, k_scale=k_scale, v_scale=v_scale)

    own = [kc, vc, lens, *scales.values()]
    step(*[t.clone() for t in own])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*own)
    for _ in range(5):
        for t, h in ((q, hq), (k, hkv), (v, hkv)):
            t.copy_(draw(h))
        other = [t.clone() for t in own]
        graph.replay()
        want = step(*other)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(own, other))
    state, n = [t.cpu() for t in (kc, vc, *scales.values())], lens.cpu()
    ref, _, mean, size = attn_blocks_ref(q.cpu(), *state, table.cpu(), n, d ** -0.5)
    assert ((out.double().cpu() - ref).abs() <= attn_blocks_bound(ref, mean, size, n, d, "bf16")).all()
