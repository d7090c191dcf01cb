"""The paged-cache calls together, as a server of a model with both kinds of
layers uses them: prompts appended, rows grown, forked, freed and compacted
while tokens are attended, the gated-delta-rule states of forked rows copied
along; every attention checked against plain histories of each row."""
import random

import pytest
import torch

import gated_deltanet_state_delta_amd as gdn
from gpu_util import require_gpu
from paged_ref import attn_bound, attn_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("page,cache", [(16, torch.bfloat16), (5, torch.float32)])
def test_a_batch_lives_through_prompts_forks_and_compaction(page, cache):
    rows, width, hkv, hq, d, n_pages = 6, 12, 2, 4, 64, 80
    r = random.Random(page)
    gen = torch.Generator().manual_seed(page)
    draw = lambda *s: torch.randn(*s, generator=gen).to(cache)
    kc, vc = (torch.full((n_pages, page, hkv, d), float("nan"), dtype=cache).cuda() for _ in range(2))
    table = torch.full((rows, width), -1, dtype=torch.int32).cuda()
    lens, refs = torch.zeros(rows, dtype=torch.int32).cuda(), torch.zeros(n_pages, dtype=torch.int32).cuda()
    hist = [(torch.zeros(0, hkv, d), torch.zeros(0, hkv, d)) for _ in range(rows)]  # what each row has seen
    # the states of the other kind of layer, one slot a row
    state = torch.randn(rows, 2, 16, 16, generator=gen).cuda()
    states = state.cpu()

    def grow(counts):
        nonlocal table, lens, refs
        table, lens, refs, ok = gdn.pages_extend(table, lens, refs, torch.tensor(counts, dtype=torch.int32).cuda(), page)
        # a row that would outgrow its table stays as it is; there are pages for all others
        fits = [h[0].shape[0] + c <= width * page for h, c in zip(hist, counts)]
        assert ok.tolist() == fits
        counts = [c if f else 0 for c, f in zip(counts, fits)]
        k, v = draw(sum(counts), hkv, d), draw(sum(counts), hkv, d)
        cu = torch.tensor([sum(counts[:i]) for i in range(rows + 1)], dtype=torch.int32)
        gdn.kv_append(k.cuda(), v.cuda(), kc, vc, table, lens, cu_seqlens=cu.cuda())
        for b in range(rows):
            hist[b] = tuple(torch.cat([h, x[cu[b]:cu[b + 1]].float()]) for h, x in zip(hist[b], (k, v)))

    def attend(T):
        q = draw(rows, T, hq, d)
        got = gdn.attn_decode(q.cuda(), kc, vc, table, lens).double().cpu()
        assert lens.tolist() == [h[0].shape[0] for h in hist]
        for b in range(rows):  # a row's own history as one page of its own
            n = hist[b][0].shape[0]
            own = [torch.zeros(1, max(n, 1), hkv, d, dtype=cache) for _ in range(2)]
            for c, h in zip(own, hist[b]):
                c[0, :n] = h.to(cache)
            ln = torch.tensor([n])
            want, _, mean, size = attn_ref(q[b:b + 1], *own, torch.zeros(1, 1, dtype=torch.int32), ln, 0.125)
            bound = attn_bound(want, mean, size, ln, d, "bf16" if cache == torch.bfloat16 else "f32")
            assert ((got[b:b + 1] - want).abs() <= bound).all(), b

    grow([40, 0, 17, 3, 55, 16])
    attend(1)
    for step in range(12):
        kind = step % 4
        if kind in (0, 2):
            T = r.choice([1, 3])
            grow([T] * rows)
            attend(T)
        elif kind == 1:  # beams: some rows continue from others
            parent = [r.choice([i, r.randrange(rows)]) for i in range(rows)]
            p = torch.tensor(parent, dtype=torch.int32).cuda()
            table, lens, refs, src, dst = gdn.pages_fork(table, lens, refs, p, page)
            for c in (kc, vc):
                gdn.pages_copy(c, src, dst)
            hist = [hist[i] for i in parent]
            # states have no sharing: a second pool receives every row's parent
            both = torch.cat([state, torch.zeros_like(state)])
            gdn.pages_copy(both, p, torch.arange(rows, 2 * rows, dtype=torch.int32).cuda())
            state = both[rows:].contiguous()
            states = states[parent]
            assert torch.equal(state.cpu(), states)
            attend(1)
        else:
            drop = torch.tensor([r.random() < 0.3 for _ in range(rows)])
            table, lens, refs = gdn.pages_free(table, lens, refs, drop.cuda(), page)
            hist = [(h[0][:0], h[1][:0]) if drop[b] else h for b, h in enumerate(hist)]
            table, refs, src, dst, n_live = gdn.pages_compact(table, refs)
            for c in (kc, vc):
                gdn.pages_copy(c, src, dst)
            live = int(n_live)
            assert (refs[:live] > 0).all() and (refs[live:] == 0).all() and int(table.max()) < live
            attend(1)
    table, lens, refs = gdn.pages_free(table, lens, refs, torch.ones(rows, dtype=torch.bool).cuda(), page)
    assert int(refs.abs().sum()) == 0 and int(lens.sum()) == 0


def test_a_decode_step_captured_once_and_replayed():
    """Grow, append and attend in one graph, in place: every replay is one more
    token of each row, checked against the rows' histories."""
    rows, width, page, hkv, hq, d, n_pages = 4, 8, 16, 2, 8, 128, 40
    gen = torch.Generator().manual_seed(1)
    draw = lambda *s: torch.randn(*s, generator=gen).bfloat16()
    kc, vc = (torch.zeros(n_pages, page, hkv, d, dtype=torch.bfloat16).cuda() for _ in range(2))
    table = torch.full((rows, width), -1, dtype=torch.int32).cuda()
    lens, refs = torch.zeros(rows, dtype=torch.int32).cuda(), torch.zeros(n_pages, dtype=torch.int32).cuda()
    one = torch.ones(rows, dtype=torch.int32).cuda()
    start = [14, 0, 31, 60]
    _, _, _, ok = gdn.pages_extend(table, lens, refs, torch.tensor(start, dtype=torch.int32).cuda(), page, out=(table, lens, refs))
    k, v = draw(sum(start), hkv, d), draw(sum(start), hkv, d)
    cu = [sum(start[:i]) for i in range(rows + 1)]
    gdn.kv_append(k.cuda(), v.cuda(), kc, vc, table, lens, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    hist = [(k[cu[b]:cu[b + 1]], v[cu[b]:cu[b + 1]]) for b in range(rows)]
    q1, k1, v1 = (torch.zeros(rows, 1, h, d, dtype=torch.bfloat16).cuda() for h in (hq, hkv, hkv))
    gdn.attn_decode(q1, kc, vc, table, lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.pages_extend(table, lens, refs, one, page, out=(table, lens, refs))
        gdn.kv_append(k1, v1, kc, vc, table, lens)
        out = gdn.attn_decode(q1, kc, vc, table, lens)
    for step in range(6):
        q, k, v = draw(rows, 1, hq, d), draw(rows, 1, hkv, d), draw(rows, 1, hkv, d)
        q1.copy_(q), k1.copy_(k), v1.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        got = out.double().cpu()
        assert torch.equal(gdn.attn_decode(q1, kc, vc, table, lens), out)  # eager work between the replays
        for b in range(rows):
            hist[b] = tuple(torch.cat([h, x[b]]) for h, x in zip(hist[b], (k, v)))
            ln = torch.tensor([start[b] + step + 1])
            want, _, mean, size = attn_ref(q[b:b + 1], hist[b][0][None], hist[b][1][None], torch.zeros(1, 1, dtype=torch.int32),
                                           ln, d ** -0.5)
            assert ((got[b:b + 1] - want).abs() <= attn_bound(want, mean, size, ln, d, "bf16")).all(), (step, b)
    assert lens.tolist() == [s + 6 for s in start] and int(refs.sum()) == sum(-(-(s + 6) // page) for s in start)
