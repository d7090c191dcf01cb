"""The page-management calls on the GPU against the sequential references:
whole numbers, equal in every entry."""
import random

import pytest
import torch

import gated_deltanet_state_delta_amd as gdn
from gpu_util import require_gpu
from paged_ref import compact_ref, extend_ref, fork_ref, free_ref, random_state

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _same(got, want):
    assert len(got) == len(want)
    for i, (a, b) in enumerate(zip(got, want)):
        assert a.dtype == torch.int32 and a.cpu().tolist() == b, "output %d differs" % i


# rows, pages a row, page size, pages, pages shared by long rows
SIZES = [(1, 1, 1, 1, 0), (1, 3, 16, 2, 0), (5, 4, 16, 21, 2), (7, 3, 1, 9, 0), (40, 9, 5, 300, 3),
         (300, 17, 16, 1024, 1), (257, 40, 64, 5000, 0), (600, 12, 3, 4097, 2), (3, 700, 16, 1500, 5),
         (2500, 6, 16, 9000, 1)]


def _state(size, seed):
    rows, width, page, n_pages, shared = size
    return random_state(rows, width, page, n_pages, seed, shared=min(shared, width, n_pages))


def _cuda(*ts):
    return [t.cuda() for t in ts]


@pytest.mark.parametrize("seed", [0, 1])
@pytest.mark.parametrize("size", SIZES)
def test_extend(size, seed):
    table, lens, refs = _state(size, seed)
    r, page = random.Random(seed + 50), size[2]
    add = torch.tensor([r.choice([0, 1, 1, 4, page, 3 * page, -2, 1 << 30]) for _ in range(size[0])], dtype=torch.int32)
    want = extend_ref(table, lens, refs, add, page)
    t, n, f, a = _cuda(table, lens, refs, add)
    _same(gdn.pages_extend(t, n, f, a, page), want)
    assert torch.equal(t.cpu(), table) and torch.equal(n.cpu(), lens) and torch.equal(f.cpu(), refs)
    got = gdn.pages_extend(t, n, f, a, page, out=(t, n, f))
    assert got[0] is t and got[1] is n and got[2] is f
    _same(got, want)


@pytest.mark.parametrize("seed", [0, 1])
@pytest.mark.parametrize("size", SIZES)
def test_fork(size, seed):
    table, lens, refs = _state(size, seed)
    r = random.Random(seed + 70)
    rows = size[0]
    refs[r.randrange(size[3])] += 1  # a page held from outside the table
    parent = torch.tensor([r.choice([i, i, r.randrange(rows), -1, rows]) for i in range(rows)], dtype=torch.int32)
    want = fork_ref(table, lens, refs, parent, size[2])
    t, n, f, p = _cuda(table, lens, refs, parent)
    _same(gdn.pages_fork(t, n, f, p, size[2]), want)
    got = gdn.pages_fork(t, n, f, p, size[2], out=(torch.empty_like(t), torch.empty_like(n), f))  # counts in place
    assert got[2] is f
    _same(got, want)
    assert torch.equal(t.cpu(), table)


@pytest.mark.parametrize("seed", [0, 1])
@pytest.mark.parametrize("size", SIZES)
def test_free(size, seed):
    table, lens, refs = _state(size, seed)
    r = random.Random(seed + 90)
    mask = torch.tensor([r.random() < 0.5 for _ in range(size[0])])
    want = free_ref(table, lens, refs, mask, size[2])
    t, n, f, m = _cuda(table, lens, refs, mask)
    _same(gdn.pages_free(t, n, f, m, size[2]), want)
    _same(gdn.pages_free(t, n, f, m.to(torch.uint8), size[2], out=(t, n, f)), want)


@pytest.mark.parametrize("seed", [0, 1])
@pytest.mark.parametrize("size", SIZES)
def test_compact(size, seed):
    table, lens, refs = _state(size, seed)
    want = compact_ref(table, refs)
    t, f = _cuda(table, refs)
    _same(gdn.pages_compact(t, f), want)
    got = gdn.pages_compact(t, f, out=(t, f))
    _same(got, want)
    # a compact cache stays as it is
    again = gdn.pages_compact(t, f)
    assert torch.equal(again[0], t) and torch.equal(again[1], f) and (again[2] == -1).all()


def test_fork_every_kind_of_part_filled_page():
    """One page as the part-filled last page of several rows, as a whole page
    of another, and held from outside; more copies than free pages."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)
    table = i32([[0, 1], [0, 1], [2, 3], [2, -1], [4, -1], [-1, -1]])
    lens = i32([20, 20, 32, 9, 3, 0])
    refs = i32([2, 2, 2, 1, 2, 0, 0])
    for parent in ([0, 1, 2, 3, 4, 5], [0, 0, 2, 3, 4, 0], [3, 3, 3, 3, 3, 3], [4, 4, 4, 4, -1, -1], [1, 0, 3, 2, 5, 4]):
        want = fork_ref(table, lens, refs, i32(parent), 16)
        _same(gdn.pages_fork(*_cuda(table, lens, refs, i32(parent)), 16), want)


@pytest.mark.parametrize("call", ["extend", "fork", "free"])
def test_lengths_and_entries_outside_their_range(call):
    """Negative and over-long lengths are clamped, entries outside the cache
    are skipped, int64 inputs do not wrap."""
    table = torch.tensor([[0, 1 << 20, 2], [3, -7, 4], [5, 6, 7], [8, -1, -1]], dtype=torch.int64)
    lens = torch.tensor([1 << 40, 21, -5, 3], dtype=torch.int64)
    refs = torch.tensor([1, 0, 1, 1, 1, 0, 0, 0, 1, 0, 0], dtype=torch.int64)
    arg = {"extend": [1, 8, 9, 0], "fork": [1, 0, 1 << 33, 3], "free": [True, True, True, False]}[call]
    arg = torch.tensor(arg)
    ref = {"extend": extend_ref, "fork": fork_ref, "free": free_ref}[call]
    want = ref(table, lens.clamp(-1, 1 << 30), refs, [min(x, 99) if call != "free" else x for x in arg.tolist()], 8)
    _same(getattr(gdn, "pages_" + call)(*_cuda(table, lens, refs, arg), 8), want)


def test_needs_far_past_the_cache():
    """Rows that need more pages than there are: they and those behind them
    that need any are not served, the others are."""
    rows, n = 1300, 1000
    table = torch.full((rows, 64), -1, dtype=torch.int32)
    lens, refs = torch.zeros(rows, dtype=torch.int32), torch.zeros(n, dtype=torch.int32)
    r = random.Random(4)
    add = torch.tensor([r.choice([0, 0, 0, 1, 1]) for _ in range(rows)], dtype=torch.int32)
    add[700:] = torch.tensor([r.choice([0, 1, 64]) for _ in range(rows - 700)], dtype=torch.int32)
    want = extend_ref(table, lens, refs, add, 1)
    assert 0 < sum(want[3]) < rows
    _same(gdn.pages_extend(*_cuda(table, lens, refs, add), 1), want)


def test_strided_tables():
    table, lens, refs = _state(SIZES[4], 3)
    wide = torch.full((table.shape[0], table.shape[1] + 6), 99, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    w = wide.cuda()
    view = w[:, :table.shape[1]]
    add = torch.ones(table.shape[0], dtype=torch.int32)
    n, f, a = _cuda(lens, refs, add)
    want = extend_ref(table, lens, refs, add, 5)
    _same(gdn.pages_extend(view, n, f, a, 5, out=(view, n, f)), want)
    assert (w[:, table.shape[1]:] == 99).all()


def test_no_rows():
    e, z = torch.zeros((0, 3), dtype=torch.int32).cuda(), torch.zeros(0, dtype=torch.int32).cuda()
    refs = torch.tensor([0, 1, 0, 2], dtype=torch.int32).cuda()
    assert gdn.pages_extend(e, z, refs, z, 16)[2].tolist() == [0, 1, 0, 2]
    assert gdn.pages_fork(e, z, refs, z, 16)[2].tolist() == [0, 1, 0, 2]
    assert gdn.pages_free(e, z, refs, z.bool(), 16)[2].tolist() == [0, 1, 0, 2]
    _, packed, src, dst, n = gdn.pages_compact(e, refs)
    assert packed.tolist() == [2, 1, 0, 0] and src.tolist() == [3, -1] and dst.tolist() == [0, -1] and n.tolist() == [2]


@pytest.mark.parametrize("inner,dtype", [((16, 2, 64), torch.bfloat16), ((3,), torch.uint8), ((1,), torch.float32),
                                         ((4, 33, 7), torch.float32), ((40000,), torch.float32), ((12345,), torch.bfloat16),
                                         ((8, 128), torch.float8_e4m3fn)])
def test_copy(inner, dtype):
    """Whole pages of every size: the listed ones change, the others do not."""
    n = 23
    pool = (torch.randn(n, *inner, generator=torch.Generator().manual_seed(1)) * 50).clamp(-400, 400).to(dtype)
    order = torch.randperm(n, generator=torch.Generator().manual_seed(2)).to(torch.int32)
    src, dst = order[:9].clone(), order[9:18].clone()
    src[3], dst[5], src[6] = -1, n, 1 << 30
    want = pool.clone()
    bits = lambda t: t.contiguous().view(torch.uint8)
    for s, d in zip(src.tolist(), dst.tolist()):
        if 0 <= s < n and 0 <= d < n:
            bits(want)[d] = bits(pool)[s]
    got = pool.cuda()
    assert gdn.pages_copy(got, src.cuda(), dst.cuda()) is got
    assert torch.equal(bits(got.cpu()), bits(want))


def test_copy_strided_and_permuted_pools_and_long_lists():
    wide = torch.randn(10, 100, generator=torch.Generator().manual_seed(1)).cuda()
    view, before = wide[:, 3:50], wide.clone()
    s, d = torch.tensor([0, 5], dtype=torch.int64).cuda(), torch.tensor([9, 2], dtype=torch.int64).cuda()
    gdn.pages_copy(view, s, d)
    before[[9, 2], 3:50] = before[[0, 5], 3:50]
    assert torch.equal(wide, before)
    heads_first = torch.randn(6, 2, 16, 32).cuda()
    want = heads_first.clone()
    want[4] = want[1]
    gdn.pages_copy(heads_first.transpose(1, 2), torch.tensor([1]).cuda(), torch.tensor([4]).cuda())
    assert torch.equal(heads_first, want)
    src = torch.full((50000,), -1, dtype=torch.int32)  # a padded list
    dst = src.clone()
    src[49999], dst[49999] = 0, 3
    want[3] = want[0]
    gdn.pages_copy(heads_first, src.cuda(), dst.cuda())
    assert torch.equal(heads_first, want)
    gdn.pages_copy(heads_first, src[:0].cuda(), dst[:0].cuda())
    assert torch.equal(heads_first, want)


def test_captured_calls_follow_their_inputs():
    """extend and fork in one graph, replayed over changing inputs."""
    size = SIZES[4]
    table, lens, refs = _state(size, 5)
    rows, page = size[0], size[2]
    t, n, f = _cuda(table, lens, refs)
    add = torch.ones(rows, dtype=torch.int32).cuda()
    parent = torch.arange(rows, dtype=torch.int32).cuda()
    gdn.pages_extend(t, n, f, add, page)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        e = gdn.pages_extend(t, n, f, add, page)
        k = gdn.pages_fork(e[0], e[1], e[2], parent, page)
    for step in range(4):
        r = random.Random(step)
        a = torch.tensor([r.choice([0, 1, 2, 7]) for _ in range(rows)], dtype=torch.int32)
        p = torch.tensor([r.choice([i, r.randrange(rows), -1]) for i in range(rows)], dtype=torch.int32)
        add.copy_(a), parent.copy_(p)
        graph.replay()
        torch.cuda.synchronize()
        want = extend_ref(table, lens, refs, a, page)
        _same(e, want)
        tt = [torch.tensor(x, dtype=torch.int32) for x in want[:3]]
        _same(k, fork_ref(*tt, p, page))
        table, lens, refs = (x.cpu() for x in k[:3])
        t.copy_(table), n.copy_(lens), f.copy_(refs)
