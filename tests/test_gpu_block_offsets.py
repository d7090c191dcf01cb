"""kv_append over block scales with offsets that decrease: codes and scales of keys and of values."""
import pytest
import torch

import gated_deltanet_state_delta_amd as gdn
from blocks_ref import append_ref, blocks_cache
from gpu_util import require_gpu
from paged_ref import paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cu", [[0, 20, 10, 30], [-5, 12, 50, 30], [30, 20, 10, 0], [0, 40, 40, 40], [5, 9, 9, 20], [0, 10, 20, 30]])
@pytest.mark.parametrize("block", [1, 4, 16])
@pytest.mark.parametrize("cache", ["e4m3", "int8"])
def test_nothing_is_written_astray(cache, block, cu):
    """What lies in a row's range may be left out; every other code and scale stays, in K and in V."""
    require_gpu()
    table, n_pages = paged([30, 30, 30], 16, seed=4)
    kc, vc, ks, vs = blocks_cache(n_pages, 16, 2, 64, block, cache, 4)
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn(30, 2, 64, generator=g).bfloat16() for _ in range(2))
    lens = torch.tensor([30, 30, 30], dtype=torch.int32)
    dev = [t.cuda() for t in (kc, vc, ks, vs)]
    gdn.kv_append(k.cuda(), v.cuda(), dev[0], dev[1], table.cuda(), lens.cuda(), k_scale=dev[2], v_scale=dev[3],
                  cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    at = [min(max(i, 0), 30) for i in cu]
    for x, c, s, got in ((k, kc, ks, (dev[0], dev[2])), (v, vc, vs, (dev[1], dev[3]))):
        old, got = (c.float(), s), (got[0].cpu().float(), got[1].cpu())
        may = []
        for b in range(3):
            counts = [max(0, at[b + 1] - at[b]) if i == b else 0 for i in range(3)]
            new = append_ref(c, s, x[at[b]:max(at[b], at[b + 1])], counts, table, lens, cache)
            may.append((new[0].float(), new[1]))
        for i, name in enumerate(("codes", "scales")):
            ok = got[i] == old[i]
            for new in may:
                ok |= got[i] == new[i]
            assert ok.all(), name
            if at == sorted(at):  # ordinary offsets: all of it
                want = old[i]
                for new in may:
                    want = torch.where(new[i] != old[i], new[i], want)
                assert torch.equal(got[i], want), name
