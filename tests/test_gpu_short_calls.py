"""The short way into libgdn (binding/calls.cpp): the same bits as the general
way on everything that it takes, and nothing launched for what it does not take."""
import pytest
import torch

import gated_deltanet_state_delta_amd as gdn
from blocks_ref import blocks_cache
from gated_deltanet_state_delta_amd.paged import _short
from gpu_util import require_gpu
from paged_ref import DT, caches, paged

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _state(cache, page, hkv, d, heads_first=False):
    lens = torch.tensor([40, 3, 0, 100], dtype=I32)
    table, n_pages = paged(lens, page, seed=1)
    if cache in ("bf16", "f32"):
        kc, vc = caches(n_pages, page, hkv, d, cache, 1, heads_first=heads_first)
        scales = (None, None)
    else:
        kc, vc, *scales = blocks_cache(n_pages, page, hkv, d, page, cache[:4], 1, heads_first)
        if cache == "e4m3 heads":
            scales = (torch.rand(hkv) + 0.1, torch.rand(hkv) + 0.1)
    dev = lambda c: c.transpose(1, 2).contiguous().cuda().transpose(1, 2) if heads_first else c.cuda()
    return [dev(kc), dev(vc), table.cuda(), lens.cuda()], [None if s is None else s.cuda() for s in scales]


CASES = [("bf16", "bf16"), ("f32", "f32"), ("bf16", "e4m3"), ("f32", "int8"), ("bf16", "e4m3 heads"), ("bf16", "int8")]


@pytest.mark.parametrize("page,hkv,d,heads_first", [(16, 2, 64, False), (5, 1, 128, False), (16, 3, 32, True), (1, 1, 256, False)])
@pytest.mark.parametrize("io,cache", CASES)
def test_both_ways_give_the_same_bits(io, cache, page, hkv, d, heads_first):
    g = torch.Generator(device="cuda").manual_seed(1)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda").to(DT[io])
    (kc, vc, table, lens), (ks, vs) = _state(cache, page, hkv, d, heads_first)
    here = torch.cuda.current_stream()
    kw = dict(k_scale=ks, v_scale=vs)
    q = draw(4, 2, 3 * hkv, d)
    assert _short("attn_decode", q, kc, vc, table, lens, None, ks, vs) is not None
    for scale in (None, 0.3):
        assert torch.equal(gdn.attn_decode(q, kc, vc, table, lens, scale=scale, **kw),
                           gdn.attn_decode(q, kc, vc, table, lens, scale=scale, stream=here, **kw))
    cu = torch.tensor([0, 20, 21, 21, 60], dtype=I32).cuda()
    assert _short("kv_read", kc, vc, table, lens, 3, None, 1 if io == "bf16" else 0, ks, vs) is not None
    for tokens, offsets in ((3, None), (70, cu)):
        a = gdn.kv_read(kc, vc, table, lens, tokens, cu_seqlens=offsets, dtype=DT[io], **kw)
        b = gdn.kv_read(kc, vc, table, lens, tokens, cu_seqlens=offsets, dtype=DT[io], stream=here, **kw)
        assert all(x.shape == y.shape and x.dtype == y.dtype and torch.equal(x, y) for x, y in zip(a, b))
    fused = draw(60, 3 * hkv, d)
    new = [(fused[:, :hkv], fused[:, 2 * hkv:], cu), (draw(60, hkv, d), draw(60, hkv, d), cu),
           (draw(4, 1, hkv, d), draw(3, 4, hkv, d)[1][:, None], None), (draw(4, 5, hkv, d), draw(4, 5, hkv, d), None)]
    for k, v, offsets in new:
        got = []
        for way in (None, here):
            c = [t.clone() for t in (kc, vc)]
            s = [None if t is None else t.clone() for t in (ks, vs)]
            out = gdn.kv_append(k, v, *c, table, lens, cu_seqlens=offsets, k_scale=s[0], v_scale=s[1], stream=way)
            assert out[0] is c[0] and out[1] is c[1]
            got.append([t.float() for t in c + s if t is not None])
        assert all(torch.equal(x, y) for x, y in zip(*got))
        c = [t.clone() for t in (kc, vc)]
        assert _short("kv_append", k, v, *c, table, lens, offsets, ks, vs) is True
    f = gdn.rope_frequencies(d)[0].cuda()
    for x, y, where in ((q, draw(4, 2, hkv, d), dict(lens=lens)), (fused[:, hkv:], fused[:, :hkv], dict(lens=lens, cu_seqlens=cu)),
                        (q, None, dict(positions=torch.arange(8).view(4, 2).cuda())),
                        (fused, fused[:, 1:], dict(positions=torch.arange(60, dtype=I32).cuda()))):
        for turned in (dict(), dict(interleaved=True, factor=0.7)):
            a, b = gdn.rope(x, y, f, **where, **turned), gdn.rope(x, y, f, stream=here, **where, **turned)
            assert torch.equal(a[0], b[0]) and (y is None and a[1] is None or torch.equal(a[1], b[1]))
        assert _short("rope", x, y, f, where.get("lens"), where.get("cu_seqlens"), where.get("positions"), False, 1.0) is not None


def test_what_it_does_not_take_it_leaves_to_the_general_way():
    (kc, vc, table, lens), (ks, vs) = _state("int8", 16, 2, 64)
    q, k = torch.randn(4, 1, 4, 64).bfloat16().cuda(), torch.randn(4, 1, 2, 64).bfloat16().cuda()
    args = dict(q=q, kc=kc, vc=vc, table=table, lens=lens, scale=None, ks=ks, vs=vs)
    cut = torch.zeros(4, 5, 4, 64, dtype=torch.bfloat16).cuda()[:, :3]
    for over in (dict(q=q.half()), dict(q=q[0]), dict(q=cut), dict(q=q.cpu()), dict(kc=kc.cpu()), dict(vc=vc[:-1]), dict(vc=vc.float()),
                 dict(table=table.long()), dict(table=table[:3]), dict(table=table.t().contiguous().t()), dict(lens=lens.long()),
                 dict(lens=lens[:3]), dict(ks=None), dict(ks=ks.double(), vs=vs.double()), dict(ks=ks[:-1], vs=vs[:-1]),
                 dict(ks=ks.cpu(), vs=vs.cpu()), dict(ks=torch.ones(2).cuda(), vs=torch.ones(2).cuda()), dict(ks=3, vs=3),
                 dict(kc=kc.float(), vc=vc.float()), dict(scale="x"), dict(q=q[..., :48].contiguous()), dict(q=torch.zeros(4, 65, 4, 64).bfloat16().cuda())):
        assert _short("attn_decode", *dict(args, **over).values()) is None, over.keys()
    args = dict(k=k, v=k, kc=kc, vc=vc, table=table, lens=lens, cu=None, ks=ks, vs=vs)
    before = [t.clone() for t in (kc, vc, ks, vs)]
    odd = torch.zeros(4, 1, 2, 68, dtype=torch.bfloat16).cuda()[..., 3:67]
    for over in (dict(k=odd, v=odd), dict(v=k.float()), dict(v=k[:3]), dict(k=k[:3], v=k[:3]), dict(cu=torch.zeros(5, dtype=I32).cuda()),
                 dict(k=k[:, 0], v=k[:, 0]), dict(k=k[:, 0], v=k[:, 0], cu=torch.zeros(5).long().cuda()),
                 dict(k=k[:, 0], v=k[:, 0], cu=torch.zeros(4, dtype=I32).cuda()), dict(lens=lens[:, None]), dict(kc=kc[0], vc=vc[0]), dict(ks=vs.transpose(1, 2))):
        assert _short("kv_append", *dict(args, **over).values()) is None, over.keys()
    assert all(torch.equal(a, b) for a, b in zip(before, (kc, vc, ks, vs)))
    args = dict(kc=kc, vc=vc, table=table, lens=lens, tokens=3, cu=None, io=1, ks=ks, vs=vs)
    for over in (dict(tokens=-1), dict(tokens=1.0), dict(tokens=1 << 40), dict(tokens=1 << 28), dict(io=-1), dict(io=2), dict(lens=lens.long()),
                 dict(cu=torch.zeros(4, dtype=I32).cuda())):
        assert _short("kv_read", *dict(args, **over).values()) is None, over.keys()
    f, at = gdn.rope_frequencies(64)[0].cuda(), torch.zeros(4, 1, dtype=I32).cuda()
    args = dict(q=q, k=k, f=f, lens=lens, cu=None, pos=None, interleaved=False, factor=1.0)
    for over in (dict(q=q.half()), dict(k=k.float()), dict(k=k[:3]), dict(k=k[..., :32]), dict(f=f.float()), dict(f=f.cpu()), dict(f=f[:0]),
                 dict(f=torch.ones(33).double().cuda()), dict(lens=None), dict(pos=at), dict(lens=None, pos=at[:3]), dict(lens=None, pos=at.float()),
                 dict(lens=lens.long()), dict(cu=torch.zeros(5, dtype=I32).cuda()), dict(q=cut), dict(factor="x"), dict(q=q[0, 0], k=k[0, 0])):
        assert _short("rope", *dict(args, **over).values()) is None, over.keys()
    # and the public call on what the general way converts
    assert torch.equal(gdn.attn_decode(q, kc, vc, table.long(), lens.long(), k_scale=ks, v_scale=vs),
                       gdn.attn_decode(q, kc, vc, table, lens, k_scale=ks, v_scale=vs))
    assert torch.equal(gdn.rope(cut, None, f, lens=lens.long())[0], gdn.rope(cut.contiguous(), None, f, lens=lens)[0])
    for bad in (lambda: gdn.attn_decode(q.half(), kc, vc, table, lens, k_scale=ks, v_scale=vs), lambda: gdn.rope(q, k, f, lens=lens[:3]),
                lambda: gdn.kv_append(k, k[:3], kc, vc, table, lens, k_scale=ks, v_scale=vs),
                lambda: gdn.kv_read(kc, vc, table, lens, 1, dtype=torch.float16, k_scale=ks, v_scale=vs),
                lambda: gdn.attn_decode(q, kc.cpu(), vc, table, lens, k_scale=ks, v_scale=vs)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(gdn.GdnError):
        gdn.attn_decode(torch.zeros(4, 65, 4, 64).bfloat16().cuda(), kc, vc, table, lens, k_scale=ks, v_scale=vs)
    with pytest.raises(TypeError):
        _short("rope", q, k)


def test_workspaces_belong_to_the_current_stream():
    """Two streams, one after the other current, at once."""
    (kc, vc, table, lens), (ks, vs) = _state("int8", 16, 2, 128)
    table = table.repeat(1, 3)
    q = [torch.randn(4, 1, 8, 128).bfloat16().cuda() for _ in range(2)]
    want = [gdn.attn_decode(x, kc, vc, table, lens, k_scale=ks, v_scale=vs) for x in q]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(40):
        with torch.cuda.stream(streams[i % 2]):
            got.append(gdn.attn_decode(q[i % 2], kc, vc, table, lens, k_scale=ks, v_scale=vs))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i % 2]) for i, y in enumerate(got))
