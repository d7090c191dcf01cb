"""References of the calls over block-scaled 8-bit caches and of the rotary
positions: appending block by block, attention and rotation in 64 bits.
Everything on the CPU, shared with no kernel."""
from __future__ import annotations

import math

import torch

from paged_ref import DT, HALF, attn_bound, attn_ref

CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
LIMIT = {"e4m3": 448.0, "int8": 127.0}
TINY = 2.0 ** -126


def blocks_cache(n_pages, page, hkv, d, block, cache, seed, heads_first=False):
    """Random codes and scales, as earlier tokens left them: (k, v, k_scale, v_scale)."""
    g = torch.Generator().manual_seed(seed)
    lim, out = LIMIT[cache], []
    for _ in range(2):
        shape = (n_pages, hkv, page, d) if heads_first else (n_pages, page, hkv, d)
        x = (torch.randn(shape, generator=g) * lim / 3.5).clamp(-lim, lim)
        x = x.round().to(torch.int8) if cache == "int8" else x.to(torch.float8_e4m3fn)
        out.append(x.transpose(1, 2) if heads_first else x)
    for _ in range(2):
        s = (torch.rand(n_pages, hkv, page // block, generator=g) + 0.5) * 3.5 / lim
        out.append(torch.exp2(s.log2().floor()) if cache == "e4m3" else s)
    return out


def values(c, s):
    """What codes [n_pages, page, hkv, d] and scales [n_pages, hkv, blocks] stand for, in 64 bits."""
    block = c.shape[1] // s.shape[2]
    return c.float().double() * s.double().transpose(1, 2).repeat_interleave(block, 1)[..., None]


def need_scale(a, cache):
    """The scale that finite values up to a (a float) need."""
    if cache == "int8":
        return max(float(torch.tensor(a) * (torch.tensor(1.0) / torch.tensor(127.0))), TINY)
    if a == 0:
        return TINY
    m, e = math.frexp(a)  # a = m 2^e, m in [0.5, 1)
    return max(2.0 ** (e - 9 if m <= 0.875 else e - 8), TINY)


def codes(x, s, cache):
    """Quotients x / s (fp32 division) rounded to codes; NaN has no whole code."""
    q = x / s
    if cache == "int8":
        return torch.where(q.isnan(), 0.0, q.clamp(-127, 127).round()).to(torch.int8)
    return q.clamp(-448, 448).to(torch.float8_e4m3fn)


def append_ref(c, s, x, counts, table, lens, cache):
    """Codes and scales after an append of packed tokens x, block by block."""
    c, s = c.clone(), s.clone()
    n_pages, page, hkv, _ = c.shape
    block, cap, start = page // s.shape[2], table.shape[1] * page, 0
    for b, n in enumerate(counts):
        first = int(lens[b]) - n
        p = max(first, 0)
        while p < min(int(lens[b]), cap):
            to = min(int(lens[b]), cap, (p // block + 1) * block)
            e, i = int(table[b, p // page]), p % page
            if 0 <= e < n_pages:
                new = x[start + p - first:start + to - first].float()
                j, edge = i // block, i // block * block
                for h in range(hkv):
                    y = new[:, h]
                    a = float(torch.where(y.isfinite(), y.abs(), 0.0).max())
                    t = need_scale(a, cache)
                    if cache == "int8" and bool(y.isnan().any()):
                        t = float("nan")
                    old = float(s[e, h, j])
                    if i > edge:
                        t = float("nan") if math.isnan(t) or math.isnan(old) else max(t, old)
                        if t != old:
                            v = c[e, edge:i, h].float() * torch.tensor(old)
                            c[e, edge:i, h] = codes(v, torch.tensor(t), cache)
                    s[e, h, j] = t
                    c[e, i:i + to - p, h] = codes(y, torch.tensor(t), cache)
            p = to
        start += n
    return c, s


def read_ref(c, s, counts, table, lens, dtype):
    """The newest counts[b] tokens of each row, packed; zeros where nothing is held."""
    page, out = c.shape[1], []
    v = c.float() if s is None else c.float() * s.transpose(1, 2).repeat_interleave(page // s.shape[2], 1)[..., None]
    for b, n in enumerate(counts):
        for i in range(n):
            p = int(lens[b]) - n + i
            e = int(table[b, p // page]) if 0 <= p < table.shape[1] * page else -1
            out.append(v[e, p % page] if 0 <= e < c.shape[0] else torch.zeros_like(v[0, 0]))
    return torch.stack(out).to(dtype) if out else torch.zeros(0, *c.shape[2:], dtype=dtype)


def attn_blocks_ref(q, kc, vc, ks, vs, table, lens, scale):
    """attn_ref over the values that the codes stand for, in 64 bits."""
    class Exact:  # attn_ref takes a cache's .float().double(): here the values themselves
        def __init__(self, x):
            self.x, self.shape = x, x.shape

        def float(self):
            return self

        def double(self):
            return self.x
    return attn_ref(q, Exact(values(kc, ks)), Exact(values(vc, vs)), table, lens, scale)


def attn_blocks_bound(out, mean, size, lens, d, io):
    """attn_bound, and for block scales one more rounding of each score's factor
    (twice in a weight, see attn_bound) and one of each weight times its value's scale."""
    u = 2.0 ** -24
    return attn_bound(out, mean, size, lens, d, io) + (2 * u * size + u) * mean * (1 + HALF[io])


def rope_ref(x, pos, f, interleaved, factor):
    """x [tokens, heads, d] turned, and the elementwise error bound.

    Angles in fp64 are off by a few 2^-53 of themselves; cut to turns in fp32 by
    2^-26 of a turn (2^-23.3 rad); sine and cosine from the library by at most 4
    units of 2^-24; the factor, two products and their sum by 4 roundings of
    fp32: together under 2^-20.5 of factor (|x1| + |x2|).  Then one rounding."""
    rot, x = 2 * f.shape[0], x.double()
    i = torch.arange(rot // 2)
    i, j = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    a = (pos.double()[:, None] * f.double()).reshape(-1, 1, rot // 2)
    y, size = x.clone(), torch.zeros_like(x)
    y[..., i] = factor * (x[..., i] * a.cos() - x[..., j] * a.sin())
    y[..., j] = factor * (x[..., i] * a.sin() + x[..., j] * a.cos())
    size[..., i] = size[..., j] = abs(factor) * (x[..., i].abs() + x[..., j].abs())
    return y, size


def rope_bound(y, size, pos, f, io):
    """See rope_ref; far angles: 8 roundings of fp64 relative to the largest."""
    far = float(max([abs(int(p)) for p in pos] + [0])) * float(f.abs().max())
    return HALF[io] * y.abs() + (2.0 ** -20.5 + 8 * 2.0 ** -53 * far) * size * (1 + HALF[io]) + 1e-38
