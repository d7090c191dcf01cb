"""Plain 64-bit (attention, appending) and sequential (page tables) references of the
paged-cache calls, and builders of their inputs.  Everything on the CPU."""
from __future__ import annotations

import random

import torch

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
# Half a step of each type, relative to the value.
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def attn_ref(q, kc, vc, table, lens, scale, ks=None, vs=None):
    """out, lse (both exact up to 64 bits) and the elementwise error bound's two
    parts: mean |v| under the weights, and the largest sum |q_i k_i| * scale."""
    B, T, hq, d = q.shape
    n_pages, page, hkv, _ = kc.shape
    group, cap = hq // hkv, table.shape[1] * page
    out = torch.zeros(B, T, hq, d, dtype=torch.float64)
    lse = torch.full((B, T, hq), -float("inf"), dtype=torch.float64)
    mean = torch.zeros(B, T, hq, d, dtype=torch.float64)
    size = torch.zeros(B, T, hq, 1, dtype=torch.float64)
    q, kd, vd = q.double(), kc.float().double(), vc.float().double()
    for b in range(B):
        n = min(max(int(lens[b]), 0), cap)
        held = [(j, int(table[b, j // page])) for j in range(n)]
        held = [(j, e) for j, e in held if 0 <= e < n_pages]
        pos = torch.tensor([j for j, _ in held], dtype=torch.long)
        ent = torch.tensor([e for _, e in held], dtype=torch.long)
        K, V = kd[ent, pos % page], vd[ent, pos % page]  # [n, hkv, d]
        for t in range(T):
            m = pos <= n - T + t
            if not bool(m.any()):
                continue
            for h in range(hq):
                g = h // group
                f = scale * (1.0 if ks is None else float(ks[g]))
                x, v = K[m, g] * q[b, t, h] * f, V[m, g] * (1.0 if vs is None else float(vs[g]))
                s = x.sum(-1)
                top = s.max()
                if top == -float("inf"):
                    continue
                w = torch.exp(s - top)
                out[b, t, h] = (w[:, None] * v).sum(0) / w.sum()
                lse[b, t, h] = top + torch.log(w.sum())
                mean[b, t, h] = (w[:, None] * v.abs()).sum(0) / w.sum()
                size[b, t, h] = x.abs().sum(-1).max()
    return out, lse, mean, size


def attn_bound(out, mean, size, lens, d, io):
    """Largest |got - out| that rounding explains, u = 2^-24 a rounding of fp32:
      * scores: d products (rounded, exact for bf16) summed in fp32, scaled and
        shifted: at most (d + 6) u sum|q_i k_i| scale off; a weight is off by
        that twice (numerator and its share of the sum), plus the hardware
        exp2's few u (8 u allowed);
      * sums over n keys, their rescaling and joining: n + 64 roundings;
      * bf16 weights as two bf16 terms: half a step of a half step, 2^-16;
      * the output's one rounding.
    All but the last are relative to the weighted mean of |v|."""
    u = 2.0 ** -24
    n = max([int(x) for x in lens] + [1])
    rel = 2 * ((d + 6) * u * size + 8 * u) + (n + 64) * u + (2.0 ** -16 if io == "bf16" else 0.0)
    return HALF[io] * out.abs() + rel * mean * (1 + HALF[io]) + 1e-30


def paged(lens, page, width=None, spare=3, seed=0, share=None):
    """A page table over shuffled pages (unused entries -1) and the page count."""
    r = random.Random(seed)
    need = [-(-max(int(n), 0) // page) for n in lens]
    n_pages = sum(need) + spare
    order = list(range(n_pages))
    r.shuffle(order)
    table = torch.full((len(lens), width or max(need + [1])), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    return table, n_pages


def caches(n_pages, page, hkv, d, cache, seed, fill=None, heads_first=False):
    """Random key and value caches; fill: the value of every element first
    (for slots that no row holds), then rows are written by the caller."""
    g = torch.Generator().manual_seed(seed)
    shape = (n_pages, hkv, page, d) if heads_first else (n_pages, page, hkv, d)

    def one():
        x = torch.randn(shape, generator=g)
        if cache == "e4m3":
            x = (x * 60).clamp(-448, 448)
        x = x.to(DT[cache])
        return x.transpose(1, 2) if heads_first else x
    return one(), one()


def poison_unheld(c, table, lens, page, value):
    """A copy of cache c whose slots that no row holds are `value`."""
    held = torch.zeros(c.shape[:2], dtype=torch.bool)
    for b in range(table.shape[0]):
        for j in range(min(max(int(lens[b]), 0), table.shape[1] * page)):
            e = int(table[b, j // page])
            if 0 <= e < c.shape[0]:
                held[e, j % page] = True
    w = c.float().clone()
    w[~held] = value
    return w.to(c.dtype)


# ------------------------------------------------------------ page tables --


def used(n, page):
    return -(-n // page)


def _len(lens, r, table, page):
    return min(max(int(lens[r]), 0), len(table[0]) * page)


def extend_ref(table, lens, refs, add, page):
    table, refs = [list(r) for r in table.tolist()], refs.tolist()
    rows, width = len(table), len(table[0])
    free = [p for p, n in enumerate(refs) if n == 0]
    lens_out, ok, upto, at = [], [], 0, 0
    for r in range(rows):
        n = _len(lens, r, table, page)
        grown = n + max(int(add[r]), 0)
        have = used(n, page)
        if grown > width * page:
            lens_out.append(n), ok.append(0)
            continue
        need = used(grown, page) - have
        upto += need
        if need and upto > len(free):
            lens_out.append(n), ok.append(0)
            continue
        for i in range(need):
            p = free[upto - need + i]
            table[r][have + i], refs[p] = p, 1
        lens_out.append(grown), ok.append(1)
    return table, lens_out, refs, ok


def fork_ref(table, lens, refs, parent, page):
    old, refs = [list(r) for r in table.tolist()], refs.tolist()
    rows, width, n_pages = len(old), len(old[0]), len(refs)
    valid = lambda e: 0 <= e < n_pages
    new, lens_out = [], []
    for r in range(rows):
        p = int(parent[r])
        n = _len(lens, p, old, page) if 0 <= p < rows else 0
        new.append([old[p][i] if i < used(n, page) else -1 for i in range(width)] if n else [-1] * width)
        lens_out.append(n)
    for r in range(rows):
        for e in old[r][:used(_len(lens, r, old, page), page)]:
            if valid(e):
                refs[e] -= 1
        for e in new[r][:used(lens_out[r], page)]:
            if valid(e):
                refs[e] += 1
    holders = {}
    for r in range(rows):
        if lens_out[r] % page:
            holders.setdefault(new[r][lens_out[r] // page], []).append(r)
    need = []
    for r in range(rows):
        if lens_out[r] % page:
            e = new[r][lens_out[r] // page]
            if valid(e) and not (holders[e][0] == r and len(holders[e]) == refs[e]):
                need.append(r)
    free = [p for p, n in enumerate(refs) if n == 0]
    src, dst = [-1] * rows, [-1] * rows
    for k, r in enumerate(need):
        if k < len(free):
            i = lens_out[r] // page
            src[r], dst[r] = new[r][i], free[k]
            new[r][i] = free[k]
            refs[src[r]] -= 1
            refs[dst[r]] = 1
        else:
            for e in new[r]:
                if valid(e):
                    refs[e] -= 1
            new[r], lens_out[r] = [-1] * width, 0
    return new, lens_out, refs, src, dst


def free_ref(table, lens, refs, mask, page):
    table, refs = [list(r) for r in table.tolist()], refs.tolist()
    lens_out = []
    for r in range(len(table)):
        n = _len(lens, r, table, page)
        if bool(mask[r]):
            for e in table[r][:used(n, page)]:
                if 0 <= e < len(refs):
                    refs[e] -= 1
            table[r], n = [-1] * len(table[r]), 0
        lens_out.append(n)
    return table, lens_out, refs


def compact_ref(table, refs):
    table, refs = [list(r) for r in table.tolist()], refs.tolist()
    n = len(refs)
    live = sum(x > 0 for x in refs)
    holes = [p for p in range(live) if refs[p] <= 0]
    tails = [p for p in range(live, n) if refs[p] > 0]
    to = dict(zip(tails, holes))
    out = [refs[p] if p < live else 0 for p in range(n)]
    for t, h in to.items():
        out[h] = refs[t]
    pad = [-1] * (n // 2 - len(tails))
    return [[to.get(e, e) for e in row] for row in table], out, tails + pad, holes + pad, [live]


def random_state(rows, width, page, n_pages, seed, shared=0, fill=0.8):
    """A consistent (table, lens, refs): rows of random lengths over scattered
    pages, some sharing their first `shared` pages."""
    r = random.Random(seed)
    order = list(range(n_pages))
    r.shuffle(order)
    joint, at = order[:shared], shared
    table, lens, refs = [], [], [0] * n_pages
    for _ in range(rows):
        n = r.choice([0, 1, page, width * page, r.randint(0, width * page)]) if r.random() < fill else 0
        u = used(n, page)
        mine = joint if n >= shared * page else []
        if at + u - len(mine) > n_pages:
            n, u, mine = 0, 0, []
        row = mine + order[at:at + u - len(mine)]
        at += u - len(mine)
        for e in row:
            refs[e] += 1
        table.append(row + [-1] * (width - u))
        lens.append(n)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)
    return i32(table).reshape(rows, width), i32(lens), i32(refs)
