"""The paged key-value cache operators, as cases to measure: attention of a batch's newest
tokens over the cache (gdn.attn_decode), writing new tokens into their pages (gdn.kv_append)
and managing pages (gdn.pages_copy, pages_extend, pages_fork, pages_free, pages_compact).

run() computes a case in plain torch operations, or, with `own` set, through the package's
calls; exact() gives the same values from the definitions in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

IO = {"bf16": torch.bfloat16, "f32": torch.float32}
CACHE = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f32": 4, "e4m3": 1}


def _attn(name, rows, new, hq, hkv, d, page, max_len, lens, io, cache, heads_first):
    return {"name": name, "op": "attn", "rows": rows, "new": new, "hq": hq, "hkv": hkv, "d": d, "page": page,
            "max_len": max_len, "lens": lens, "io": io, "cache": cache, "heads_first": heads_first}


def _append(name, rows, tokens, hkv, d, page, max_len, io, cache, packed):
    return {"name": name, "op": "append", "rows": rows, "tokens": tokens, "hkv": hkv, "d": d, "page": page,
            "max_len": max_len, "io": io, "cache": cache, "packed": packed}


def _pages(name, op, rows, max_pages, page, n_pages, shared):
    return {"name": name, "op": op, "rows": rows, "max_pages": max_pages, "page": page, "n_pages": n_pages,
            "shared": shared}


def listed():
    return [
        # one conversation of a few hundred tokens: a single row, where latency counts
        _attn("attn one short row", 1, 1, 32, 8, 128, 16, 777, "full", "bf16", "bf16", False),
        # an ordinary serving batch, ragged, 4 query heads on each key-value head
        _attn("attn ragged batch", 64, 1, 32, 8, 128, 16, 8192, "ragged", "bf16", "bf16", False),
        # a few long documents: the split over the length has to fill the card
        _attn("attn long documents", 4, 1, 32, 4, 128, 64, 131072, "full", "bf16", "bf16", True),
        # a large batch over an 8-bit cache with wide heads and 8 query heads on each
        _attn("attn 8-bit cache", 256, 1, 16, 2, 256, 32, 4096, "ragged", "bf16", "e4m3", False),
        # verification of 4 proposed tokens a row, fp32, pages that no tile divides
        _attn("attn verify fp32", 32, 4, 16, 16, 64, 5, 2000, "ragged", "f32", "f32", False),
        # the newest token of each row of a decode batch
        _append("append one token each", 256, 256, 8, 128, 16, 4096, "bf16", "bf16", False),
        # prompts of uneven lengths written into an 8-bit cache
        _append("append prompts 8-bit", 8, 32768, 8, 128, 16, 8192, "bf16", "e4m3", True),
        # part-filled pages of a forked batch: 32 KiB each
        {"name": "copy cache pages", "op": "copy", "n": 2048, "bytes": 32768, "pairs": 64, "io": "bf16"},
        # recurrent states of forked requests: 32 heads of 128 x 128 fp32, 2 MiB a slot
        {"name": "copy state slots", "op": "copy", "n": 1024, "bytes": 2097152, "pairs": 256, "io": "f32"},
        # beams reordered: kept, forked and dropped rows that share a prompt's pages
        _pages("fork beams", "fork", 256, 512, 16, 65536, 32),
        # every row of a batch grows by some tokens
        _pages("extend batch", "extend", 1024, 256, 16, 262144, 0),
        # a fragmented cache is packed into its lowest pages
        _pages("compact cache", "compact", 1024, 512, 16, 393216, 8),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "copy", "fork", "extend", "free", "compact"])
    if op == "attn":
        cache = rng.choice(["bf16", "bf16", "f32", "e4m3"])
        io = "f32" if cache == "f32" else rng.choice(["bf16", "bf16", "f32"]) if cache == "e4m3" else "bf16"
        d, hkv, group = rng.choice([32, 64, 128, 256]), rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 6, 8, 16])
        max_len, new = _spread(rng, 1, 65536), rng.choice([1, 1, 1, 2, 4, 7])
        # at most the values that the largest listed cases hold
        rows = _spread(rng, 1, max(1, min(256, 200_000_000 // (max_len * hkv * d * group))))
        c = _attn("", rows, new, hkv * group, hkv, d, rng.choice([1, 3, 16, 16, 32, 64, 100, 256]), max_len,
                  rng.choice(["ragged", "full"]), io, cache, rng.random() < 0.5)
    elif op == "append":
        cache = rng.choice(["bf16", "f32", "e4m3"])
        rows, packed = _spread(rng, 1, 256), rng.random() < 0.5
        tokens = _spread(rng, rows, 16384) if packed else rows * rng.choice([1, 1, 2, 5])
        c = _append("", rows, tokens, rng.choice([1, 2, 4, 8]), rng.choice([32, 64, 128, 256]),
                    rng.choice([1, 5, 16, 64, 128]), 4096 if rows <= 64 else 1024,
                    "f32" if cache == "f32" else rng.choice(["bf16", "f32"]) if cache == "e4m3" else "bf16",
                    cache, packed)
    elif op == "copy":
        io = rng.choice(["bf16", "f32"])
        size = _spread(rng, 64, 1 << 21) // BYTES[io] * BYTES[io]
        n = _spread(rng, 8, max(8, min(8192, (1 << 30) // size)))
        c = {"op": "copy", "n": n, "bytes": size, "pairs": _spread(rng, 1, n // 2), "io": io}
    else:
        rows, max_pages = _spread(rng, 1, 1024), _spread(rng, 1, 512)
        c = _pages("", op, rows, max_pages, rng.choice([1, 5, 16, 64]),
                   rows * max_pages // rng.choice([1, 2, 2]) + rng.randrange(1, 4096), rng.choice([0, 0, 1, 7]))
    c.pop("name", None)
    return c


# ------------------------------------------------------------------ inputs --


def _lens(case):
    """The tokens of each row that the cache holds: a matter of the case alone, as its work is."""
    if case["lens"] == "full":
        return [case["max_len"]] * case["rows"]
    r = random.Random(case["rows"] * 1_000_003 + case["max_len"])
    return [r.randint(0, case["max_len"]) for _ in range(case["rows"] - 1)] + [case["max_len"]]


def _counts(case):
    """The new tokens of each row of an append."""
    if not case["packed"]:
        return [case["tokens"] // case["rows"]] * case["rows"]
    r = random.Random(case["rows"] * 1_000_003 + case["tokens"])
    cut = sorted(r.randint(0, case["tokens"]) for _ in range(case["rows"] - 1))
    n = [b - a for a, b in zip([0] + cut, cut + [case["tokens"]])]
    return [min(x, case["max_len"]) for x in n]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _table(lens, width, page, seed):
    """A page table over shuffled pages, unused entries -1, and the number of pages."""
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + sum(need) // 16 + 2
    order = np.random.RandomState(seed % (1 << 31)).permutation(n_pages).astype(np.int32)
    table, at = np.full((len(lens), max(1, width)), -1, np.int32), 0
    for b, n in enumerate(need):
        table[b, :n], at = order[at:at + n], at + n
    return torch.from_numpy(table).cuda(), n_pages


def _cache(case, n_pages, g):
    """An allocated cache with earlier tokens in it, as [n_pages, page, hkv, d]."""
    shape = (n_pages, case["page"], case["hkv"], case["d"])
    if case.get("heads_first"):
        shape = (n_pages, case["hkv"], case["page"], case["d"])
    if case["cache"] == "e4m3":
        c = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(100)
        c = c.clamp_(-448, 448).to(torch.float8_e4m3fn)
    else:
        c = torch.randn(shape, generator=g, device="cuda", dtype=CACHE[case["cache"]])
    return c.transpose(1, 2) if case.get("heads_first") else c


def _scales(case, g):
    """One factor a key-value head for an 8-bit cache: about the largest value over 448."""
    if case["cache"] != "e4m3":
        return None, None
    return tuple(torch.rand(case["hkv"], generator=g, device="cuda") * 0.01 + 0.005 for _ in range(2))


def _prepare_pages(case, seed):
    """Rows of part-filled tables over a cache whose free pages lie scattered, with counts of holders."""
    r = np.random.RandomState(seed % (1 << 31))
    rows, width, page, n = case["rows"], case["max_pages"], case["page"], case["n_pages"]
    lens = r.randint(0, width * page + 1, rows)
    if case["op"] == "extend":  # room to grow in most rows
        lens = lens * 3 // 4
    shared = min(case["shared"], width, n)
    order, at = r.permutation(n).astype(np.int32), shared
    table, refs = np.full((rows, width), -1, np.int32), np.zeros(n, np.int32)
    for b in range(rows):
        used = -(-int(lens[b]) // page)
        joint = min(shared, used) if lens[b] >= shared * page else 0
        if at + used - joint > n:  # the cache is full: an idle row
            lens[b] = used = joint = 0
        table[b, :joint] = order[:joint]
        table[b, joint:used], at = order[at:at + used - joint], at + used - joint
        refs[table[b, :used]] += 1
    s = {"table": table, "lens": lens.astype(np.int32), "refs": refs}
    if case["op"] == "extend":
        s["add"] = r.choice([1, 1, 1, 4, 4 * page], rows).astype(np.int32)
    elif case["op"] == "fork":
        kind, other = r.rand(rows), r.randint(0, rows, rows)
        s["parent"] = np.where(kind < 0.5, np.arange(rows), np.where(kind < 0.9, other, -1)).astype(np.int32)
    elif case["op"] == "free":
        s["mask"] = r.rand(rows) < 0.4
    return {k: torch.from_numpy(v).cuda() for k, v in s.items()}


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op == "attn":
        lens, page = _lens(case), case["page"]
        s["table"], n_pages = _table(lens, -(-case["max_len"] // page), page, seed)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["k"], s["v"] = _cache(case, n_pages, g), _cache(case, n_pages, g)
        s["ks"], s["vs"] = _scales(case, g)
        s["q"] = torch.randn(case["rows"], case["new"], case["hq"], case["d"], generator=g, device="cuda",
                             dtype=IO[case["io"]])
    elif op == "append":
        counts, page = _counts(case), case["page"]
        r = random.Random(case["tokens"])
        lens = [n + r.randint(0, case["max_len"] - n) for n in counts]
        s["table"], n_pages = _table(lens, -(-case["max_len"] // page), page, seed)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["k"], s["v"] = _cache(case, n_pages, g), _cache(case, n_pages, g)
        s["ks"], s["vs"] = _scales(case, g)
        shape = (sum(counts),) if case["packed"] else (case["rows"], counts[0])
        s["new_k"], s["new_v"] = (torch.randn(*shape, case["hkv"], case["d"], generator=g, device="cuda",
                                              dtype=IO[case["io"]]) for _ in range(2))
        s["cu"] = None
        if case["packed"]:
            s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    elif op == "copy":
        s["pool"] = torch.randn(case["n"], case["bytes"] // BYTES[case["io"]], generator=g, device="cuda",
                                dtype=IO[case["io"]])
        p = np.random.RandomState(seed % (1 << 31)).permutation(case["n"]).astype(np.int32)
        s["src"], s["dst"] = (torch.from_numpy(p[k * case["pairs"]:(k + 1) * case["pairs"]].copy()).cuda()
                              for k in range(2))
    else:
        s.update(_prepare_pages(case, seed))
    return s


# ------------------------------------------------------------- plain forms --


def _plain_attn(s):
    """Scores over every position that a row's table covers, masked to those that its tokens see."""
    q, k, v, table, lens = s["q"], s["k"], s["v"], s["table"].long(), s["lens"].long()
    rows, new, hq, d = q.shape
    n_pages, page, hkv, _ = k.shape
    at = torch.arange(table.shape[1] * page, device=q.device)
    entry = table[:, at // page]
    held = (entry >= 0) & (entry < n_pages)
    entry = entry.clamp(0, n_pages - 1)
    kk, vv = (_values(c, entry, at % page).permute(0, 2, 1, 3) for c in (k, v))  # rows, hkv, length, d
    last = lens[:, None] - new + torch.arange(new, device=q.device)  # each new token's own position
    sees = (at <= last[..., None]) & held[:, None]  # rows, new, length
    kk = torch.where((at < lens[:, None])[:, None, :, None], kk, 0.0)
    vv = torch.where((at < lens[:, None])[:, None, :, None], vv, 0.0)
    qq = q.float().reshape(rows, new, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(rows, hkv, -1, d)
    score = torch.matmul(qq, kk.transpose(2, 3).contiguous()).reshape(rows, hkv, new, hq // hkv, -1) / math.sqrt(d)
    if s["ks"] is not None:
        score = score * s["ks"][None, :, None, None, None]
    score = torch.where(sees[:, None, :, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = weight.sum(-1, keepdim=True)
    out = torch.matmul(weight.reshape(rows, hkv, -1, weight.shape[-1]), vv).reshape(rows, hkv, new, -1, d)
    out = torch.where(total > 0, out / total, 0.0)
    if s["vs"] is not None:
        out = out * s["vs"][None, :, None, None, None]
    return out.permute(0, 2, 1, 3, 4).reshape(rows, new, hq, d).to(q.dtype)


def _values(cache, entry, slot):
    """A cache's rows at (entry, slot), in 32 bits."""
    if cache.dtype == torch.float8_e4m3fn:
        return cache.view(torch.uint8)[entry, slot].view(torch.float8_e4m3fn).float()
    return cache[entry, slot].float()


def _places(s):
    """For each new token its row and its position in it; tokens before a row's start have none."""
    lens = s["lens"].long()
    if s["cu"] is None:
        rows, new = s["new_k"].shape[:2]
        row = torch.arange(rows, device=lens.device).repeat_interleave(new)
        at = (lens[:, None] - new + torch.arange(new, device=lens.device)).reshape(-1)
    else:
        cu, i = s["cu"].long(), torch.arange(s["new_k"].shape[0], device=lens.device)
        row = torch.searchsorted(cu, i, right=True) - 1
        at = lens[row] - cu[row + 1] + i
    return row, at


def _plain_append(s):
    row, at = _places(s)
    page = s["k"].shape[1]
    entry = s["table"].long()[row, at // page]
    for x, cache, scale in ((s["new_k"], s["k"], s["ks"]), (s["new_v"], s["v"], s["vs"])):
        x = x.reshape(-1, *x.shape[-2:])
        if scale is None:
            cache[entry, at % page] = x.to(cache.dtype)
        else:
            x = (x.float() / scale[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
            cache.view(torch.uint8)[entry, at % page] = x.view(torch.uint8)
    return s["k"], s["v"]


def _used(lens, page, width):
    """The mask of each row's table entries that hold its tokens."""
    need = (lens.long() + page - 1) // page
    return torch.arange(width, device=lens.device) < need[:, None]


def _free_list(refs):
    """The free pages, lowest first, in the front of a list of all pages' length, and how many there are."""
    free = refs == 0
    at, n_free = torch.arange(refs.numel(), device=refs.device), free.sum()
    rank = torch.where(free, free.cumsum(0) - 1, n_free + (~free).cumsum(0) - 1)
    return torch.empty_like(at).scatter_(0, rank, at), n_free


def _count(refs, table, mask, by):
    """refs with `by` added for each masked table entry (the others add zero, each at a place of its own)."""
    apart = torch.arange(table.numel(), device=table.device).reshape(table.shape) % refs.numel()
    return refs.scatter_add(0, torch.where(mask, table, apart).reshape(-1), (mask * by).reshape(-1).to(refs.dtype))


def _plain_extend(s):
    table, lens, refs, page = s["table"].long(), s["lens"].long(), s["refs"].long(), s["case"]["page"]
    grown = lens + s["add"].long()
    fits = grown <= table.shape[1] * page
    have = (lens + page - 1) // page
    need = torch.where(fits, (grown + page - 1) // page - have, 0)
    upto = need.cumsum(0)
    pages, n_free = _free_list(refs)
    ok = fits & ((need == 0) | (upto <= n_free))
    i = torch.arange(table.shape[1], device=table.device) - have[:, None]
    new = (i >= 0) & (i < need[:, None]) & ok[:, None]
    table = torch.where(new, pages[((upto - need)[:, None] + i).clamp(0, refs.numel() - 1)], table)
    refs = _count(refs, table, new, 1)
    return table.int(), torch.where(ok, grown, lens).int(), refs.int(), ok.int()


def _plain_fork(s):
    table, lens, refs, page = s["table"].long(), s["lens"].long(), s["refs"].long(), s["case"]["page"]
    rows, width = table.shape
    n, parent = refs.numel(), s["parent"].long()
    kept = (parent >= 0) & (parent < rows)
    row = torch.arange(rows, device=table.device)
    refs = _count(refs, table, _used(lens, page, width), -1)
    lens = torch.where(kept, lens[parent.clamp(0, rows - 1)], 0)
    used = _used(lens, page, width)
    table = torch.where(used, table[parent.clamp(0, rows - 1)], -1)
    refs = _count(refs, table, used, 1)
    # the part-filled last pages: the lowest row keeps one that nobody holds otherwise, the others copy it
    part = lens % page != 0
    end = (lens // page).clamp(max=width - 1)
    last = torch.where(part, table.gather(1, end[:, None])[:, 0], n)
    owner = torch.full((n + 1,), rows, device=table.device).scatter_reduce_(0, last, row, "amin")
    holders = torch.zeros(n + 1, dtype=torch.long, device=table.device).scatter_add_(0, last, part.long())
    at = last.clamp(max=n - 1)
    copies = part & ((owner[last] != row) | (holders[last] != refs[at]))
    pages, n_free = _free_list(refs)
    rank = copies.cumsum(0) - 1
    served = copies & (rank < n_free)
    fresh = pages[rank.clamp(0, n - 1)]
    refs = refs.scatter_add(0, at, -served.long()).scatter_add(0, fresh, served.long())
    table = table.scatter(1, end[:, None], torch.where(served, fresh, table.gather(1, end[:, None])[:, 0])[:, None])
    failed = copies & ~served
    refs = _count(refs, table, used & failed[:, None], -1)
    table, lens = torch.where(failed[:, None], -1, table), torch.where(failed, 0, lens)
    return (table.int(), lens.int(), refs.int(), torch.where(served, at, -1).int(),
            torch.where(served, fresh, -1).int())


def _plain_free(s):
    table, lens, refs = s["table"].long(), s["lens"].long(), s["refs"].long()
    out = s["mask"][:, None] & _used(lens, s["case"]["page"], table.shape[1])
    refs = _count(refs, table, out, -1)
    return torch.where(s["mask"][:, None], -1, table).int(), torch.where(s["mask"], 0, lens).int(), refs.int()


def _plain_compact(s):
    table, refs = s["table"].long(), s["refs"].long()
    n = refs.numel()
    live, at = refs > 0, torch.arange(n, device=refs.device)
    n_live = live.sum()
    hole, tail = ~live & (at < n_live), live & (at >= n_live)
    holes, tails = (torch.full((n + 1,), -1, dtype=torch.long, device=refs.device)
                    .scatter_(0, torch.where(m, m.cumsum(0) - 1, n), torch.where(m, at, -1)) for m in (hole, tail))
    to = torch.where(tail, holes[torch.where(tail, tail.cumsum(0) - 1, 0)], at)
    held = (table >= 0) & (table < n)
    table = torch.where(held, to[table.clamp(0, n - 1)], table)
    packed = torch.zeros(n, dtype=torch.long, device=refs.device).scatter_add_(0, to, refs)
    return table.int(), packed.int(), tails[:n // 2].int(), holes[:n // 2].int(), n_live.reshape(1).int()


def _plain(s):
    op = s["case"]["op"]
    if op == "copy":
        s["pool"][s["dst"].long()] = s["pool"][s["src"].long()]
        return s["pool"]
    return {"attn": _plain_attn, "append": _plain_append, "extend": _plain_extend, "fork": _plain_fork,
            "free": _plain_free, "compact": _plain_compact}[op](s)


# --------------------------------------------------------------------- run --


def run(state):
    if not own:
        return _plain(state)
    import gated_deltanet_state_delta_amd as gdn
    s, op = state, state["case"]["op"]
    if op == "attn":
        return gdn.attn_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], k_scale=s["ks"], v_scale=s["vs"])
    if op == "append":
        return gdn.kv_append(s["new_k"], s["new_v"], s["k"], s["v"], s["table"], s["lens"], cu_seqlens=s["cu"],
                             k_scale=s["ks"], v_scale=s["vs"])
    if op == "copy":
        return gdn.pages_copy(s["pool"], s["src"], s["dst"])
    if op == "compact":
        return gdn.pages_compact(s["table"], s["refs"])
    page = s["case"]["page"]
    if op == "extend":
        return gdn.pages_extend(s["table"], s["lens"], s["refs"], s["add"], page)
    if op == "fork":
        return gdn.pages_fork(s["table"], s["lens"], s["refs"], s["parent"], page)
    return gdn.pages_free(s["table"], s["lens"], s["refs"], s["mask"], page)


def work(case):
    op = case["op"]
    if op == "attn":
        lens = _lens(case)
        seen = sum(max(0, n - t) for n in lens for t in range(case["new"]))
        held, row = sum(lens), case["hkv"] * case["d"] * BYTES[case["cache"]]
        q = case["rows"] * case["new"] * case["hq"] * case["d"]
        return {"bytes": 2 * held * row + 2 * q * BYTES[case["io"]] + 4 * sum(-(-n // case["page"]) for n in lens),
                "flops": 4 * seen * case["hq"] * case["d"]}
    if op == "append":
        one = sum(_counts(case)) * case["hkv"] * case["d"]
        return {"bytes": 2 * one * (BYTES[case["io"]] + BYTES[case["cache"]]), "flops": 0}
    if op == "copy":
        return {"bytes": 2 * case["pairs"] * case["bytes"], "flops": 0}
    # the table and the counts once each way
    entries = case["rows"] * (case["max_pages"] + 2) + case["n_pages"]
    return {"bytes": 8 * entries + (4 * case["n_pages"] if op == "compact" else 0), "flops": 0}


# ------------------------------------------------------------------- exact --


def _exact_attn(case, s):
    """Row by row and token by token: a softmax over the tokens that it sees, in 64 bits."""
    q, table = s["q"].double(), s["table"].cpu().tolist()
    out, group, page = torch.zeros_like(q), case["hq"] // case["hkv"], case["page"]
    ks, vs = (torch.ones(case["hkv"], device="cuda") if x is None else x for x in (s["ks"], s["vs"]))
    as_bytes = case["cache"] == "e4m3"
    k, v = ((c.view(torch.uint8) if as_bytes else c) for c in (s["k"], s["v"]))
    for b, n in enumerate(s["lens"].tolist()):
        if n <= 0:
            continue
        ids = torch.tensor(table[b][:-(-n // page)], device="cuda")
        kb, vb = (c[ids] for c in (k, v))
        if as_bytes:
            kb, vb = kb.view(torch.float8_e4m3fn).float(), vb.view(torch.float8_e4m3fn).float()
        for h in range(case["hkv"]):
            kh, vh = (c[:, :, h].reshape(-1, case["d"])[:n].double() for c in (kb, vb))
            x = torch.matmul(q[b, :, h * group:(h + 1) * group].reshape(-1, case["d"]), (kh * ks[h].double()).T.contiguous())
            x = x.reshape(case["new"], group, n) * case["d"] ** -0.5
            for t in range(case["new"]):
                m = n - case["new"] + t + 1
                if m > 0:
                    w = torch.softmax(x[t, :, :m], -1)
                    out[b, t, h * group:(h + 1) * group] = torch.matmul(w, vh[:m]) * vs[h].double()
    return out


def _exact_append(case, s):
    caches, start = [], 0
    for x, cache, scale in ((s["new_k"], s["k"], s["ks"]), (s["new_v"], s["v"], s["vs"])):
        x, c = x.double().reshape(-1, case["hkv"], case["d"]), cache.double()
        if scale is not None:
            x = torch.clamp(x / scale.double()[:, None], -448, 448)
        start = 0
        for b, (n, end) in enumerate(zip(_counts(case), s["lens"].tolist())):
            at = torch.arange(end - n, end, device="cuda")
            c[s["table"][b].long()[at // case["page"]], at % case["page"]] = x[start:start + n]
            start += n
        caches.append(c)
    return tuple(caches)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn":
        return _exact_attn(case, s)
    if case["op"] == "append":
        return _exact_append(case, s)
    if case["op"] == "copy":
        pool = s["pool"].double()
        for i, j in zip(s["src"].tolist(), s["dst"].tolist()):
            pool[j].copy_(s["pool"][i])
        return pool
    return None  # whole numbers: the plain form's own
