"""Cases of the shared-prefix decode and of the page pool: their inputs, a plain form in torch, and exact values.

Shared-prefix decode: a batch of sequences in groups; the sequences of a group begin with the same cache blocks
(samples of one prompt, beams, requests behind one system prompt) and each goes on in blocks of its own.  One query
token each: out[b][h] = softmax(scale * q[b][h] . K^T) V over the sequence's whole context, on a bf16 or an INT8 cache.

Page pool: block tables, context lengths and reference counts of a cache's pages, held on the device beside the pages
of all layers.  append gives rows their next tokens' slots (new pages: the lowest free ids, in row order), fork makes a
row share another's full pages and copies its partly filled one, free returns pages, compact moves the used pages to
the lowest ids.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # eight samples of one 300-token prompt right after its prefill: one page shared, everything else latency
        {"name": "shared 8x300", "op": "shared", "kind": "bf16", "hq": 16, "hkv": 8, "d": 128, "bs": 256, "groups": 1,
         "size": 8, "prefix": 256, "tail": 64, "lens": 1},
        # a system prompt of 4096 tokens before 64 conversations of up to 1024 tokens
        {"name": "shared 64x4096", "op": "shared", "kind": "bf16", "hq": 28, "hkv": 4, "d": 128, "bs": 16, "groups": 1,
         "size": 64, "prefix": 4096, "tail": 1024, "lens": 2},
        # a 32768-token document and 256 questions on it: products, not bytes, bound the prefix
        {"name": "shared 256x32768", "op": "shared", "kind": "bf16", "hq": 28, "hkv": 4, "d": 128, "bs": 16, "groups": 1,
         "size": 256, "prefix": 32768, "tail": 1024, "lens": 3},
        # 24 prompts, each sampled 1 to 16 times, prompts of very different lengths
        {"name": "shared ragged groups", "op": "shared", "kind": "bf16", "hq": 16, "hkv": 8, "d": 128, "bs": 256,
         "groups": 24, "size": 16, "prefix": 8192, "tail": 700, "lens": 4},
        # four beams of a 1000-token prompt on an INT8 cache, heads of 64
        {"name": "shared int8 4x1000", "op": "shared", "kind": "int8", "hq": 12, "hkv": 1, "d": 64, "bs": 64, "groups": 1,
         "size": 4, "prefix": 1000, "tail": 77, "lens": 5},
        # 64 conversations behind a 16384-token prompt on an INT8 cache
        {"name": "shared int8 64x16384", "op": "shared", "kind": "int8", "hq": 28, "hkv": 4, "d": 128, "bs": 16,
         "groups": 1, "size": 64, "prefix": 16384, "tail": 1024, "lens": 6},
        # eight prompts of a prefill batch get their pages, take one decode step and leave again
        {"name": "append 8 prompts", "op": "append", "blocks": 64, "bs": 256, "rows": 16, "live": 4, "ctx": 600, "n": 8,
         "new": 256, "lens": 7},
        # 256 prompts of up to 2048 tokens in a pool of 131072 small pages, most of it free
        {"name": "append 256 prompts", "op": "append", "blocks": 131072, "bs": 16, "rows": 512, "live": 200, "ctx": 2048,
         "n": 256, "new": 2048, "lens": 8},
        # a 300-token prompt branches into eight samples: 44 rows of its last page, 28 layers
        {"name": "fork 1 into 8", "op": "fork", "kind": "bf16", "layers": 28, "hkv": 8, "d": 128, "bs": 256, "blocks": 24,
         "live": 3, "ctx": 300, "n": 8, "each": 8, "lens": 9},
        # 64 running sequences branch into four beams each, pages of 16 tokens
        {"name": "fork 64 into 256", "op": "fork", "kind": "bf16", "layers": 28, "hkv": 4, "d": 128, "bs": 16,
         "blocks": 2048, "live": 64, "ctx": 330, "n": 256, "each": 4, "lens": 10},
        # a small pool after a few sequences have left
        {"name": "compact 64 pages", "op": "compact", "kind": "bf16", "layers": 4, "hkv": 4, "d": 128, "bs": 16,
         "blocks": 64, "live": 6, "ctx": 100, "lens": 11},
        # half of a pool's 2048 pages in use and scattered, 28 layers
        {"name": "compact 2048 pages", "op": "compact", "kind": "bf16", "layers": 28, "hkv": 4, "d": 128, "bs": 16,
         "blocks": 2048, "live": 48, "ctx": 680, "lens": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = ((16, 8, 128), (28, 4, 128), (12, 1, 64), (7, 1, 128), (8, 8, 128), (4, 2, 64), (16, 1, 128))


def draw(rng):
    op = rng.choice(("shared", "shared", "shared", "append", "fork", "compact"))
    lens = rng.randrange(100, 1 << 20)
    if op == "shared":
        hq, hkv, d = rng.choice(HEADS)
        groups = _log(rng, 1, 24)
        size = _log(rng, 1, 256 // groups)
        # at most the keys and heads of 256 sequences behind 32768 tokens of 4 heads of 128
        most = min(32768 if groups == 1 else 8192, (1 << 32) // (groups * size * hkv * d))
        return {"op": op, "kind": rng.choice(("bf16", "bf16", "int8")), "hq": hq, "hkv": hkv, "d": d,
                "bs": 1 << rng.randint(4, 8), "groups": groups, "size": size, "prefix": _log(rng, 16, most),
                "tail": _log(rng, 1, 1024), "lens": lens}
    if op == "append":
        bs = 1 << rng.randint(4, 8)
        n, new, live, ctx = _log(rng, 1, 256), _log(rng, 1, 2048), _log(rng, 1, 200), _log(rng, 1, 2048)
        least = n * (-(-(new + 1) // bs)) + live * (-(-ctx // bs))
        return {"op": op, "blocks": least + _log(rng, 1, 100000), "bs": bs, "rows": n + live + rng.randrange(32),
                "live": live, "ctx": ctx, "n": n, "new": new, "lens": lens}
    layers = _log(rng, 1, 28)
    hkv, d = rng.choice(((4, 128), (8, 128), (1, 64), (2, 64)))
    kind = rng.choice(("bf16", "int8"))
    bs = 1 << rng.randint(4, 6)
    live, ctx = _log(rng, 1, 64), _log(rng, 1, 400)
    pages = live * (-(-ctx // bs))
    if op == "fork":
        each = rng.randint(1, 8)
        n = rng.randint(1, live) * each
        # a child takes at most two pages of its own: the copy of the partly filled one and its next token's
        return {"op": op, "kind": kind, "layers": layers, "hkv": hkv, "d": d, "bs": bs,
                "blocks": pages + 2 * n + rng.randrange(64), "live": live, "ctx": ctx, "n": n, "each": each,
                "lens": lens}
    return {"op": op, "kind": kind, "layers": layers, "hkv": hkv, "d": d, "bs": bs,
            "blocks": pages + _log(rng, 1, 600), "live": live, "ctx": ctx, "lens": lens}


# ---------------------------------------------------------------- lengths (of the case, not of the seed)

def _shared_lens(c):
    """(group sizes, shared tokens of each group, context of each sequence)."""
    r = random.Random(c["lens"])
    if c["groups"] == 1:
        sizes, prefix = [c["size"]], [c["prefix"]]
    else:
        sizes = [r.randint(1, c["size"]) for _ in range(c["groups"])]
        prefix = [_log(r, 1, c["prefix"]) for _ in range(c["groups"])]
    shared = [p // c["bs"] * c["bs"] for p in prefix]  # whole pages; what is left of the prompt is each one's own copy
    ctx = [p + r.randint(1, c["tail"]) for p, n in zip(prefix, sizes) for _ in range(n)]
    return sizes, shared, ctx


def _pool_lens(c):
    """(context of each live row, tokens that each of n new rows brings)."""
    r = random.Random(c["lens"])
    ctx = [c["ctx"] if c["live"] <= 3 else r.randint(max(1, c["ctx"] // 8), c["ctx"]) for _ in range(c["live"])]
    new = [r.randint(max(1, c["new"] // 16), c["new"]) for _ in range(c["n"])] if c["op"] == "append" else []
    return ctx, new


def work(case):
    c = case
    if c["op"] == "shared":
        sizes, shared, ctx = _shared_lens(c)
        keys = sum(shared) + sum(ctx) - sum(s * n for s, n in zip(shared, sizes))  # each page read once
        row = c["hkv"] * (2 * c["d"] if c["kind"] == "bf16" else c["d"] + 2)
        return {"bytes": 2 * keys * row + 2 * 2 * len(ctx) * c["hq"] * c["d"], "flops": 4 * c["hq"] * c["d"] * sum(ctx)}
    ctx, new = _pool_lens(c)
    bs = c["bs"]
    if c["op"] == "append":
        pages = sum(-(-(n + 1) // bs) for n in new)
        # page ids and counts taken and given back; a slot for each token; the lengths
        return {"bytes": 4 * (4 * pages + 2 * sum(new) + len(new) * 6), "flops": 0}
    row = 2 * c["hkv"] * (2 * c["d"] if c["kind"] == "bf16" else c["d"] + 2) * c["layers"]
    if c["op"] == "fork":
        par = [ctx[i // c["each"] % len(ctx)] for i in range(c["n"])]
        return {"bytes": 2 * row * sum(p % bs for p in par) + 4 * sum(4 * (p // bs) + 8 for p in par), "flops": 0}
    used = sum(-(-x // bs) for x in ctx)
    # on average used * (1 - used / blocks) pages lie above the first `used` ids
    return {"bytes": int(2 * row * bs * used * (1 - used / c["blocks"])) + 16 * c["blocks"], "flops": 0}


# ---------------------------------------------------------------- inputs

def _values(shape, g):
    """N(0, 1) in bf16, drawn in pieces."""
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    flat = out.view(-1)
    for s in range(0, flat.numel(), 1 << 26):
        e = min(flat.numel(), s + (1 << 26))
        flat[s:e] = torch.randn(e - s, generator=g, device=DEV).to(torch.bfloat16)
    return out


def _codes(shape, g):
    """INT8 codes of N(0, 1) rows and their fp16 scales, [..., blocks, heads, block] as the cache holds them."""
    codes = torch.empty(shape, dtype=torch.int8, device=DEV)
    scale = torch.empty(shape[:-1], dtype=torch.float16, device=DEV)
    flat, sflat = codes.view(-1, shape[-1]), scale.view(-1)
    for s in range(0, flat.shape[0], 1 << 19):
        e = min(flat.shape[0], s + (1 << 19))
        x = torch.randn(e - s, shape[-1], generator=g, device=DEV)
        a = x.abs().amax(1) / 127
        flat[s:e] = torch.round(x / a[:, None]).to(torch.int8)
        sflat[s:e] = a.to(torch.float16)
    return codes, scale.transpose(-1, -2).contiguous()


def _cache(c, shape, g):
    if c["kind"] == "bf16":
        return {"k": _values(shape, g), "v": _values(shape, g)}
    k, ks = _codes(shape, g)
    v, vs = _codes(shape, g)
    return {"k": k, "v": v, "ks": ks, "vs": vs}


def _i32(x):
    return torch.tensor(np.asarray(x, np.int32), device=DEV)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = np.random.default_rng(seed)
    if c["op"] == "shared":
        sizes, shared, ctx = _shared_lens(c)
        bs = c["bs"]
        first = np.repeat(np.arange(len(sizes)), sizes)
        own_pages = [-(-x // bs) - shared[i] // bs for x, i in zip(ctx, first)]
        blocks = sum(s // bs for s in shared) + sum(own_pages)
        ids = r.permutation(blocks + 3).astype(np.int32)
        cut = np.cumsum([0] + [s // bs for s in shared] + own_pages)
        runs = [ids[a:b] for a, b in zip(cut[:-1], cut[1:])]
        lists = [np.concatenate([runs[i], runs[len(sizes) + b]]) for b, i in enumerate(first)]
        table = np.full((len(ctx), max(len(x) for x in lists)), -1, np.int32)
        for row, x in zip(table, lists):
            row[:len(x)] = x
        s = {"c": c, "scale": c["d"] ** -0.5, "table": _i32(table), "ctx": _i32(ctx),
             "q": _values((len(ctx), c["hq"], c["d"]), g), **_cache(c, (blocks + 3, bs, c["hkv"], c["d"]), g)}
        s["out"] = torch.empty_like(s["q"])
        if own:
            from paged_kv_cache_kvcache_gb300 import pagedattn as pa
            s["dims"] = pa.make_dims(blocks + 3, bs, c["hq"], c["hkv"], c["d"])
            s["plan"] = pa.pa_pack_decode_shared(s["dims"], ctx, np.cumsum([0] + sizes), block_lists=lists).upload()
            s["ws"] = pa.shared_workspace(s["plan"])
        return s
    ctx, new = _pool_lens(c)
    bs, blocks = c["bs"], c["blocks"]
    rows = {"append": c.get("rows"), "fork": c["live"] + c.get("n", 0), "compact": c["live"]}[c["op"]]
    width = max(-(-(max(ctx) + 1) // bs), -(-(max(new, default=0) + 1) // bs))
    ids, place = r.permutation(blocks).astype(np.int32), r.permutation(rows)
    table, lens, refs, at = np.full((rows, width), -1, np.int32), np.zeros(rows, np.int32), np.zeros(blocks, np.int32), 0
    for x, row in zip(ctx, place):
        n = -(-x // bs)
        table[row, :n], lens[row] = ids[at:at + n], x
        refs[ids[at:at + n]] += 1
        at += n
    s = {"c": c, "table": _i32(table), "ctx": _i32(lens), "refs": _i32(refs)}
    if c["op"] == "append":
        shape = (1, blocks, bs, 1, 64)  # the pages themselves take no part
        s.update(k=torch.empty(shape, dtype=torch.bfloat16, device=DEV), v=torch.empty(shape, dtype=torch.bfloat16, device=DEV))
        s["rows"], total = _i32(place[c["live"]:c["live"] + c["n"]]), sum(new)
        s["cu"], s["step"] = _i32(np.cumsum([0] + new)), _i32(np.arange(c["n"] + 1))
        s["slots"] = torch.empty(total, dtype=torch.int32, device=DEV)
        s["slots1"] = torch.empty(c["n"], dtype=torch.int32, device=DEV)
    else:
        s.update(_cache(c, (c["layers"], blocks, bs, c["hkv"], c["d"]), g))
        if c["op"] == "fork":
            s["parents"] = _i32([place[i // c["each"] % c["live"]] for i in range(c["n"])])
            s["children"], s["step"] = _i32(place[c["live"]:]), _i32(np.arange(c["n"] + 1))
            s["slots1"] = torch.empty(c["n"], dtype=torch.int32, device=DEV)
        else:
            s["remap"] = torch.empty(blocks, dtype=torch.int32, device=DEV)
            s["table_out"], s["refs_out"] = torch.empty_like(s["table"]), torch.empty_like(s["refs"])
    if own:
        from paged_kv_cache_kvcache_gb300 import pagedattn as pa
        hkv, d = s["k"].shape[3:]
        s["dims"] = pa.make_dims(blocks, bs, hkv, hkv, d)
        s["pool"] = pa.PagePool(s["dims"], s["k"], s["v"], s["table"], s["ctx"], s["refs"], k_scale=s.get("ks"),
                                v_scale=s.get("vs"))
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    s = state
    op = s["c"]["op"]
    if own:
        from paged_kv_cache_kvcache_gb300 import pagedattn as pa
        if op == "shared":
            if s["c"]["kind"] == "bf16":
                pa.pa_decode_shared(s["dims"], s["q"], s["k"], s["v"], s["plan"], s["scale"], s["out"], s["ws"])
            else:
                pa.pa_decode_shared_int8(s["dims"], s["q"], s["k"], s["v"], s["ks"], s["vs"], s["plan"], s["scale"],
                                         s["out"], s["ws"])
        elif op == "append":
            pa.pa_pool_append(s["dims"], s["pool"], s["rows"], s["cu"], s["slots"])
            pa.pa_pool_append(s["dims"], s["pool"], s["rows"], s["step"], s["slots1"])
            pa.pa_pool_free(s["dims"], s["pool"], s["rows"])
        elif op == "fork":
            pa.pa_pool_fork(s["dims"], s["pool"], s["parents"], s["children"])
            pa.pa_pool_append(s["dims"], s["pool"], s["children"], s["step"], s["slots1"])
            pa.pa_pool_free(s["dims"], s["pool"], s["children"])
        else:
            pa.pa_pool_compact(s["dims"], s["pool"], s["remap"], s["table_out"], s["refs_out"])
    elif op == "shared":
        s["out"] = _plain_shared(s)
    elif op == "append":
        s["slots"] = _plain_append(s, s["rows"], s["cu"], s["slots"].numel())
        s["slots1"] = _plain_append(s, s["rows"], s["step"], s["slots1"].numel())
        _plain_free(s, s["rows"])
    elif op == "fork":
        _plain_fork(s)
        s["slots1"] = _plain_append(s, s["children"], s["step"], s["slots1"].numel())
        _plain_free(s, s["children"])
    else:
        _plain_compact(s)
    return _outputs(s)


def _outputs(s):
    op = s["c"]["op"]
    if op == "shared":
        return {"out": s["out"]}
    if op == "append":
        return {n: s[n] for n in ("slots", "slots1", "table", "ctx", "refs")}
    names = ("slots1", "table", "ctx", "refs") if op == "fork" else ("remap", "table_out", "refs_out")
    got = {n: s[n] for n in names + ("k", "v")}
    if "ks" in s:  # what is held in 8 bits, as the values it stands for
        got["k"] = s["k"].float() * s["ks"].transpose(-1, -2)[..., None].float()
        got["v"] = s["v"].float() * s["vs"].transpose(-1, -2)[..., None].float()
    return got


def _plain_shared(s):
    c, q = s["c"], s["q"].float()
    b, bs = q.shape[0], c["bs"]
    page = s["table"].clamp_min(0).long()
    k, v = s["k"][page].float(), s["v"][page].float()  # [b, pages, bs, hkv, d]
    if "ks" in s:
        k = k * s["ks"][page].transpose(-1, -2)[..., None].float()
        v = v * s["vs"][page].transpose(-1, -2)[..., None].float()
    k, v = (x.reshape(b, -1, c["hkv"], c["d"]).transpose(1, 2) for x in (k, v))
    sc = torch.matmul(q.view(b, c["hkv"], -1, c["d"]) * s["scale"], k.transpose(2, 3))  # [b, hkv, group, keys]
    seen = torch.arange(k.shape[2], device=DEV)[None, :] < s["ctx"][:, None]
    sc = torch.where(seen[:, None, None, :], sc, torch.full_like(sc, -math.inf))
    p = torch.exp(sc - sc.amax(-1, keepdim=True))
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
    return o.reshape(q.shape).to(s["q"].dtype)


def _free_ids(s):
    """The free pages' ids, ascending; -1 behind the last."""
    n = s["refs"].numel()
    free = s["refs"] == 0
    rank = torch.cumsum(free, 0) - 1
    ids = torch.full((n + 1,), -1, dtype=torch.int64, device=DEV)
    ids[torch.where(free, rank, n)] = torch.arange(n, device=DEV)
    ids[n] = -1
    return ids


def _count(s, pages, sign):
    """sign * how often each page is named (-1: none)."""
    n = s["refs"].numel()
    at = torch.where(pages >= 0, pages, n).reshape(-1).long()
    s["refs"] += torch.zeros(n + 1, dtype=torch.int32, device=DEV).index_add_(
        0, at, torch.full(at.shape, sign, dtype=torch.int32, device=DEV))[:n]


def _plain_append(s, rows, cu, total):
    bs, rows, cu = s["c"]["bs"], rows.long(), cu.long()
    have, new = s["ctx"][rows].long(), cu[1:] - cu[:-1]
    old, all_ = (have + bs - 1) // bs, (have + new + bs - 1) // bs
    start = torch.cumsum(all_ - old, 0) - (all_ - old)
    col = torch.arange(s["table"].shape[1], device=DEV)[None, :]
    fresh = (col >= old[:, None]) & (col < all_[:, None])
    ids = _free_ids(s)
    page = ids[torch.where(fresh, start[:, None] + col - old[:, None], ids.numel() - 1)]
    table = torch.where(fresh, page, s["table"][rows].long())
    _count(s, page, 1)
    s["table"][rows] = table.to(torch.int32)
    s["ctx"][rows] = (have + new).to(torch.int32)
    t = torch.arange(total, device=DEV)
    i = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = have[i] + t - cu[i]
    return (table[i, pos // bs] * bs + pos % bs).to(torch.int32)


def _plain_free(s, rows):
    rows = rows.long()
    _count(s, s["table"][rows], -1)
    s["table"][rows] = -1
    s["ctx"][rows] = 0


def _plain_fork(s):
    bs, par, chi = s["c"]["bs"], s["parents"].long(), s["children"].long()
    ctx = s["ctx"][par].long()
    full, rest = ctx // bs, ctx % bs
    part = rest > 0
    fresh = _free_ids(s)[torch.cumsum(part, 0) - part.long()]
    col = torch.arange(s["table"].shape[1], device=DEV)[None, :]
    old = s["table"][par].long()
    table = torch.where((col == full[:, None]) & part[:, None], fresh[:, None], old)
    _count(s, table, 1)
    s["table"][chi] = table.to(torch.int32)
    s["ctx"][chi] = ctx.to(torch.int32)
    at = torch.nonzero(part)[:, 0]
    src, dst = old[at, full[at]], fresh[at]
    live = torch.arange(bs, device=DEV)[None, :] < rest[at][:, None]  # [copies, bs]
    for name, mask in (("k", live[None, :, :, None, None]), ("v", live[None, :, :, None, None]),
                       ("ks", live[None, :, None, :]), ("vs", live[None, :, None, :])):
        if name in s:
            s[name][:, dst] = torch.where(mask, s[name][:, src], s[name][:, dst])


def _plain_compact(s):
    refs, ids = s["refs"], torch.arange(s["refs"].numel(), device=DEV)
    used = refs > 0
    low = ids < used.sum()
    src, dst = torch.nonzero(used & ~low)[:, 0], torch.nonzero(~used & low)[:, 0]
    remap = torch.where(used, ids, -1)
    remap[src] = dst
    s["remap"] = remap.to(torch.int32)
    s["table_out"] = torch.where(s["table"] >= 0, remap[s["table"].clamp_min(0).long()], -1).to(torch.int32)
    s["refs_out"] = refs.clone()
    s["refs_out"][dst] = refs[src]
    s["refs_out"][src] = 0
    for name in ("k", "v", "ks", "vs"):
        if name in s:
            s[name][:, dst] = s[name][:, src]


# ---------------------------------------------------------------- exact values

def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "shared":
        return {"out": _exact_shared(s)}
    bs = c["bs"]
    table, ctx, refs = s["table"].tolist(), s["ctx"].tolist(), s["refs"].tolist()

    def lowest(n):
        got = []
        for p, x in enumerate(refs):
            if len(got) == n:
                break
            if x == 0:
                got.append(p)
        return got

    def grow(rows, counts):
        need = sum(-(-(ctx[r] + n) // bs) - -(-ctx[r] // bs) for r, n in zip(rows, counts))
        pages, slots = iter(lowest(need)), []
        for r, n in zip(rows, counts):
            for pos in range(ctx[r], ctx[r] + n):
                if pos % bs == 0:
                    table[r][pos // bs] = p = next(pages)
                    refs[p] += 1
                slots.append(table[r][pos // bs] * bs + pos % bs)
            ctx[r] += n
        return _i32(slots)

    def drop(rows):
        for r in rows:
            for j, p in enumerate(table[r]):
                if p >= 0:
                    refs[p] -= 1
                table[r][j] = -1
            ctx[r] = 0

    got = {}
    if c["op"] == "append":
        rows = s["rows"].tolist()
        got["slots"] = grow(rows, np.diff(s["cu"].tolist()).tolist())
        got["slots1"] = grow(rows, [1] * len(rows))
        drop(rows)
        return {**got, "table": _i32(table), "ctx": _i32(ctx), "refs": _i32(refs)}
    if c["op"] == "fork":
        par, chi = s["parents"].tolist(), s["children"].tolist()
        pages = iter(lowest(sum(ctx[p] % bs > 0 for p in par)))
        for p, r in zip(par, chi):
            n, rest = divmod(ctx[p], bs)
            table[r][:n] = table[p][:n]
            if rest:
                src, dst = table[p][n], next(pages)
                table[r][n] = dst
                for name in ("k", "v"):
                    s[name][:, dst, :rest] = s[name][:, src, :rest]
                for name in ("ks", "vs"):
                    if name in s:
                        s[name][:, dst, :, :rest] = s[name][:, src, :, :rest]
            for page in table[r]:
                if page >= 0:
                    refs[page] += 1
            ctx[r] = ctx[p]
        s["slots1"] = grow(chi, [1] * len(chi))
        drop(chi)
        s.update(table=_i32(table), ctx=_i32(ctx), refs=_i32(refs))
        return _outputs(s)
    used = [p for p, x in enumerate(refs) if x]
    holes = iter([p for p, x in enumerate(refs) if not x])
    remap, out = [-1] * len(refs), [0] * len(refs)
    for p in used:
        remap[p] = p if p < len(used) else next(holes)
        out[remap[p]] = refs[p]
        if remap[p] != p:
            for name in ("k", "v", "ks", "vs"):
                if name in s:
                    s[name][:, remap[p]] = s[name][:, p]
    s.update(remap=_i32(remap), refs_out=_i32(out), table_out=_i32([[remap[p] if p >= 0 else -1 for p in t] for t in table]))
    return _outputs(s)


def _exact_shared(s):
    c = s["c"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    for b, (n, pages) in enumerate(zip(s["ctx"].tolist(), s["table"].tolist())):
        pages = torch.tensor(pages[:-(-n // c["bs"])], device=DEV)
        k, v = s["k"][pages].double(), s["v"][pages].double()
        if "ks" in s:
            k *= s["ks"][pages].double().permute(0, 2, 1)[..., None]
            v *= s["vs"][pages].double().permute(0, 2, 1)[..., None]
        k, v = k.flatten(0, 1)[:n], v.flatten(0, 1)[:n]
        q = s["q"][b].double().view(c["hkv"], -1, c["d"])
        p = torch.softmax(torch.einsum("hgd,thd->hgt", q, k) * s["scale"], -1)
        out[b] = torch.einsum("hgt,thd->hgd", p, v).reshape(c["hq"], c["d"])
    return out
