"""Cases of a decode step over a bounded cache: inputs, plain forms in torch, and exact values.

rope: the queries' and keys' norm for each head, their rotation by the token's position (one position, or one per
axis), and the store of the new keys and values into the paged cache (bf16 or INT8), in one pass.

prefill_window, decode_window: attention that sees the first `sinks` keys of a sequence and the last `window` ones.

decode_weights: a decode step that also adds each key's attention weight to the score that is kept for it.

evict: rows of a page pool shrink to `budget` tokens: their first ones, their last ones, and of the others those of the
highest scores; what stays moves together, in order, and the pages left over go back to the pool.
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
        # one decode step of eight sequences: a row per head, everything else latency
        {"name": "rope 8 tokens", "op": "rope", "kind": "bf16", "hq": 16, "hkv": 8, "d": 128, "bs": 256, "tokens": 8,
         "pad": 0, "rot": 128, "axes": 1, "pairs": "half", "norm": True, "packed": True, "far": 32768, "lens": 1},
        # four prompts of 4096 tokens, no norm
        {"name": "rope 16384 tokens", "op": "rope", "kind": "bf16", "hq": 28, "hkv": 4, "d": 128, "bs": 16,
         "tokens": 16384, "pad": 0, "rot": 128, "axes": 1, "pairs": "half", "norm": False, "packed": True, "far": 32768,
         "lens": 2},
        # images and text (time, height, width) into an INT8 cache, a batch padded to a bucket
        {"name": "rope 5000 tokens int8", "op": "rope", "kind": "int8", "hq": 16, "hkv": 8, "d": 128, "bs": 16,
         "tokens": 5000, "pad": 120, "rot": 128, "axes": 3, "pairs": "half", "norm": True, "packed": False,
         "far": 32768, "lens": 3},
        # four prompts of 4096 tokens in a layer that sees 1024 of them
        {"name": "prefill 4x4096", "op": "prefill", "kind": "bf16", "hq": 28, "hkv": 4, "d": 128, "bs": 16, "seqs": 4,
         "prefix": 0, "new": 4096, "least": 4096, "window": 1024, "sinks": 4, "lens": 4},
        # chunks of prompts behind cached prefixes, INT8 cache, pages in front of the window given back
        {"name": "prefill 16 chunks int8", "op": "prefill", "kind": "int8", "hq": 16, "hkv": 8, "d": 128, "bs": 32,
         "seqs": 16, "prefix": 2000, "new": 1000, "least": 1, "window": 512, "sinks": 100, "lens": 5},
        # eight short conversations: latency
        {"name": "window 8x900", "op": "window", "kind": "bf16", "hq": 16, "hkv": 8, "d": 128, "bs": 256, "seqs": 8,
         "ctx": 900, "least": 100, "window": 512, "sinks": 4, "lens": 6},
        # long contexts of which 4096 + 64 tokens are kept
        {"name": "window 64x32768", "op": "window", "kind": "bf16", "hq": 28, "hkv": 4, "d": 128, "bs": 16, "seqs": 64,
         "ctx": 32768, "least": 20000, "window": 4096, "sinks": 64, "lens": 7},
        # many conversations of very different lengths
        {"name": "window 200x8192 int8", "op": "window", "kind": "int8", "hq": 28, "hkv": 4, "d": 128, "bs": 16,
         "seqs": 200, "ctx": 8192, "least": 1, "window": 1000, "sinks": 4, "lens": 8},
        {"name": "weights 8x600", "op": "weights", "kind": "bf16", "hq": 16, "hkv": 8, "d": 128, "bs": 256, "seqs": 8,
         "ctx": 600, "least": 100, "decay": 1.0, "lens": 9},
        # a full batch at its budget of 8192 tokens
        {"name": "weights 64x8192", "op": "weights", "kind": "bf16", "hq": 28, "hkv": 4, "d": 128, "bs": 16, "seqs": 64,
         "ctx": 8192, "least": 4096, "decay": 0.95, "lens": 10},
        # one layer's cache, a few rows at their limit
        {"name": "evict 4x2048", "op": "evict", "kind": "bf16", "layers": 1, "hkv": 8, "d": 128, "bs": 16, "rows": 4,
         "ctx": 2048, "least": 2000, "budget": 1024, "first": 4, "last": 256, "lens": 11},
        # all layers' pages of sixteen long rows
        {"name": "evict 16x4096 28 layers", "op": "evict", "kind": "bf16", "layers": 28, "hkv": 4, "d": 128, "bs": 16,
         "rows": 16, "ctx": 4096, "least": 4096, "budget": 2048, "first": 4, "last": 1024, "lens": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = ((16, 8, 128), (28, 4, 128), (12, 1, 64), (7, 1, 128), (8, 8, 128), (4, 2, 64), (16, 1, 128))


def draw(rng):
    op = rng.choice(("rope", "prefill", "window", "weights", "evict"))
    lens = rng.randrange(100, 1 << 20)
    hq, hkv, d = rng.choice(HEADS)
    c = {"op": op, "kind": rng.choice(("bf16", "int8")), "hq": hq, "hkv": hkv, "d": d, "bs": 1 << rng.randint(4, 8),
         "lens": lens}
    if op == "rope":
        tokens = _log(rng, 1, min(16384, 16384 * 36 * 128 // ((hq + 2 * hkv) * d)))
        rot = rng.choice((d, d, d, d // 2, d // 4))
        return {**c, "tokens": tokens, "pad": rng.choice((0, 0, _log(rng, 1, 200))), "rot": rot,
                "axes": rng.choice((1, 1, 2, 3)), "pairs": rng.choice(("half", "half", "next")),
                "norm": rng.random() < 0.6, "packed": rng.random() < 0.6, "far": _log(rng, 2048, 131072)}
    if op == "prefill":
        seqs, window, sinks = _log(rng, 1, 16), _log(rng, 1, 4096), rng.choice((0, 1, 4, _log(rng, 1, 300)))
        # at most the pairs that the mask is made for in four prompts of 4096 tokens and 28 heads
        most = max(1, int(math.sqrt((1 << 30) / (seqs * hq))))
        new = _log(rng, 1, most)
        return {**c, "seqs": seqs, "prefix": rng.choice((0, _log(rng, 1, most))), "new": new, "least": 1,
                "window": window, "sinks": sinks}
    if op == "window":
        seqs = _log(rng, 1, 256)
        most = min(32768, (1 << 28) // (seqs * hkv * d))  # keys seen
        window = _log(rng, 1, min(8192, most))
        return {**c, "seqs": seqs, "ctx": _log(rng, 1, 65536), "least": 1, "window": window,
                "sinks": rng.choice((0, 1, 4, _log(rng, 1, 300)))}
    if op == "weights":
        seqs = _log(rng, 1, 128)
        most = min(16384, (1 << 28) // (seqs * hkv * d))
        return {**c, "seqs": seqs, "ctx": _log(rng, 1, most), "least": 1,
                "decay": rng.choice((1.0, 0.95, 0.5, 0.0))}
    layers, rows, hkv, d = _log(rng, 1, 28), _log(rng, 1, 64), *rng.choice(((4, 128), (8, 128), (1, 64), (2, 64)))
    ctx = _log(rng, 32, min(8192, 28 * 16 * 4096 * 512 // (layers * rows * hkv * d)))
    budget = rng.randint(max(1, ctx // 8), ctx)
    first = min(budget, rng.choice((0, 4, 64)))
    return {**c, "hkv": hkv, "d": d, "bs": 1 << rng.randint(4, 6), "layers": layers, "rows": rows, "ctx": ctx,
            "least": max(1, ctx // 2), "budget": budget, "first": first, "last": rng.randint(0, budget - first)}


# ---------------------------------------------------------------- lengths (of the case, not of the seed)

def _lens(c, n, least, most):
    r = random.Random(c["lens"])
    return [r.randint(min(least, most), most) for _ in range(n)]


def _prefill_lens(c):
    """(new tokens, cached tokens) of each sequence."""
    r = random.Random(c["lens"])
    new = [r.randint(min(c["least"], c["new"]), c["new"]) for _ in range(c["seqs"])]
    return new, [r.randint(0, c["prefix"]) for _ in range(c["seqs"])]


def _seen(pos, c):
    """Keys that a query at a position sees."""
    return min(pos + 1, c["window"]) + min(c["sinks"], max(0, pos + 1 - c["window"]))


def work(case):
    c, d, hkv = case, case["d"], case["hkv"]
    row = 2 * (2 * d if c["kind"] == "bf16" else d + 2)  # a token's key and value of one head, in the cache
    if c["op"] == "rope":
        n, t = c["tokens"], c["tokens"] + c["pad"]
        heads = t * c["hq"] + n * hkv
        # queries in and out, keys and values in and into the cache, positions and slots; angles are shared
        return {"bytes": t * (4 * c["hq"] * d + 4 * c["axes"] + 4) + n * hkv * (4 * d + row),
                "flops": heads * (4 * c["rot"] + (4 * d if c["norm"] else 0))}
    if c["op"] == "prefill":
        new, old = _prefill_lens(c)
        pairs = sum(_seen(o + i, c) for n, o in zip(new, old) for i in range(n))
        keys = sum(min(n + o, n - 1 + c["window"]) + min(c["sinks"], max(0, o + 1 - c["window"])) for n, o in zip(new, old))
        return {"bytes": keys * hkv * row + 4 * sum(new) * c["hq"] * d, "flops": 4 * pairs * c["hq"] * d}
    if c["op"] == "window":
        keys = sum(_seen(x - 1, c) for x in _lens(c, c["seqs"], c["least"], c["ctx"]))
        return {"bytes": keys * hkv * row + 4 * c["seqs"] * c["hq"] * d, "flops": 4 * keys * c["hq"] * d}
    if c["op"] == "weights":
        keys = sum(_lens(c, c["seqs"], c["least"], c["ctx"]))
        return {"bytes": keys * hkv * (row + 8) + 4 * c["seqs"] * c["hq"] * d, "flops": 4 * keys * c["hq"] * d}
    lens = [x for x in _lens(c, c["rows"], c["least"], c["ctx"]) if x > c["budget"]]
    moved = len(lens) * (c["budget"] - c["first"])
    return {"bytes": 2 * moved * hkv * row * c["layers"] + 4 * hkv * (sum(lens) + len(lens) * c["budget"]) + 1, "flops": 0}


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


def _tables(c, lens, seen_from, r):
    """Block tables of rows of these lengths, and the pool's pages. A row's pages between the sinks and the first key
    that its queries see (seen_from) have been given back: -1."""
    bs = c["bs"]
    table = np.full((len(lens), max(1, max(-(-x // bs) for x in lens))), -1, np.int32)
    for row, x, lo in zip(table, lens, seen_from):
        page = np.arange(-(-x // bs))
        row[:len(page)][(page * bs < c.get("sinks", 0)) | ((page + 1) * bs > lo)] = 0
    live = table >= 0
    blocks = int(live.sum()) + 3
    table[live] = r.permutation(blocks)[:int(live.sum())]
    return table, blocks


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = np.random.default_rng(seed)
    s = {"rope": _prepare_rope, "evict": _prepare_evict}.get(c["op"], _prepare_attention)(c, g, r)
    s["c"] = c
    return s


def _prepare_rope(c, g, r):
    n, t, bs, d, hq, hkv = c["tokens"], c["tokens"] + c["pad"], c["bs"], c["d"], c["hq"], c["hkv"]
    lens, q = random.Random(c["lens"]), []
    while sum(q) < n:  # the tokens of several prompts, or one each of many sequences
        q.append(min(n - sum(q), 1 if n <= 256 else lens.randint(1, n)))
    blocks = sum(-(-x // bs) for x in q) + 2
    ids, slots, pos, at = r.permutation(blocks), [], [], 0
    for x in q:
        i = np.arange(x) if x > 1 else r.integers(0, bs, 1)
        slots.append(ids[at + i // bs] * bs + i % bs)
        first = int(r.integers(0, c["far"] - x + 1)) if x < c["far"] else 0
        pos.append(first + np.arange(x) % c["far"])
        at += -(-x // bs)
    slots = np.concatenate(slots + [np.full(c["pad"], -1)])
    pos = np.concatenate(pos + [np.zeros(c["pad"], np.int64)])
    # the axes of text agree; an image's rows and columns run on their own
    pos = np.stack([pos] + [np.minimum(pos // 2 + r.integers(0, 64, t), c["far"] - 1) for _ in range(c["axes"] - 1)])
    half = c["rot"] // 2
    angle = torch.arange(c["far"], device=DEV, dtype=torch.float64)[:, None] * \
        1e6 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
    s = {"cos_sin": torch.cat([angle.cos(), angle.sin()], 1).float(),
         "positions": _i32(pos), "slots": _i32(slots), "pair_axis": np.arange(half) * c["axes"] // half}
    if c["packed"]:  # the output of one projection
        qkv = _values((t, (hq + 2 * hkv), d), g)
        s["q"], s["kn"], s["vn"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        s["q"], s["kn"], s["vn"] = _values((t, hq, d), g), _values((t, hkv, d), g), _values((t, hkv, d), g)
    s["qw"], s["kw"] = ((1 + 0.3 * torch.randn(2, d, generator=g, device=DEV)).to(torch.bfloat16).unbind(0) if c["norm"]
                        else (None, None))
    s["q_out"] = torch.empty((t, hq, d), dtype=torch.bfloat16, device=DEV)
    shape = (blocks, bs, hkv, d)
    kind = torch.bfloat16 if c["kind"] == "bf16" else torch.int8
    s["k"], s["v"] = torch.zeros(shape, dtype=kind, device=DEV), torch.zeros(shape, dtype=kind, device=DEV)
    if c["kind"] == "int8":
        s["ks"], s["vs"] = (torch.zeros((blocks, hkv, bs), dtype=torch.float16, device=DEV) for _ in range(2))
    if own:
        from paged_kv_cache_kvcache_gb300 import pagedattn as pa
        s["dims"] = pa.make_dims(blocks, bs, hq, hkv, d)
        s["rope"] = pa.Rope(s["dims"], s["cos_sin"], axes=c["axes"], pair_axis=s["pair_axis"],
                            interleaved=c["pairs"] == "next", q_weight=s["qw"], k_weight=s["kw"], eps=1e-6)
    return s


def _prepare_attention(c, g, r):
    bs = c["bs"]
    if c["op"] == "prefill":
        new, old = _prefill_lens(c)
        lens, tokens = [n + o for n, o in zip(new, old)], sum(new)
        lo = [max(0, o + 1 - c["window"]) for o in old]
    else:
        lens = _lens(c, c["seqs"], c["least"], c["ctx"])
        tokens, lo = len(lens), [max(0, x - c.get("window", x)) for x in lens]
    table, blocks = _tables(c, lens, lo, r)
    s = {"scale": c["d"] ** -0.5, "table": _i32(table), "ctx": _i32(lens),
         "q": _values((tokens, c["hq"], c["d"]), g), **_cache(c, (blocks, bs, c["hkv"], c["d"]), g)}
    s["out"] = torch.empty_like(s["q"])
    if c["op"] == "prefill":
        s["new"], s["first"] = _i32(new), _i32(np.cumsum([0] + new))
    if c["op"] == "weights":
        shape = (len(lens), c["hkv"], table.shape[1] * bs)
        s["scores"] = torch.empty(shape, device=DEV).exponential_(generator=g)
        s["scores"].masked_fill_(torch.arange(shape[2], device=DEV) >= s["ctx"][:, None, None] - 1, 0)
        s["scores_out"] = torch.zeros_like(s["scores"])
    if own:
        from paged_kv_cache_kvcache_gb300 import pagedattn as pa
        s["dims"] = pa.make_dims(blocks, bs, c["hq"], c["hkv"], c["d"])
        if c["op"] == "prefill":
            # the host's lists name a page it still knows in the place of one that was given back
            lists = [np.where(t[:-(-x // bs)] < 0, 0, t[:-(-x // bs)]) for t, x in zip(table, lens)]
            s["plan"] = pa.pa_pack_prefill(s["dims"], lens, new, lists).upload()
            s["ws"] = pa.prefill_workspace(s["plan"]) if c["kind"] == "int8" else None
        elif c["op"] == "weights":
            s["ws"] = pa.weights_workspace(s["dims"], len(lens), table.shape[1])
    return s


def _prepare_evict(c, g, r):
    bs, n = c["bs"], c["rows"]
    lens = _lens(c, n, c["least"], c["ctx"])
    pages = [-(-x // bs) for x in lens]
    blocks, width, rows = sum(pages) + 5, max(pages) + 1, n + 2
    meta = torch.zeros(rows * width + rows + -(-blocks // 4) * 4 + 16, dtype=torch.int32, device=DEV)
    refs, at = meta[:blocks], -(-blocks // 4) * 4
    table, ctx = meta[at:at + rows * width].view(rows, width), meta[at + rows * width:at + rows * width + rows]
    ids, place = r.permutation(blocks).astype(np.int32), r.permutation(rows)[:n]
    host, end = np.full((rows, width), -1, np.int32), 0
    for row, x in zip(place, pages):
        host[row, :x] = ids[end:end + x]
        end += x
    table.copy_(_i32(host))
    ctx[torch.as_tensor(place, device=DEV)] = _i32(lens)
    refs[torch.as_tensor(ids[:end], device=DEV).long()] = 1
    # weight gathers on few tokens
    scores = torch.empty((rows, c["hkv"], width * bs), device=DEV).exponential_(generator=g).pow_(2)
    scores.masked_fill_(torch.arange(width * bs, device=DEV) >= ctx[:, None, None], 0)
    s = {"meta": meta, "meta0": meta.clone(), "table": table, "ctx": ctx, "refs": refs, "rows": _i32(place),
         "scores": scores, "scores_out": torch.zeros_like(scores),
         "kept": torch.empty((n, c["budget"]), dtype=torch.int32, device=DEV),
         **_cache(c, (c["layers"], blocks, bs, c["hkv"], c["d"]), g)}
    if own:
        from paged_kv_cache_kvcache_gb300 import pagedattn as pa
        s["dims"] = pa.make_dims(blocks, bs, c["hkv"], c["hkv"], c["d"])
        s["pool"] = pa.PagePool(s["dims"], s["k"], s["v"], table, ctx, refs, k_scale=s.get("ks"), v_scale=s.get("vs"))
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    s, c = state, state["c"]
    op, int8 = c["op"], c["kind"] == "int8"
    if op == "evict":  # the rows at their limit again
        s["meta"].copy_(s["meta0"])
    if not own:
        {"rope": _plain_rope, "prefill": _plain_prefill, "window": _plain_decode, "weights": _plain_decode,
         "evict": _plain_evict}[op](s)
        return _outputs(s)
    from paged_kv_cache_kvcache_gb300 import pagedattn as pa
    if op == "rope":
        if int8:
            pa.pa_rope_store_int8(s["dims"], s["rope"], s["q"], s["kn"], s["vn"], s["positions"], s["slots"], s["q_out"],
                                  s["k"], s["v"], s["ks"], s["vs"])
        else:
            pa.pa_rope_store(s["dims"], s["rope"], s["q"], s["kn"], s["vn"], s["positions"], s["slots"], s["q_out"],
                             s["k"], s["v"])
    elif op == "prefill":
        if int8:
            pa.pa_prefill_window_int8(s["dims"], s["q"], s["k"], s["v"], s["ks"], s["vs"], s["plan"], c["window"],
                                      c["sinks"], s["scale"], s["out"], s["ws"])
        else:
            pa.pa_prefill_window(s["dims"], s["q"], s["k"], s["v"], s["plan"], c["window"], c["sinks"], s["scale"],
                                 s["out"])
    elif op == "window":
        if int8:
            pa.pa_decode_window_int8(s["dims"], s["q"], s["k"], s["v"], s["ks"], s["vs"], s["table"], s["ctx"],
                                     c["window"], c["sinks"], s["scale"], s["out"])
        else:
            pa.pa_decode_window(s["dims"], s["q"], s["k"], s["v"], s["table"], s["ctx"], c["window"], c["sinks"],
                                s["scale"], s["out"])
    elif op == "weights":
        if int8:
            pa.pa_decode_weights_int8(s["dims"], s["q"], s["k"], s["v"], s["ks"], s["vs"], s["table"], s["ctx"],
                                      s["scale"], s["out"], s["scores"], s["ws"], decay=c["decay"],
                                      scores_out=s["scores_out"])
        else:
            pa.pa_decode_weights(s["dims"], s["q"], s["k"], s["v"], s["table"], s["ctx"], s["scale"], s["out"],
                                 s["scores"], s["ws"], decay=c["decay"], scores_out=s["scores_out"])
    else:
        pa.pa_pool_evict(s["dims"], s["pool"], s["rows"], s["scores"], c["budget"], s["kept"], first=c["first"],
                         last=c["last"], scores_out=s["scores_out"])
    return _outputs(s)


def _outputs(s):
    op = s["c"]["op"]
    names = {"rope": ("q_out", "k", "v"), "weights": ("out", "scores_out"),
             "evict": ("kept", "table", "ctx", "refs", "scores_out", "k", "v")}.get(op, ("out",))
    got = {n: s[n] for n in names}
    if op in ("rope", "evict") and "ks" in s:  # what is held in 8 bits, as the values it stands for
        got["k"] = s["k"] * s["ks"].transpose(-1, -2)[..., None]
        got["v"] = s["v"] * s["vs"].transpose(-1, -2)[..., None]
    return got


def _turn(x, w, s, c):
    """Norm and rotation of [tokens, heads, d], in 32 bits."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    half = c["rot"] // 2
    pair = torch.arange(half, device=DEV)
    axis = torch.as_tensor(s["pair_axis"], device=DEV)
    at = s["positions"].long()[axis].t() * (2 * half) + pair  # [tokens, pairs]
    cos, sin = s["cos_sin"].view(-1)[at][:, None], s["cos_sin"].view(-1)[at + half][:, None]
    a, b = (pair, pair + half) if c["pairs"] == "half" else (2 * pair, 2 * pair + 1)
    y = x.clone()
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _quantise(x):
    """(codes, fp16 scales) of rows: max|x| / 127, halves away from zero."""
    scale = (x.abs().amax(-1) / 127).clamp_min(1e-8)
    q = x / scale[..., None]
    return torch.trunc(q + torch.where(q >= 0, 0.5, -0.5)).to(torch.int8), scale.to(torch.float16)


def _plain_rope(s):
    c = s["c"]
    bs, at = c["bs"], s["slots"][:c["tokens"]].long()
    s["q_out"] = _turn(s["q"], s["qw"], s, c).to(torch.bfloat16)
    k = _turn(s["kn"], s["kw"], s, c)[:c["tokens"]]
    v = s["vn"][:c["tokens"]]
    for name, x in (("k", k), ("v", v)):
        if c["kind"] == "bf16":
            s[name].flatten(0, 1)[at] = x.to(torch.bfloat16)
        else:
            codes, scale = _quantise(x.float())
            s[name].flatten(0, 1)[at] = codes
            s[name + "s"][at // bs, :, at % bs] = scale


def _pages(s):
    """Keys and values of each row of the table, [rows, hkv, tokens, d] in 32 bits; a page that is not there is zeros."""
    page = s["table"].clamp_min(0).long()
    gone = (s["table"] < 0)[:, :, None, None, None]
    got = []
    for name in ("k", "v"):
        x = s[name][page].float()
        if "ks" in s:
            x = x * s[name + "s"][page].transpose(-1, -2)[..., None].float()
            if s["c"]["op"] == "prefill":  # a prompt reads the INT8 cache as bf16 values
                x = x.to(torch.bfloat16).float()
        x = x.masked_fill(gone, 0)
        got.append(x.reshape(page.shape[0], -1, *x.shape[3:]).transpose(1, 2))
    return got


def _softmax(sc, seen):
    sc = torch.where(seen, sc, torch.full_like(sc, -math.inf))
    p = torch.exp(sc - sc.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _plain_prefill(s):
    c = s["c"]
    k, v = _pages(s)
    n, most, hq, hkv, d = s["new"].numel(), k.shape[2], c["hq"], c["hkv"], c["d"]
    new, ctx, first = s["new"].long(), s["ctx"].long(), s["first"].long()
    i = torch.arange(_prefill_most(c), device=DEV)
    live = i < new[:, None]
    row = torch.where(live, first[:-1, None] + i, 0)
    pos = (ctx - new)[:, None] + i  # [seqs, queries]
    key = torch.arange(most, device=DEV)
    seen = (key <= pos[..., None]) & ((key > pos[..., None] - c["window"]) | (key < c["sinks"]))
    seen |= ~live[..., None]  # rows of no query: anything finite
    q = s["q"].float()[row].view(n, -1, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    sc = torch.matmul(q.reshape(n, hkv, -1, d) * s["scale"], k.transpose(2, 3)).view(n, hkv, hq // hkv, -1, most)
    p = _softmax(sc, seen[:, None, None])
    o = torch.matmul(p.view(n, hkv, -1, most), v).view(n, hkv, hq // hkv, -1, d)
    s["out"] = o.permute(0, 3, 1, 2, 4).reshape(n, -1, hq, d)[live].to(torch.bfloat16)


def _prefill_most(c):
    return max(_prefill_lens(c)[0])


def _plain_decode(s):
    c = s["c"]
    n, hq, hkv, d, bs = s["ctx"].numel(), c["hq"], c["hkv"], c["d"], c["bs"]
    ctx, width = s["ctx"].long(), s["table"].shape[1] * bs
    if c["op"] == "window":  # the keys that are seen, and no others
        lo = (ctx - c["window"]).clamp_min(0)
        most = min(c["window"] + c["sinks"], width)
        i = torch.arange(most, device=DEV)
        sink = torch.minimum(lo, torch.full_like(lo, c["sinks"]))[:, None]
        key = torch.where(i < sink, i, lo[:, None] + i - sink)
    else:
        key = torch.arange(width, device=DEV).expand(n, -1)
    seen = key < ctx[:, None]
    key = torch.where(seen, key, 0)
    page = torch.gather(s["table"].clamp_min(0).long(), 1, key // bs)
    kv = []
    for name in ("k", "v"):
        x = s[name][page, key % bs].float()  # [n, keys, hkv, d]
        if "ks" in s:
            x = x * s[name + "s"][page, :, key % bs][..., None].float()
        kv.append(x.transpose(1, 2))
    sc = torch.matmul(s["q"].float().view(n, hkv, -1, d) * s["scale"], kv[0].transpose(2, 3))
    p = _softmax(sc, seen[:, None, None])
    s["out"] = torch.matmul(p, kv[1]).view(n, hq, d).to(torch.bfloat16)
    if c["op"] == "weights":
        old = s["scores"] * c["decay"] if c["decay"] else torch.zeros_like(s["scores"])
        s["scores_out"] = torch.where(seen[:, None], old + p.sum(2), s["scores_out"])


def _plain_evict(s):
    c, bs = s["c"], s["c"]["bs"]
    rows, budget = s["rows"].long(), c["budget"]
    ctx = s["ctx"][rows].long()
    width = s["table"].shape[1] * bs
    key = torch.arange(width, device=DEV)
    total = s["scores"][rows].double().sum(1).float()
    total = torch.where((key < c["first"]) | (key >= ctx[:, None] - c["last"]), math.inf, total)
    total = torch.where(key < ctx[:, None], total, -math.inf)
    # of equal ones the lowest index
    got = torch.sort(total, dim=1, descending=True, stable=True).indices[:, :budget]
    got = torch.sort(torch.where(torch.arange(budget, device=DEV) < ctx[:, None], got, width), 1).values
    live = got < width
    s["kept"] = torch.where(live, got, -1).to(torch.int32)
    left = torch.minimum(ctx, torch.full_like(ctx, budget))
    at = got.clamp_max(width - 1)
    # scores
    moved = torch.gather(s["scores"][rows], 2, at[:, None].expand(-1, c["hkv"], -1))
    fresh = torch.zeros((rows.numel(), c["hkv"], width), device=DEV)
    fresh[:, :, :budget] = torch.where(live[:, None], moved, 0)
    s["scores_out"][rows] = torch.where(key < ctx[:, None, None], fresh, s["scores_out"][rows])
    # pages
    table = s["table"][rows].long()
    src = torch.gather(table, 1, at // bs) * bs + at % bs
    j = torch.arange(budget, device=DEV).expand_as(at)
    dst = torch.gather(table, 1, j // bs) * bs + j % bs
    src, dst = src[live], dst[live]
    for name in ("k", "v"):
        x = s[name].flatten(1, 2)
        x[:, dst] = x[:, src]
        if name + "s" in s:
            y = s[name + "s"]
            y[:, dst // bs, :, dst % bs] = y[:, src // bs, :, src % bs]
    gone = torch.arange(table.shape[1], device=DEV) * bs >= left[:, None]
    page = table[gone & (table >= 0)]
    s["refs"].index_add_(0, page, torch.full_like(page, -1, dtype=torch.int32))
    s["table"][rows] = torch.where(gone, -1, table).to(torch.int32)
    s["ctx"][rows] = left.to(torch.int32)


# ---------------------------------------------------------------- exact values

def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "rope":
        return _exact_rope(s, c)
    if c["op"] == "evict":
        return _exact_evict(s, c)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    bs, group = c["bs"], c["hq"] // c["hkv"]
    new = s["new"].tolist() if c["op"] == "prefill" else [1] * s["ctx"].numel()
    got = {"out": out}
    if c["op"] == "weights":
        got["scores_out"] = torch.zeros(s["scores"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for b, (n, x) in enumerate(zip(new, s["ctx"].tolist())):
        pages = s["table"][b, :-(-x // bs)].long()
        there = (pages >= 0).repeat_interleave(bs)[:x]
        kv = []
        for name in ("k", "v"):
            t = s[name][pages.clamp_min(0)].double()
            if "ks" in s:
                t = t * s[name + "s"][pages.clamp_min(0)].double().permute(0, 2, 1)[..., None]
                if c["op"] == "prefill":
                    t = t.to(torch.bfloat16).double()
            kv.append(t.flatten(0, 1)[:x])
        j = torch.arange(x, device=DEV)
        for i0 in range(0, n, 512):
            i = torch.arange(i0, min(n, i0 + 512), device=DEV)
            pos = (x - n + i)[:, None]
            mask = j <= pos
            if c["op"] != "weights":
                mask &= (pos - j < c["window"]) | (j < c["sinks"])
            cols = torch.nonzero(mask.any(0) & there)[:, 0]
            q = s["q"][at + i].double().view(len(i), c["hkv"], group, c["d"])
            sc = torch.einsum("ihgd,jhd->hgij", q, kv[0][cols]) * s["scale"]
            p = torch.softmax(sc.masked_fill(~mask[:, cols], -math.inf), -1)
            out[at + i] = torch.einsum("hgij,jhd->ihgd", p, kv[1][cols]).reshape(len(i), c["hq"], c["d"])
            if c["op"] == "weights":
                got["scores_out"][b, :, :x] = p[:, :, 0].sum(1) + c["decay"] * s["scores"][b, :, :x].double()
        at += n
    return got


def _exact_rope(s, c):
    half, n = c["rot"] // 2, c["tokens"]
    axis = torch.as_tensor(s["pair_axis"], device=DEV).tolist()
    pos = s["positions"].long()
    cos = torch.stack([s["cos_sin"][pos[a], i] for i, a in enumerate(axis)], 1).double()[:, None]
    sin = torch.stack([s["cos_sin"][pos[a], half + i] for i, a in enumerate(axis)], 1).double()[:, None]

    def turned(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["d"] + 1e-6) * w.double()
        z = x[..., :2 * half]
        z = torch.stack(z.split(half, -1), -1) if c["pairs"] == "half" else z.unflatten(-1, (half, 2))
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * torch.complex(cos, sin))
        z = torch.cat(z.unbind(-1), -1) if c["pairs"] == "half" else z.flatten(-2)
        return torch.cat([z, x[..., 2 * half:]], -1)

    got = {"q_out": turned(s["q"], s["qw"])}
    for name, x in (("k", turned(s["kn"], s["kw"])), ("v", s["vn"].double())):
        cache = torch.zeros(s[name].shape, dtype=torch.float64, device=DEV)
        x = x[:n]
        if c["kind"] == "int8":
            step = x.abs().amax(-1, keepdim=True) / 127
            code = torch.floor(x.abs() / step + 0.5) * torch.sign(x)
            x = code * step.to(torch.float16).double()
        cache.flatten(0, 1)[s["slots"][:n].long()] = x
        got[name] = cache
    return got


def _exact_evict(s, c):
    bs, budget = c["bs"], c["budget"]
    table, ctx, refs = s["table"].cpu().numpy().copy(), s["ctx"].cpu().numpy().copy(), s["refs"].cpu().numpy().copy()
    kept = np.full((c["rows"], budget), -1, np.int32)
    scores = s["scores"].cpu().numpy()
    out = np.zeros(scores.shape, np.float64)
    for i, row in enumerate(s["rows"].tolist()):
        n = int(ctx[row])
        if n > budget:
            total = scores[row, :, :n].astype(np.float64).sum(0).astype(np.float32)
            middle = np.arange(c["first"], n - c["last"])
            best = middle[np.lexsort((middle, -total[middle]))][:budget - c["first"] - c["last"]]
            keep = np.sort(np.concatenate([np.arange(c["first"]), best, np.arange(n - c["last"], n)]))
        else:
            keep = np.arange(n)
        kept[i, :len(keep)] = keep
        out[row, :, :len(keep)] = scores[row][:, keep]
        for p in range(-(-len(keep) // bs), -(-n // bs)):
            refs[table[row, p]] -= 1
            table[row, p] = -1
        ctx[row] = len(keep)
    # the pages move once; a pass on rows that were set back moves them again
    return {"kept": _i32(kept), "table": _i32(table), "ctx": _i32(ctx), "refs": _i32(refs),
            "scores_out": torch.tensor(out, device=DEV), "k": None, "v": None}
