"""Attention over a bounded cache in 64 bits on the CPU, from the formulas, and cases to run it on."""
import numpy as np
import torch

from paged_kv_cache_kvcache_gb300 import pagedattn as pa


def seen(n, pos, window, sinks):
    """Which of n keys a query at a position sees."""
    j = np.arange(n)
    return (j <= pos) & ((pos - j < window) | (j < sinks))


def attend(q, k, v, mask, scale):
    """(out, sum of w |v|, w) for q [hq, d] over k, v [n, hkv, d] where mask [n]; float64."""
    hkv = k.shape[1]
    g = q.shape[0] // hkv
    out, size, w = np.zeros(q.shape), np.zeros(q.shape), np.zeros((q.shape[0], k.shape[0]))
    at = np.flatnonzero(mask)
    if len(at):
        for h in range(q.shape[0]):
            s = k[at, h // g] @ q[h] * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            w[h, at] = p
            out[h], size[h] = p @ v[at, h // g], p @ np.abs(v[at, h // g])
    return out, size, w


class Case:
    """Rows of a block table and a cache whose unseen places hold NaN (INT8: NaN scales)."""

    def __init__(self, lens, hq, hkv, d, bs, window, sinks, int8, seed=0, first_new=None):
        r = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.lens, self.window, self.sinks, self.int8 = list(lens), window, sinks, int8
        self.hq, self.hkv, self.d, self.bs, self.scale = hq, hkv, d, bs, 1.3 * d ** -0.5
        rows, self.width = len(lens), max(1, max(-(-n // bs) for n in lens)) + 1
        self.blocks = sum(-(-n // bs) for n in lens) + 2
        table = np.full((rows, self.width), -7, np.int32)  # behind a row, and pages given back: not ids
        slots, ids = [], r.permutation(self.blocks)
        at = 0
        self.visible = []
        for b, n in enumerate(lens):
            pages = -(-n // bs)
            # positions that some query of the call is at: the last only, or all from first_new on
            first = n - 1 if first_new is None else first_new[b]
            vis = np.zeros(n, bool)
            for pos in {first, n - 1}:
                vis |= seen(n, pos, window, sinks) if n else False
            if n and first < n - 1:
                vis |= (np.arange(n) > first - window) & (np.arange(n) < n)
            row = ids[at:at + pages]
            for p in range(pages):
                if vis[p * bs:(p + 1) * bs].any():
                    table[b, p] = row[p]
            slots.append(np.concatenate([row[:, None] * bs + np.arange(bs)]).reshape(-1)[:n] if pages else
                         np.zeros(0, int))
            self.visible.append(vis)
            at += pages
        self.table, self.slots = table, slots
        shape = (self.blocks * bs, hkv, d)
        self.k, self.v = (torch.randn(shape, generator=g).to(torch.bfloat16) for _ in range(2))
        live = np.zeros(self.blocks * bs, bool)
        for s, vis in zip(slots, self.visible):
            live[s[vis]] = True
        self.live = torch.as_tensor(live)
        page = (self.blocks, bs, hkv, d)
        self.dims = pa.make_dims(self.blocks, bs, hq, hkv, d)
        if int8:
            x = [t.float() for t in (self.k, self.v)]
            self.scales = [(t.abs().amax(-1) / 127).to(torch.float16) for t in x]
            codes = [torch.round(t / s.float()[..., None]).clamp(-127, 127).to(torch.int8) for t, s in zip(x, self.scales)]
            self.kd, self.vd = ((c.double() * s.double()[..., None]).numpy() for c, s in zip(codes, self.scales))
            for s in self.scales:
                s[~self.live] = float("nan")
            self.gpu = [c.view(page).cuda() for c in codes] + \
                [s.view(self.blocks, bs, hkv).transpose(1, 2).contiguous().cuda() for s in self.scales]
        else:
            self.kd, self.vd = self.k.double().numpy(), self.v.double().numpy()
            bad = [t.clone() for t in (self.k, self.v)]
            for t in bad:
                t[~self.live] = float("nan")
                t[~self.live, :, ::3] = float("inf")
            self.gpu = [t.view(page).cuda() for t in bad]
        self.bt = torch.as_tensor(table).cuda()
        self.ctx = torch.tensor(self.lens, dtype=torch.int32).cuda()

    def fine(self, w, slots):
        """What an INT8 cache's fp16 weights P v_scale (P relative to the largest) add to an error where they are below
        fp16's normal numbers, 2^-14: half its smallest step, 2^-25, or at most the weight itself, times a code of up to
        127, over sum P = 1 / max w."""
        top = w.max(-1, keepdims=True, initial=0) + 1e-300
        vs = self.scales[1].double().nan_to_num().numpy()[slots].T.repeat(self.hq // self.hkv, 0)  # [hq, n]
        p = w / top * vs
        return 127 * (np.where(p < 2.0 ** -14, np.minimum(p, 2.0 ** -25), 0).sum(-1, keepdims=True) * top)

    def decode(self, q):
        """(out, size, weights summed over each KV head's heads, per row [hkv, n]) of one query per row."""
        got = [attend(x, self.kd[s], self.vd[s], seen(n, n - 1, self.window, self.sinks), self.scale)
               for x, s, n in zip(q.double().numpy(), self.slots, self.lens)]
        g = self.hq // self.hkv
        if self.int8:
            got = [(o, size + 2.0 ** 8 * self.fine(w, s), w) for (o, size, w), s in zip(got, self.slots)]
        return (np.stack([x[0] for x in got]), np.stack([x[1] for x in got]),
                [x[2].reshape(self.hkv, g, -1).sum(1) for x in got])


def near(got, want, size):
    """A bf16 result is off by half a step (2^-8), its weights' rounding by 2^-8 of sum w |v|, and what fp32 does
    before that by under 2e-4 of it (scores of a few hundred products, exponents, sums)."""
    got = got.double().cpu().numpy()
    err = np.abs(got - want)
    assert (err <= 2.0 ** -8 * (size + np.abs(want)) + 2e-4 * size + 1e-30).all(), float(np.nanmax(err))
