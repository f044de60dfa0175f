"""Windows in which every key counts for itself: one that is left out, or seen too many, shows however long the window is.

Queries are 0, so that every key that is seen weighs the same and the softmax's sums are whole numbers, exactly.  Key j's
value is 1 in component (j + head) mod D and 0 in the others, unseen keys' too: an output component is the share of the keys
that fall on it, rounded to bf16 (2^-8 of itself; the reciprocal 2^-22), and one key more or less moves it by over 2^-7 of
itself while fewer than 127 of those seen share a component."""
import numpy as np
import pytest
import torch

from paged_kv_cache_kvcache_gb300 import pagedattn as pa

pytestmark = pytest.mark.gpu


class Keys:
    """n keys of random scores-to-be and their values, in pages in random order, bf16 or INT8."""

    def __init__(self, n, hkv, d, bs, int8, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.n, self.hkv, self.d, self.bs, self.int8, pages = n, hkv, d, bs, int8, -(-n // bs)
        self.blocks = pages + 2
        self.ids = np.random.default_rng(seed).permutation(self.blocks)[:pages].astype(np.int32)
        slots = torch.as_tensor((self.ids[:, None].astype(np.int64) * bs + np.arange(bs)).reshape(-1)[:n], device="cuda")
        j = torch.arange(n, device="cuda")
        v = torch.zeros(self.blocks * bs, hkv, d, device="cuda")
        for h in range(hkv):
            v[slots, h, (j + h) % d] = 1
        shape = (self.blocks, bs, hkv, d)
        if int8:
            k = torch.randint(-127, 128, shape, dtype=torch.int8, device="cuda", generator=g)
            scale = torch.full((self.blocks, hkv, bs), 2.0 ** -6, dtype=torch.float16, device="cuda")
            self.cache = [k, (64 * v).to(torch.int8).view(shape), scale, scale.clone()]
        else:
            self.cache = [torch.randn(shape, device="cuda", generator=g).to(torch.bfloat16), v.to(torch.bfloat16).view(shape)]
        # ones[j][h][x]: keys before j whose value is in component x of head h
        hot = np.zeros((n + 1, hkv, d), np.int32)
        for h in range(hkv):
            hot[1 + np.arange(n), h, (np.arange(n) + h) % d] = 1
        self.ones = np.cumsum(hot, 0)

    def shares(self, pos, window, sinks):
        """[queries, hkv, d] of queries at these positions."""
        pos = np.asarray(pos)
        lo = np.maximum(0, pos + 1 - window)
        seen = self.ones[pos + 1] - self.ones[lo] + self.ones[np.minimum(sinks, lo)]
        return seen / seen.sum(-1, keepdims=True)

    def check(self, out, want):
        got = out.double().cpu().numpy().reshape(*want.shape[:2], -1, self.d)
        want = want[:, :, None]
        assert (np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -20) * want).all(), float(np.abs(got - want).max())


# lengths, window, sinks, heads, block size: with as many (sequence, KV head)s as take one CTA each, a warp has up to 67
# chunks of 16 keys; with few, clusters of up to 16 CTAs share them
DECODE = [
    ([5000, 4321, 4999, 1, 4270, 33] * 30, 4200, 70, (8, 4, 128), 16),
    ([6001, 5007, 2100, 4095] * 48, 5100, 3, (4, 4, 64), 64),
    ([3333, 2222, 1111] * 40, 2500, 17, (28, 4, 128), 256),
    ([15000, 14001], 13000, 40, (16, 1, 128), 16),
    ([7777] * 6, 7000, 0, (12, 1, 64), 32),
    ([4096, 4097, 4111, 4112], 2 ** 31 - 1, 0, (8, 8, 64), 16),
    ([1200, 1201, 1215, 1216, 1217] * 20, 513, 31, (7, 1, 128), 1024),
]


@pytest.mark.parametrize("int8", [False, True], ids=["bf16", "int8"])
@pytest.mark.parametrize("c", range(len(DECODE)))
def test_decode(c, int8):
    lens, window, sinks, (hq, hkv, d), bs = DECODE[c]
    x = Keys(max(lens), hkv, d, bs, int8, seed=c)
    dims = pa.make_dims(x.blocks, bs, hq, hkv, d)
    table = torch.as_tensor(np.tile(x.ids, (len(lens), 1)), device="cuda")
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.zeros(len(lens), hq, d, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 9)
    call = pa.pa_decode_window_int8 if int8 else pa.pa_decode_window
    call(dims, q, *x.cache, table, ctx, window, sinks, d ** -0.5, out)
    x.check(out, x.shares(np.array(lens) - 1, window, sinks))
    # the same keys seen whole, with weights: each 1 / n, times the group
    out.fill_(9)
    scores = torch.zeros(len(lens), hkv, len(x.ids) * bs, device="cuda")
    call = pa.pa_decode_weights_int8 if int8 else pa.pa_decode_weights
    call(dims, q, *x.cache, table, ctx, d ** -0.5, out, scores, pa.weights_workspace(dims, len(lens), len(x.ids)))
    x.check(out, x.shares(np.array(lens) - 1, max(lens), 0))
    want = (torch.arange(scores.shape[2], device="cuda") < ctx[:, None]) * (hq // hkv / ctx[:, None].double())
    assert ((scores.double() - want[:, None]).abs() <= 2.0 ** -20 * want[:, None]).all()


PREFILL = [  # (length, new) of each sequence
    ([(6000, 2500), (4000, 1000), (33, 33), (5001, 1)], 4200, 70, (16, 2, 128), 16),
    ([(2000, 2000)] * 3, 777, 5, (8, 8, 64), 32),
    ([(1500, 300)] * 40, 1023, 18, (28, 4, 128), 64),
    ([(700, 700), (129, 129), (128, 1)], 1, 0, (7, 1, 128), 16),
    ([(900, 900)] * 2, 300, 400, (4, 2, 64), 256),
]


@pytest.mark.parametrize("int8", [False, True], ids=["bf16", "int8"])
@pytest.mark.parametrize("c", range(len(PREFILL)))
def test_prefill(c, int8):
    seqs, window, sinks, (hq, hkv, d), bs = PREFILL[c]
    lens, new = [list(t) for t in zip(*seqs)]
    x = Keys(max(lens), hkv, d, bs, int8, seed=c)
    dims = pa.make_dims(x.blocks, bs, hq, hkv, d)
    plan = pa.pa_pack_prefill(dims, lens, new, [list(x.ids[:-(-n // bs)]) for n in lens]).upload()
    q = torch.zeros(sum(new), hq, d, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 9)
    if int8:
        pa.pa_prefill_window_int8(dims, q, *x.cache, plan, window, sinks, d ** -0.5, out, pa.prefill_workspace(plan))
    else:
        pa.pa_prefill_window(dims, q, *x.cache, plan, window, sinks, d ** -0.5, out)
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)])
    x.check(out, x.shares(pos, window, sinks))
