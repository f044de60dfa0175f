"""Decodes over an INT8 cache where a few first keys outweigh the others by far and values are of any size.

The others' weights are then small against the largest, and many of them together still move the result."""
import numpy as np
import pytest
import torch

from paged_kv_cache_kvcache_gb300 import pagedattn as pa
from tests.bounded_model import attend, near

pytestmark = pytest.mark.gpu

BS = 16


class Rows:
    """Sequences of one length that read the same pages: n keys, of which every 16th of the first `high * 16` scores `gap`
    above the others; values of size[j] around half of it."""

    def __init__(self, seqs, hq, hkv, d, n, gap, size, high=16, seed=0):
        r = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.n, self.seqs, self.scale = n, seqs, d ** -0.5
        k = 0.2 * torch.randn(n, hkv, d, generator=g)
        k[:, :, 0] = 0
        k[0:16 * high:16, :, 0] = gap / (8 * self.scale)
        v = torch.as_tensor(size, dtype=torch.float32).view(n, 1, 1) * (0.5 + 0.1 * torch.randn(n, hkv, d, generator=g))
        v[0:16 * high:16] *= -1
        self.q = torch.randn(4, hq, d, generator=g).to(torch.bfloat16)
        self.q[:, :, 0] = 8
        pages = -(-n // BS)
        self.blocks = pages + 3
        ids = r.permutation(self.blocks)[:pages]
        slots = (ids[:, None] * BS + np.arange(BS)).reshape(-1)[:n]
        self.dims = pa.make_dims(self.blocks, BS, hq, hkv, d)
        self.gpu, scales, self.exact = [], [], []
        for x in (k, v):
            s = (x.abs().amax(-1) / 127).to(torch.float16)
            c = torch.where(s[..., None] > 0, torch.round(x / s.float()[..., None]), 0.0).clamp(-127, 127)
            self.exact.append((c.double() * s.double()[..., None]).numpy())
            codes = torch.zeros(self.blocks * BS, hkv, d, dtype=torch.int8)
            codes[slots] = c.to(torch.int8)
            sc = torch.full((self.blocks * BS, hkv), float("nan"), dtype=torch.float16)
            sc[slots] = s
            self.gpu.append(codes.view(self.blocks, BS, hkv, d).cuda())
            scales.append(sc.view(self.blocks, BS, hkv).transpose(1, 2).contiguous().cuda())
        self.gpu += scales
        self.ids = ids
        self.table = torch.tensor(np.tile(ids.astype(np.int32), (seqs, 1)), device="cuda")
        self.ctx = torch.full((seqs,), n, dtype=torch.int32, device="cuda")
        self.q_gpu = self.q[torch.arange(seqs) % 4].cuda()
        got = [attend(x, *self.exact, np.ones(n, bool), self.scale) for x in self.q.double().numpy()]
        self.want, self.size, self.w = (np.stack([x[i] for x in got]) for i in range(3))

    def check(self, out):
        """fp16 products P v_scale of 11 bits (2^-11), within what near() allows the weights (2^-8)."""
        pick = np.arange(self.seqs) % 4
        near(out, self.want[pick], self.size[pick])


# sequences, heads, keys, how far the first keys stand out, size of the values
CASES = [
    (40, (16, 8, 128), 8192, 8.5, 0.02),
    (160, (28, 4, 128), 4096, 8.0, 0.1),
    (160, (28, 4, 128), 1024, 7.0, 0.01),
    (3, (4, 2, 64), 32000, 10.0, 0.02),
    (1, (16, 1, 128), 32000, 10.0, 0.1),
    (8, (12, 1, 64), 16000, 9.0, 0.002),
    (6, (8, 8, 128), 900, 3.0, 1e-4),
    (6, (8, 8, 128), 900, 3.0, 3e5),
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: f"{c[0]}x{c[2]}-{c[3]}-{c[4]}")
@pytest.mark.parametrize("call", ["window", "weights", "plan"])
def test_small_weights_count(c, call):
    seqs, heads, n, gap, size = c
    decode(Rows(seqs, *heads, n, gap, np.full(n, size)), call)


def decode(x, call):
    out = torch.empty_like(x.q_gpu)
    if call == "window":
        pa.pa_decode_window_int8(x.dims, x.q_gpu, *x.gpu, x.table, x.ctx, 2 ** 31 - 1, 0, x.scale, out)
    elif call == "weights":
        scores = torch.zeros(x.seqs, x.dims.num_kv_heads, x.table.shape[1] * BS, device="cuda")
        pa.pa_decode_weights_int8(x.dims, x.q_gpu, *x.gpu, x.table, x.ctx, x.scale, out, scores,
                                  pa.weights_workspace(x.dims, x.seqs, x.table.shape[1]))
        group = x.q.shape[1] // x.dims.num_kv_heads
        want = x.w.reshape(4, x.dims.num_kv_heads, group, -1).sum(2)[np.arange(x.seqs) % 4]
        got = scores[:, :, :x.n].double().cpu().numpy()
        assert (np.abs(got - want) <= 2e-4 * want + 1e-30).all()
    else:
        plan = pa.pa_pack_decode(x.dims, [x.n] * x.seqs, [list(x.ids)] * x.seqs).upload()
        ws = torch.empty(max(256, plan.meta.workspace_bytes), dtype=torch.uint8, device="cuda")
        pa.pa_decode_int8(x.dims, x.q_gpu, *x.gpu, plan, x.scale, out, ws)
    x.check(out)


SIZES = {  # of the values along the context
    "rising": lambda n: 10.0 ** np.linspace(-4, 5, n),
    "falling": lambda n: 10.0 ** np.linspace(5, -4, n),
    "mixed": lambda n: 10.0 ** np.random.default_rng(3).uniform(-3, 3, n),
    "zeros first": lambda n: np.where(np.arange(n) < n // 2, 0.0, 0.3),
    "zeros last": lambda n: np.where(np.arange(n) >= n // 2, 0.0, 0.3),
    "zeros": lambda n: np.zeros(n),
    "largest": lambda n: np.full(n, 4e6),
}


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("call", ["window", "weights", "plan"])
def test_values_of_different_sizes(size, call):
    decode(Rows(5, 28, 4, 128, 2001, 2.0, SIZES[size](2001), high=2), call)
