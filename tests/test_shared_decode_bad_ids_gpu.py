"""INT8 shared decode with block ids outside the pool while page 0 belongs to nobody and its scales are NaN or
infinite: what is outside reads as zeros, whichever launch reads it."""
import numpy as np
import pytest
import torch

from paged_kv_cache_kvcache_gb300 import pagedattn as pa
from tests.test_shared_decode_gpu import assert_within, decode8, int8_pool, reference, values
from tests.test_shared_pack import make_batch

pytestmark = pytest.mark.gpu

SHAPES = [  # sequences, shared blocks, tails, split, meta.direct, meta.apart
    (2, 8, [20, 40], 0, 3, None),                              # decoded whole, eight warps each
    (60, 2, [1 + 5 * i % 90 for i in range(60)], 0, 3, None),  # decoded whole, four warps each
    (2, 8, [20, 40], 128, 0, 0),                               # every part through the converted copy
    (90, 30, [1 + 7 * i for i in range(90)], 128, 0, 1),       # single sequences' parts beside the others
]


@pytest.mark.parametrize("scale0", [float("nan"), float("inf")])
@pytest.mark.parametrize("shape", SHAPES, ids=["few", "many", "copied", "apart"])
@pytest.mark.parametrize("heads", [(4, 2, 64), (28, 4, 128), (16, 1, 128)], ids=str)
def test_ids_outside_the_pool_and_a_spoilt_page_0(shape, heads, scale0):
    n, sh, tails, split, direct, apart = shape
    bs, (hq, hkv, d) = 16, heads
    ctx, lists, groups, nb = make_batch(9, [n], [sh], tails, bs)
    lists, nb = [[int(x) + 1 for x in ids] for ids in lists], nb + 1  # nobody's page 0
    cache, dense = int8_pool(nb, bs, hkv, d, 90, ctx, lists)
    for s in cache[2:]:
        s[0] = scale0
    q = values((n, hq, d), 92)
    dims = pa.make_dims(nb, bs, hq, hkv, d)
    width = max(len(x) for x in lists)
    table = np.full((n, width), -1, np.int32)
    for b, x in enumerate(lists):
        table[b, :len(x)] = x
    table[:, 1] = -1                                           # a shared block, as a refused append leaves it
    own = [b for b in range(n) if len(lists[b]) > sh]
    for b, bad in zip(own[::max(1, len(own) // 7)], (nb, -1, 1 << 30, -(1 << 31), nb + 100) * 2):
        table[b, sh] = bad                                     # first blocks of their own
    plan = pa.pa_pack_decode_shared(dims, ctx, groups, shared_lens=[sh * bs], max_blocks=width, split_tokens=split).upload()
    if direct != plan.meta.direct or apart not in (None, plan.meta.apart):
        # (with few KV heads the same parts may all have lanes, and short contexts may be worth a cut)
        assert heads[1] < 4
    out = decode8(dims, q, cache, plan, d ** -0.5, block_tables=torch.tensor(table, device="cuda"))
    torch.cuda.synchronize()
    assert pa.pa_read_device_error() == 1 << 6
    kz, vz = (torch.cat([c, torch.zeros_like(c[:1])]) for c in dense)
    zeroed = [[x if 0 <= x < nb else nb for x in table[b, :len(lists[b])].tolist()] for b in range(n)]
    assert_within(out, *reference(q, kz, vz, zeroed, ctx, bs, d ** -0.5), f"bad ids {shape[:2]} {heads}")
