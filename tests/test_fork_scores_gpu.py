"""A forked row and its scores: copied from the parent's by the caller, kept up by both rows' decodes, read by an eviction."""
import numpy as np
import pytest
import torch

from paged_kv_cache_kvcache_gb300 import pagedattn as pa
from tests import evict_model
from tests.bounded_model import attend
from tests.test_pool_gpu import append, assert_same, both, host, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_a_forked_row_goes_on_with_its_parents_scores(kind):
    int8, hkv, group, d, bs, width = kind == "int8", 2, 2, 64, 16, 8
    hq, parent, child, other = hkv * group, 2, 0, 3
    dims, pool, model = both(kind, 1, 40, bs, hkv, d, 4, width, seed=3)
    qdims = pa.make_dims(40, bs, hq, hkv, d)
    caches = [x[0] if x.dim() == 5 or (x.dim() == 4 and x.dtype == torch.float16) else x
              for x in (pool.k_cache, pool.v_cache, pool.k_scale, pool.v_scale) if x is not None]
    if int8:
        for x in caches[2:]:
            x.fill_(0.01)
        model.scales = [host(x) for x in (pool.k_scale, pool.v_scale)]  # (as the pool's, 16 bits each)
    scores = torch.zeros(4, hkv, width * bs, device="cuda")
    ws = pa.weights_workspace(qdims, 4, width)
    g = torch.Generator().manual_seed(2)
    scale = d ** -0.5
    want = np.zeros(scores.shape)

    def step(rows):
        """A token of its own for each row, and a decode with weights; the model's scores in 64 bits."""
        append(dims, pool, model, rows, [1] * len(rows))
        q = torch.randn(len(rows), hq, d, generator=g).to(torch.bfloat16)
        out = torch.empty_like(q, device="cuda")
        call = pa.pa_decode_weights_int8 if int8 else pa.pa_decode_weights
        call(qdims, q.cuda(), *caches, pool.block_tables, pool.context_lens, scale, out, scores, ws, table_rows=i32(rows))
        kv = [x.double().cpu().numpy().reshape(-1, hkv, d) for x in caches[:2]]
        if int8:
            kv = [x * s.double().cpu().numpy().transpose(0, 2, 1).reshape(-1, hkv)[..., None] for x, s in zip(kv, caches[2:])]
        for b, r in enumerate(rows):
            n = int(model.ctx[r])
            at = model.tables[r, np.arange(n) // bs] * bs + np.arange(n) % bs
            w = attend(q[b].double().numpy(), kv[0][at], kv[1][at], np.ones(n, bool), scale)[2]
            want[r, :, :n] += w.reshape(hkv, group, n).sum(1)

    append(dims, pool, model, [parent, child], [40, 90])
    step([parent, child])
    step([parent, child])
    # the child's row held another sequence, whose scores go with it
    pa.pa_pool_free(dims, pool, i32([child]))
    model.free([child])
    pa.pa_pool_fork(dims, pool, i32([parent]), i32([child]))
    assert model.fork([parent], [child])
    assert_same(pool, model)
    n = int(model.ctx[parent])
    scores[child] = 0
    scores[child, :, :n] = scores[parent, :, :n]
    want[child] = 0
    want[child, :, :n] = want[parent, :, :n]
    for _ in range(6):
        step([child, parent])
    got = scores.double().cpu().numpy()
    assert (np.abs(got - want) <= 1e-4 * want + 1e-30).all() and not got[other].any()
    # the child shrinks behind the pages that it shares with its parent
    before, budget, first = scores.cpu().numpy(), 40, 32
    kept = torch.empty(1, budget, dtype=torch.int32, device="cuda")
    pa.pa_pool_evict(dims, pool, i32([child]), scores, budget, kept, first=first, last=3)
    torch.cuda.synchronize()
    places, after = evict_model.evict(model, [child], before, budget, first, 3)
    assert kept.tolist() == places.tolist() and np.array_equal(scores.cpu().numpy(), after)
    assert_same(pool, model)
    # without the pages of its own the eviction would write into the parent's: refused
    pa.pa_pool_evict(dims, pool, i32([child]), scores, 20, kept[:, :20].contiguous())
    assert pa.pa_read_device_error() == 1 << 8
    assert_same(pool, model)
