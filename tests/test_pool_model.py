"""CPU tests: the pool model keeps its own invariants, and the pa_pool calls refuse bad arguments on the host."""
import ctypes

import numpy as np
import pytest
import torch

from paged_kv_cache_kvcache_gb300 import pagedattn as pa
from tests.pool_model import PoolModel


def test_model_worked_example():
    """Pages of 4 tokens: a 6-token prompt, two forks of it, one more token each, one leaves, compaction."""
    kv = np.arange(10 * 4).reshape(1, 10, 4)
    m = PoolModel(5, 3, 10, 4, [kv.copy()])
    assert m.append([2], [6]) == [0, 1, 2, 3, 4, 5]
    assert m.fork([2, 2], [0, 4])
    assert m.tables[[0, 2, 4], :2].tolist() == [[0, 2], [0, 1], [0, 3]] and m.refs[:4].tolist() == [3, 1, 1, 1]
    assert m.pages[0][0, 2].tolist() == [4, 5, 10, 11] and m.pages[0][0, 3].tolist() == [4, 5, 14, 15]
    assert m.append([0, 4, 2], [1, 3, 0]) == [2 * 4 + 2, 3 * 4 + 2, 3 * 4 + 3, 4 * 4]
    m.check()
    m.free([2])
    assert m.refs[:5].tolist() == [2, 0, 1, 1, 1]
    assert m.compact()[:5].tolist() == [0, -1, 2, 3, 1]
    assert m.tables[4].tolist() == [0, 3, 1] and m.ctx[4] == 9
    m.check()
    assert m.append([1], [13]) is None and m.fork([0], [0]) is False and m.fork([0, 4], [2, 2]) is False
    assert m.append([0, 0], [1, 1]) is None and m.append([0], [-1]) is None


@pytest.mark.parametrize("seed", range(4))
def test_model_invariants(seed):
    rng = np.random.default_rng(seed)
    m = PoolModel(12, 6, 30, 4)
    for _ in range(200):
        op = rng.integers(4)
        rows = rng.permutation(12)[:rng.integers(1, 5)].tolist()
        if op == 0:
            m.append(rows, rng.integers(0, 9, len(rows)).tolist())
        elif op == 1:
            m.fork([int(rng.integers(12))] * len(rows), rows)
        elif op == 2:
            m.free(rows)
        else:
            m.compact()
            used = int((m.refs > 0).sum())
            assert (m.refs[:used] > 0).all()
        m.check()


def _pool(**change):
    p = pa.pa_pool(4, 8, 2, 0, 16, 16, 16, 16, 32, None, None, 64 << 10, 0)
    for k, v in change.items():
        setattr(p, k, v)
    return p


def test_pool_calls_reject_bad_args_without_touching_the_gpu():
    dims = pa.make_dims(32, 16, 4, 2, 64)      # a layer's K: 32 * 16 * 2 * 64 * 2 = 131072 bytes
    L, ref = pa.lib(), ctypes.byref
    n = ctypes.c_uint64(0)
    assert L.pa_pool_workspace(ref(dims), ref(_pool()), ref(n)) == pa.PA_OK and n.value >= 4 * (8 * 4 + 2 * 32)
    assert L.pa_pool_workspace(ref(dims), None, ref(n)) == pa.PA_ERR_INVALID_ARG
    ws = n.value
    ok = _pool(layer_stride=131072)

    append = lambda p=ok, rows=16, cu=16, k=2, slots=16, t=3, w=256, b=ws, d=dims: L.pa_pool_append(
        ref(d), ref(p) if p else None, rows, cu, k, slots, t, w, b, None)
    fork = lambda p=ok, a=16, c=16, k=2, w=256, b=ws, d=dims: L.pa_pool_fork(ref(d), ref(p), a, c, k, w, b, None)
    free = lambda p=ok, rows=16, k=2: L.pa_pool_free(ref(dims), ref(p), rows, k, None)
    compact = lambda p=ok, m=48, t=64, r=80, w=256, b=ws: L.pa_pool_compact(ref(dims), ref(p), m, t, r, w, b, None)

    assert append(k=0, t=0) == fork(k=0) == free(k=0) == pa.PA_OK          # nothing to do: no launch
    assert append(p=None) == pa.PA_ERR_INVALID_ARG
    for call in (append, fork, free, compact):
        for bad in (dict(num_rows=0), dict(max_blocks=0), dict(num_layers=0), dict(block_tables=None),
                    dict(context_lens=None), dict(ref_counts=None), dict(ref_counts=8), dict(block_tables=18)):
            assert call(p=_pool(layer_stride=131072, **bad)) == pa.PA_ERR_INVALID_ARG, bad
        assert call(p=_pool(num_rows=1 << 16, max_blocks=1 << 15)) == pa.PA_ERR_UNSUPPORTED
    for call in (append, fork, compact):
        assert call(b=ws - 1) == pa.PA_ERR_WORKSPACE
        assert call(w=None) == call(w=16) == pa.PA_ERR_INVALID_ARG
    for bad in (dict(k=5), dict(k=-1), dict(t=-1), dict(k=0), dict(rows=None), dict(cu=None), dict(slots=None)):
        assert append(**bad) == pa.PA_ERR_INVALID_ARG, bad
    for bad in (dict(k=5), dict(k=-1), dict(a=None), dict(c=None)):
        assert fork(**bad) == pa.PA_ERR_INVALID_ARG, bad
    assert free(k=-1) == free(rows=None) == pa.PA_ERR_INVALID_ARG
    for bad in (dict(m=None), dict(t=None), dict(r=None), dict(m=16), dict(m=80)):
        assert compact(**bad) == pa.PA_ERR_INVALID_ARG, bad
    for call in (fork, compact):
        for bad in (dict(k_cache=None), dict(v_cache=None), dict(k_cache=24), dict(k_scale=16), dict(layer_stride=131071),
                    dict(layer_stride=131056), dict(layer_stride=0), dict(k_scale=16, v_scale=16, scale_layer_stride=2046),
                    dict(k_scale=16, v_scale=16, scale_layer_stride=2049)):
            assert call(p=_pool(**{**dict(layer_stride=131072), **bad})) == pa.PA_ERR_INVALID_ARG, bad
    for call in (append, fork):
        assert call(d=pa.make_dims(0, 16, 4, 2, 64)) == pa.PA_ERR_INVALID_ARG
        assert call(d=pa.make_dims(32, 17, 4, 2, 64)) == pa.PA_ERR_UNSUPPORTED


def test_page_pool_checks_its_tensors():
    dims = pa.make_dims(6, 16, 2, 2, 64)
    k = torch.zeros(3, 6, 16, 2, 64, dtype=torch.bfloat16)
    pool = pa.page_pool(dims, k, k.clone(), 4, 5)
    assert pool.struct.num_layers == 3 and pool.struct.layer_stride == 6 * 16 * 2 * 64 * 2
    assert (pool.block_tables == -1).all() and pool.block_tables.shape == (4, 5)
    wide = torch.zeros(3, 7, 16, 2, 64, dtype=torch.bfloat16)[:, :6]     # layers further apart than they are long
    assert pa.page_pool(dims, wide, wide, 4, 5).struct.layer_stride == 7 * 16 * 2 * 64 * 2
    assert pa.page_pool(dims, k[0], k[1], 4, 5).struct.num_layers == 1
    codes, scale = torch.zeros(3, 6, 16, 2, 64, dtype=torch.int8), torch.zeros(3, 6, 2, 16, dtype=torch.float16)
    pool = pa.page_pool(dims, codes, codes, 4, 5, scale, scale)
    assert pool.struct.scale_layer_stride == 6 * 2 * 16 * 2
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    for bad in (lambda: pa.page_pool(dims, k, k[:2], 4, 5), lambda: pa.page_pool(dims, k, codes, 4, 5),
                lambda: pa.page_pool(dims, k[:, :5], k, 4, 5), lambda: pa.page_pool(dims, k, k, 4, 5, scale),
                lambda: pa.page_pool(dims, codes, codes, 4, 5), lambda: pa.page_pool(dims, k, wide, 4, 5),
                lambda: pa.page_pool(dims, k.transpose(2, 3), k, 4, 5),
                lambda: pa.PagePool(dims, k, k, i32(4, 5), i32(3), i32(6)),
                lambda: pa.PagePool(dims, k, k, i32(4, 5), i32(4), i32(7)),
                lambda: pa.PagePool(dims, k, k, i32(4, 5).long(), i32(4), i32(6)),
                lambda: pa.PagePool(dims, k, k, i32(4, 10)[:, ::2], i32(4), i32(6)),
                lambda: pa.pa_pool_append(dims, pool, i32(2), i32(2), i32(4)),
                lambda: pa.pa_pool_append(dims, pool, i32(2), i32(3).long(), i32(4)),
                lambda: pa.pa_pool_fork(dims, pool, i32(2), i32(1)),
                lambda: pa.pa_pool_free(dims, pool, i32(2).long()),
                lambda: pa.pa_pool_compact(dims, pool, i32(5))):
        with pytest.raises(ValueError, match="expected|must|agree|go together"):
            bad()
    more = pa.make_dims(7, 16, 2, 2, 64)
    for bad in (lambda: pa.pa_pool_append(more, pool, i32(2), i32(3), i32(4)), lambda: pa.pa_pool_free(more, pool, i32(2)),
                lambda: pa.pa_pool_fork(more, pool, i32(2), i32(2)), lambda: pa.pa_pool_compact(more, pool, i32(6))):
        with pytest.raises(ValueError, match="other dims"):
            bad()
    with pytest.raises(ValueError, match="current CUDA device"):
        pa.pa_pool_free(dims, pool, i32(2))
