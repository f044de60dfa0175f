"""A compaction of a pool whose tables name pages that are outside it or free, or whose counts are negative, is
refused: nothing moves, and remap and the out arrays say so."""
import numpy as np
import pytest
import torch

from paged_kv_cache_kvcache_gb300 import pagedattn as pa
from tests.test_pool_gpu import MALFORMED, append, assert_same, both, i32

pytestmark = pytest.mark.gpu


def state(pool):
    tensors = (pool.block_tables, pool.context_lens, pool.ref_counts, pool.k_cache, pool.v_cache, pool.k_scale, pool.v_scale)
    return [x.clone() for x in tensors if x is not None]


def check_refused(dims, pool, what):
    before = state(pool)
    nb = pool.ref_counts.numel()
    stay = torch.where(pool.ref_counts != 0, torch.arange(nb, dtype=torch.int32, device="cuda"), -1)
    for in_place in (True, False):
        remap = torch.full((nb,), 99, dtype=torch.int32, device="cuda")
        tables, refs = torch.full_like(pool.block_tables, 99), torch.full_like(pool.ref_counts, 99)
        pa.pa_pool_compact(dims, pool, remap, *(() if in_place else (tables, refs)))
        torch.cuda.synchronize()
        assert pa.pa_read_device_error() == MALFORMED, (what, in_place)
        assert all(torch.equal(a, b) for a, b in zip(before, state(pool))), (what, in_place)
        assert torch.equal(remap, stay), (what, in_place)
        if not in_place:
            assert torch.equal(tables, pool.block_tables) and torch.equal(refs, pool.ref_counts), what


# (pages, rows, table width): checked by the plan, by the cluster's plan, by a launch before either; several rounds
SIZES = [(60, 12, 6), (20000, 12, 6), (300, 12, 70000), (20000, 12, 70000), (150000, 3000, 8)]


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_tables_and_counts_that_do_not_fit_together(kind, size):
    nb, rows, width = size
    dims, pool, m = both(kind, layers=1 if nb > 10000 else 2, nb=nb, rows=rows, width=width, hkv=1, seed=12)
    assert append(dims, pool, m, [4, 0, 7, rows - 1], [53, 32, 90, 20])
    pa.pa_pool_free(dims, pool, i32([0]))                      # pages 4 and 5 are free, used ones lie behind them
    m.free([0])
    for row, entry in ((4, 0), (4, 3), (7, 5), (rows - 1, 1)):
        page = int(pool.block_tables[row, entry])
        for bad in (nb, -2, -(1 << 31), (1 << 31) - 1, 4, nb - 1):    # outside the pool, free pages
            pool.block_tables[row, entry] = bad
            check_refused(dims, pool, (row, entry, bad))
        pool.block_tables[row, entry] = page
        pool.ref_counts[page] = 0
        check_refused(dims, pool, (row, entry, "free"))
        pool.ref_counts[page] = 1
    for row, entry in ((4, 4), (0, 0), (rows - 1, width - 1)):        # entries behind the lengths name pages too
        pool.block_tables[row, entry] = 5
        check_refused(dims, pool, (row, entry, "behind"))
        pool.block_tables[row, entry] = -1
    for page in (0, 13, 14, nb - 1):                                  # used and free ones
        count = int(pool.ref_counts[page])
        pool.ref_counts[page] = -1
        check_refused(dims, pool, (page, "negative"))
        pool.ref_counts[page] = count
    remap = torch.empty(nb, dtype=torch.int32, device="cuda")
    pa.pa_pool_compact(dims, pool, remap)                             # all is well again
    assert np.array_equal(remap.cpu().numpy(), m.compact())
    assert_same(pool, m, "after")
    assert pa.pa_read_device_error() == 0


def test_refused_compactions_in_a_graph():
    """A captured compaction is refused while a table names a free page and carried out when it does not."""
    dims, pool, m = both(nb=60)
    assert append(dims, pool, m, [4, 0, 7], [53, 32, 90])
    remap = torch.empty(60, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_pool_compact(dims, pool, remap)
    pa.pa_pool_free(dims, pool, i32([0]))
    m.free([0])
    pool.block_tables[3, 0] = 5
    before = state(pool)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(before, state(pool)))
    assert pa.pa_read_device_error() == MALFORMED
    pool.block_tables[3, 0] = -1
    graph.replay()
    assert np.array_equal(m.compact(), remap.cpu().numpy())
    assert_same(pool, m, "graph")
    assert pa.pa_read_device_error() == 0
