"""A fork whose parents name pages that are outside the pool or free is refused and changes nothing."""
import pytest
import torch

from paged_kv_cache_kvcache_gb300 import pagedattn as pa
from tests.test_pool_gpu import MALFORMED, append, assert_same, both, i32

pytestmark = pytest.mark.gpu


def state(pool):
    tensors = (pool.block_tables, pool.context_lens, pool.ref_counts, pool.k_cache, pool.v_cache, pool.k_scale, pool.v_scale)
    return [x.clone() for x in tensors if x is not None]


def check_refused(dims, pool, parents, children, what):
    before = state(pool)
    pa.pa_pool_fork(dims, pool, i32(parents), i32(children))
    torch.cuda.synchronize()
    assert pa.pa_read_device_error() == MALFORMED, what
    assert all(torch.equal(a, b) for a, b in zip(before, state(pool))), what


# (pages, rows, table width): checked by the plan, by the cluster's plan, by a launch before either
SIZES = [(60, 12, 6), (40000, 12, 6), (300, 12, 70000), (40000, 12, 70000), (9000, 3000, 8)]


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_parents_of_pages_that_are_not_in_use(kind, size):
    nb, rows, width = size
    dims, pool, m = both(kind, layers=1 if nb > 10000 else 2, nb=nb, rows=rows, width=width, hkv=1, seed=11)
    assert append(dims, pool, m, [4, 0, 7], [53, 32, 90])      # 4, 2 and 6 pages: ids 0 to 11
    many = list(range(12, min(rows, 2900)))                    # a large call where the pool has the rows
    for row, entry in ((4, 0), (4, 2), (4, 3), (0, 1), (7, 4), (7, 5)):   # full pages and partly filled ones
        page = int(pool.block_tables[row, entry])
        calls = [([row], [5]), ([7, 4, 0, 7], [5, 11, 1, 2])]
        if many:
            calls += [([0, 7, 4] * (len(many) // 3), many[:len(many) // 3 * 3])]
        for parents, children in calls:
            for bad in (-1, nb, -(1 << 31), (1 << 31) - 1, 20):    # outside the pool; page 20 is free
                pool.block_tables[row, entry] = bad
                check_refused(dims, pool, parents, children, (row, entry, bad, parents[:4]))
            pool.block_tables[row, entry] = page
            for count in (0, -1):                                  # the page itself counted as free, or below
                pool.ref_counts[page] = count
                check_refused(dims, pool, parents, children, (row, entry, "count", count, parents[:4]))
            pool.ref_counts[page] = 1
    pa.pa_pool_fork(dims, pool, i32([7, 4, 0, 7]), i32([5, 11, 1, 2]))   # all is well again
    assert m.fork([7, 4, 0, 7], [5, 11, 1, 2])
    assert_same(pool, m, "after")
    assert pa.pa_read_device_error() == 0


def test_what_stands_behind_a_parents_length_does_not_matter():
    """Entries behind a parent's pages, and other rows' entries, have no part in a fork."""
    dims, pool, m = both(nb=60)
    assert append(dims, pool, m, [4, 0], [53, 32])
    pool.block_tables[4, 4], pool.block_tables[0, 2:] = 77, -9
    pool.block_tables[8, 0] = 1000
    pa.pa_pool_fork(dims, pool, i32([4, 0, 9]), i32([5, 1, 2]))          # row 9 is empty
    assert m.fork([4, 0, 9], [5, 1, 2])
    torch.cuda.synchronize()
    assert pa.pa_read_device_error() == 0
    assert torch.equal(pool.block_tables[[5, 1, 2]].cpu(), torch.tensor(m.tables[[5, 1, 2]]))
    assert torch.equal(pool.ref_counts.cpu(), torch.tensor(m.refs))


def test_refused_forks_in_a_graph():
    """A captured fork is refused while a page is marked as free and carried out when it is in use again."""
    dims, pool, m = both(nb=60)
    assert append(dims, pool, m, [4], [53])
    parents, children = i32([4, 4]), i32([5, 6])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_pool_fork(dims, pool, parents, children)
    for _ in range(3):
        pool.ref_counts[1] = 0
        before = state(pool)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(before, state(pool)))
        assert pa.pa_read_device_error() == MALFORMED
        pool.ref_counts[1] = 1
        graph.replay()
        assert m.fork([4, 4], [5, 6])
        assert_same(pool, m, "graph")
        assert pa.pa_read_device_error() == 0
        pa.pa_pool_free(dims, pool, children)
        m.free([5, 6])
