"""CPU tests of the largest sizes that the calls over a bounded cache take, and of the shapes that their bindings refuse."""
import ctypes

import pytest

from paged_kv_cache_kvcache_gb300 import pagedattn as pa

DIMS = (6, 16, 4, 2, 64)


def test_a_budget_near_2_31_is_refused():
    """The choice fills a row of `kept` in steps of a thousand places: a budget of that many below 2^31 ran past it."""
    L = pa.lib()
    d, need = pa.make_dims(*DIMS), ctypes.c_uint64()
    p = pa.pa_pool(5, 4, 1, 0, block_tables=64, context_lens=64, ref_counts=64, k_cache=64, v_cache=64)
    assert L.pa_pool_workspace(ctypes.byref(d), ctypes.byref(p), ctypes.byref(need)) == pa.PA_OK

    def rc(budget, n):
        return L.pa_pool_evict(ctypes.byref(d), ctypes.byref(p), 64, n, 64, 64, budget, 0, 0, 64, 256, need.value, None)

    for budget in (2 ** 31 - 1, 2 ** 31 - 1024, 2 ** 31 - 4096):
        assert rc(budget, 0) == pa.PA_ERR_UNSUPPORTED
    assert rc(2 ** 31 - 1 - 4096, 0) == pa.PA_OK
