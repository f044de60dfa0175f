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


@pytest.mark.parametrize("fn", ["pa_decode_weights", "pa_decode_weights_int8"])
def test_a_workspace_past_2_64_bytes_is_refused(fn):
    """Scores of 2^27 + 65 (sequence, head)s of nearly 2^31 keys and 16 heads take 2^64 bytes and a few more: the size came
    out as those few."""
    L = pa.lib()
    d, need = pa.make_dims(6, 1024, 16, 1, 64), ctypes.c_uint64(5)
    assert L.pa_decode_weights_workspace(ctypes.byref(d), 1, 2 ** 21 - 1, ctypes.byref(need)) == pa.PA_OK
    assert need.value == (2 ** 31 - 1024) * 64
    for seqs, blocks in ((2 ** 27 + 65, 2 ** 21 - 1), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 28, 2 ** 20), (1, 2 ** 21)):
        assert L.pa_decode_weights_workspace(ctypes.byref(d), seqs, blocks, ctypes.byref(need)) == pa.PA_ERR_UNSUPPORTED
    f, scales = ctypes.c_float, (64, 64) if fn.endswith("int8") else ()
    assert getattr(L, fn)(ctypes.byref(d), 64, 64, 64, *scales, 64, 64, 64, 2 ** 27 + 65, 1, 2 ** 21 - 1, f(0.1), f(1.0), 64,
                          64, 64, 256, 1 << 40, None) == pa.PA_ERR_UNSUPPORTED
