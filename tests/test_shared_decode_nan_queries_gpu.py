"""NaN queries: the rows that hold one are NaN on both caches, however the plan cuts the contexts; the others are not
touched.  Infinite queries on an INT8 cache are taken as +-65504, which the products' fp16 holds."""
import pytest
import torch

from paged_kv_cache_kvcache_gb300 import pagedattn as pa
from tests.test_shared_decode_gpu import decode, decode8, int8_pool, pool, reference
from tests.test_shared_decode_nan_gpu import HEADS, SHAPES, assert_same_nans, batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("shape", SHAPES)
def test_nan_queries(shape, heads, int8):
    dims, plan, ctx, lists, nb, q = batch(shape, heads)
    bs, (hq, hkv, d) = 16, heads
    q[0, 0, 0] = q[1, hq - 1, d - 1] = q[len(ctx) - 1, 1, 7] = float("nan")
    if int8:
        cache, dense = int8_pool(nb, bs, hkv, d, 561, ctx, lists)
        out = decode8(dims, q, cache, plan, d ** -0.5)
    else:
        dense = pool(nb, bs, hkv, d, 562, ctx, lists)
        out = decode(dims, q, *dense, plan, d ** -0.5)
    ref, a = reference(q, *dense, lists, ctx, bs, d ** -0.5)
    assert int(ref.isnan().any(-1).sum()) == 3
    assert_same_nans(out, ref, a, "queries")


@pytest.mark.parametrize("shape", SHAPES)
def test_infinite_queries_on_an_int8_cache_are_clamped(shape):
    dims, plan, ctx, lists, nb, q = batch(shape, HEADS[0])
    bs, (hq, hkv, d) = 16, HEADS[0]
    cache, dense = int8_pool(nb, bs, hkv, d, 563, ctx, lists)
    for c in dense:
        c[..., 2] = 0
    for c in cache[:2]:
        c[..., 2] = 0  # the clamped component meets zeros: it has no part in the scores
    q[0, 3, 2], q[1, 4, 2] = float("inf"), float("-inf")
    clamped = q.clone()
    clamped[0, 3, 2], clamped[1, 4, 2] = 65504.0, -65504.0
    ref, a = reference(clamped, *dense, lists, ctx, bs, d ** -0.5)
    out = decode8(dims, q, cache, plan, d ** -0.5)
    assert_same_nans(out, ref, a, "clamped")
