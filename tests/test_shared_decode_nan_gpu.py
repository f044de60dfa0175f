"""NaN and infinities in queries, keys and values: the shared decode shows them wherever the formula has them, and
nowhere else, however the plan cuts the contexts.

Expected is the formula in fp64, softmax(scale q K^T) V, which is NaN for a (sequence, query head) that meets a NaN
score, and in one component for a NaN value.  The finite elements keep the tolerance of the finite cases."""
import pytest
import torch

from paged_kv_cache_kvcache_gb300 import pagedattn as pa
from tests.test_shared_decode_gpu import U, decode, decode8, int8_pool, pool, reference, values
from tests.test_shared_pack import make_batch

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")

SHAPES = {  # sequences, shared blocks, tails, split
    "few whole": (4, 4, [60, 200, 33, 1], 0),
    "many whole": (60, 2, [1 + 5 * i % 90 for i in range(60)], 0),
    "lanes": (4, 40, [60, 200, 33, 1], 128),
    "one part": (5, 0, [300, 200, 33, 1, 90], 1024),
    "apart": (90, 30, [1 + 7 * i for i in range(90)], 128),
}
HEADS = [(28, 4, 128), (16, 1, 64)]


def assert_same_nans(out, ref, a, what):
    out = out.double()
    assert torch.equal(out.isnan(), ref.isnan()), (what, int(out.isnan().sum()), int(ref.isnan().sum()))
    ok = ~ref.isnan()
    err, tol = (out - ref).abs()[ok], (U * (a + ref.abs()) + 2e-4 * a)[ok]
    assert (err <= tol).all(), (what, float((err / tol.clamp_min(1e-30)).max()))


def batch(shape, heads):
    (n, sh, tails, split), bs, (hq, hkv, d) = SHAPES[shape], 16, heads
    ctx, lists, groups, nb = make_batch(51, [n], [sh], tails, bs)
    dims = pa.make_dims(nb, bs, hq, hkv, d)
    shared = [sh * bs] if shape != "one part" else [0]
    plan = pa.pa_pack_decode_shared(dims, ctx, groups, shared_lens=shared, block_lists=lists, split_tokens=split).upload()
    return dims, plan, ctx, lists, nb, values((n, hq, d), 520)


def place(lists, b, pos, bs=16):
    return int(lists[b][pos // bs]), pos % bs


@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("shape", SHAPES)
def test_nan_keys_and_values(shape, heads):
    dims, plan, ctx, lists, nb, q = batch(shape, heads)
    (n, sh, _, _), bs, (hq, hkv, d) = SHAPES[shape], 16, heads
    kc, vc = pool(nb, bs, hkv, d, 521, ctx, lists)
    g = hkv - 1
    last = lambda b: place(lists, b, ctx[b] - 1)
    kc[last(0)][0, 3] = NAN                 # a key of one sequence: its rows of KV head 0
    vc[last(1)][g, 5] = NAN                 # a value: one component of its heads behind the last KV head
    if sh:
        vc[place(lists, 0, 17)][0, d - 1] = NAN  # a value that all sequences share
    ref, a = reference(q, kc, vc, lists, ctx, bs, d ** -0.5)
    assert ref.isnan().any() and not ref[2].isnan().all()
    assert_same_nans(decode(dims, q, kc, vc, plan, d ** -0.5), ref, a, "values")
    if sh:                                  # a key that all share: nothing of KV head g is left
        kc[place(lists, 0, 2)][g, 0] = NAN
        ref, a = reference(q, kc, vc, lists, ctx, bs, d ** -0.5)
        assert_same_nans(decode(dims, q, kc, vc, plan, d ** -0.5), ref, a, "shared key")


@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("shape", SHAPES)
def test_nan_scales_of_an_int8_cache(shape, heads):
    dims, plan, ctx, lists, nb, q = batch(shape, heads)
    (n, sh, _, _), bs, (hq, hkv, d) = SHAPES[shape], 16, heads
    cache, dense = int8_pool(nb, bs, hkv, d, 531, ctx, lists)
    g = hkv - 1

    def spoil(which, b, pos, head):
        page, off = place(lists, b, pos)
        cache[2 + which][page, head, off] = NAN
        dense[which][page, off, head] = NAN

    spoil(0, 0, ctx[0] - 1, 0)
    spoil(1, 1, ctx[1] - 1, g)
    ref, a = reference(q, *dense, lists, ctx, bs, d ** -0.5)
    assert_same_nans(decode8(dims, q, cache, plan, d ** -0.5), ref, a, "scales")
    if sh:
        spoil(0, 0, 2, g)
        ref, a = reference(q, *dense, lists, ctx, bs, d ** -0.5)
        assert_same_nans(decode8(dims, q, cache, plan, d ** -0.5), ref, a, "shared scale")


@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("shape", SHAPES)
def test_infinite_keys(shape, heads):
    """A score of +inf makes its row NaN, keys of score -inf have no weight: one alone, and so many of a context's
    first ones that whole steps of the running maximum see nothing else."""
    dims, plan, ctx, lists, nb, q = batch(shape, heads)
    (n, sh, _, _), bs, (hq, hkv, d) = SHAPES[shape], 16, heads
    kc, vc = pool(nb, bs, hkv, d, 541, ctx, lists)
    q[:, :, 0] = 1.0
    q[1, :, 0] = -1.0
    kc[place(lists, 0, ctx[0] - 1)][0, 0] = INF
    if sh:
        kc[place(lists, 0, 5)][hkv - 1, 0] = -INF
        first = [place(lists, 0, i) for i in range(32)]
    else:
        first = [place(lists, 2, i) for i in range(32)]
    for page, off in first:
        kc[page, off, 0, 0] = -INF
    ref, a = reference(q, kc, vc, lists, ctx, bs, d ** -0.5)
    assert ref.isnan().any() and not ref.isnan().all()
    assert_same_nans(decode(dims, q, kc, vc, plan, d ** -0.5), ref, a, "infinite keys")


def test_contexts_of_keys_without_weight_are_zeros():
    """Every score -inf: nothing has a weight, as in an empty context."""
    for split in (0, 128):
        bs, hq, hkv, d, n = 16, 8, 2, 64, 3
        ctx, lists, groups, nb = make_batch(52, [n], [10], [70, 3, 200], bs)
        kc, vc = pool(nb, bs, hkv, d, 551, ctx, lists)
        kc[..., 0] = -INF
        q = values((n, hq, d), 552)
        q[:, :, 0] = 1.0
        dims = pa.make_dims(nb, bs, hq, hkv, d)
        plan = pa.pa_pack_decode_shared(dims, ctx, groups, block_lists=lists, split_tokens=split).upload()
        kc[torch.isnan(kc)] = 0.0  # (rows behind the contexts; no NaN stays in a live one)
        kc[..., 0] = -INF
        assert (decode(dims, q, kc, vc, plan, d ** -0.5) == 0).all(), split
