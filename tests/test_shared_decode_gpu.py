"""Shared-prefix decode against an fp64 evaluation of its formula.

Tolerance, per output element, from the roundings alone: the softmax weights are rounded to
bf16 before the value product (at most 2^-8 of each weight) and the result once more (2^-8 of
it); everything else is fp32 (scores of up to 128 products and a few hundred in magnitude,
2^-24 each: below 2e-4 of the weights).  With a = sum_j w_j |v_j| >= |out|:
    |err| <= 2^-8 (a + |out|) + 2e-4 a.
On an INT8 cache the weights and the products' values are fp16 (2^-11 each), which leaves 2^-8 a - 2^-10 a for the
scores' error d: |err| <= 2 d a, so d up to 1.4e-3.  It comes from the keys' fp16 rounding, 2^-11 / sqrt(3) of each
product in the mean, with signs of its own: about 3e-4 for the sums of 64 and 128 products here.
"""
import numpy as np
import pytest
import torch

from paged_kv_cache_kvcache_gb300 import pagedattn as pa
from tests.test_shared_pack import make_batch

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


def reference(q, kc, vc, lists, ctx, bs, scale):
    """(out, a) in fp64 for q [B, Hq, D] over dense copies of each context."""
    B, hq, d = q.shape
    hkv = kc.shape[2]
    out = torch.zeros(B, hq, d, dtype=torch.float64, device=q.device)
    a = torch.zeros_like(out)
    for b, n in enumerate(ctx):
        if n == 0:
            continue
        ids = torch.tensor([int(x) for x in lists[b][:-(-n // bs)]], device=q.device)
        k, v = (c[ids].reshape(-1, hkv, d)[:n].double() for c in (kc, vc))
        s = torch.einsum("hgd,thd->hgt", q[b].double().view(hkv, -1, d), k) * scale
        w = torch.softmax(s, -1)
        out[b] = torch.einsum("hgt,thd->hgd", w, v).reshape(hq, d)
        a[b] = torch.einsum("hgt,thd->hgd", w, v.abs()).reshape(hq, d)
    return out, a


def assert_within(out, ref, a, what=""):
    err = (out.double() - ref).abs()
    tol = U * (a + ref.abs()) + 2e-4 * a
    assert torch.isfinite(out.float()).all(), what
    worst = float((err / tol.clamp_min(1e-30)).max())
    print(f"[shared] {what}: worst error is {worst:.3f} of its bound")
    assert worst <= 1.0, (what, worst)


def values(shape, seed, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=device).to(torch.bfloat16)


def pool(nb, bs, hkv, d, seed, ctx, lists):
    """Caches whose rows behind every context hold NaN."""
    kc, vc = values((nb, bs, hkv, d), seed), values((nb, bs, hkv, d), seed + 1)
    live = torch.zeros(nb * bs, dtype=torch.bool)
    for n, blocks in zip(ctx, lists):
        for pos in range(n):
            live[int(blocks[pos // bs]) * bs + pos % bs] = True
    dead = ~live.cuda()
    kc.view(nb * bs, hkv, d)[dead] = float("nan")
    vc.view(nb * bs, hkv, d)[dead] = float("nan")
    return kc, vc


def decode(dims, q, kc, vc, plan, scale, block_tables=None, stream=None, junk=True):
    out = torch.full_like(q, 7.0)
    ws = pa.shared_workspace(plan)
    if ws is not None and junk:
        ws.fill_(0xFF)  # NaN in every partial that nobody writes
    pa.pa_decode_shared(dims, q, kc, vc, plan, scale, out, ws, block_tables=block_tables, stream=stream)
    return out


def int8_pool(nb, bs, hkv, d, seed, ctx, lists):
    """INT8 caches [codes, codes, scales, scales] whose rows behind every context have the scale NaN, and the
    values they stand for in fp64 (0 there)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = [torch.randint(-127, 128, (nb, bs, hkv, d), generator=g, device="cuda", dtype=torch.int8) for _ in range(2)]
    scales = [(torch.rand(nb, hkv, bs, generator=g, device="cuda") * 0.03 + 0.002).to(torch.float16) for _ in range(2)]
    dead = torch.ones(nb, bs, dtype=torch.bool)
    for n, blocks in zip(ctx, lists):
        for pos in range(n):
            dead[int(blocks[pos // bs]), pos % bs] = False
    dead = dead.cuda()
    dense = []
    for c, s in zip(codes, scales):
        s.masked_fill_(dead[:, None, :], float("nan"))
        dense.append(c.double() * s.double().nan_to_num(0.0).transpose(1, 2)[..., None])
    return codes + scales, dense


def decode8(dims, q, cache, plan, scale, block_tables=None):
    out = torch.full_like(q, 7.0)
    ws = pa.shared_workspace(plan)
    if ws is not None:
        ws.fill_(0xFF)
    pa.pa_decode_shared_int8(dims, q, *cache, plan, scale, out, ws, block_tables=block_tables)
    return out


CASES = [  # sizes, shared blocks, tails, bs, hq, hkv, d
    ([1], [0], [1], 16, 1, 1, 64),                                 # one sequence, one key, one head
    ([2], [1], [1, 2], 16, 2, 1, 64),
    ([4], [3], [1, 0, 16, 40], 16, 8, 2, 64),                      # a context that is all prefix
    ([5], [9], [130, 127, 128, 129, 1], 16, 16, 8, 128),           # tails around a key tile
    ([8], [1], [44] * 8, 256, 16, 8, 128),                         # samples of a 300-token prompt
    ([3, 1, 2], [2, 4, 0], [7, 300, 1, 9, 33, 2], 32, 28, 4, 128), # several groups, one without sharing
    ([37, 20], [9, 1], [1 + 3 * i for i in range(57)], 64, 28, 4, 128),  # 18 a tile: pairs, a pair and one, one
    ([33], [5], [3 + i for i in range(33)], 16, 16, 1, 128),       # group of 16 heads: 8 a tile
    ([130], [3], [1 + i % 40 for i in range(130)], 128, 8, 8, 128),  # 128 a tile and two more
    ([5], [2], [4, None, 6, None, 9], 16, 4, 4, 64),               # entries of context 0
    ([2], [0], [None, None], 16, 4, 2, 128),                       # nothing else
    ([3], [2], [1500, 3, 700], 1024, 12, 1, 64),                   # large blocks
    ([2], [130], [5, 2000], 16, 7, 1, 128),                        # a long prefix of small blocks
]


@pytest.mark.parametrize("split", [0, 128, 384])
@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_parity(case, split):
    sizes, sh, tails, bs, hq, hkv, d = case
    ctx, lists, groups, nb = make_batch(5, sizes, sh, tails, bs)
    kc, vc = pool(nb, bs, hkv, d, 50, ctx, lists)
    q = values((len(ctx), hq, d), 52)
    dims = pa.make_dims(nb, bs, hq, hkv, d)
    plan = pa.pa_pack_decode_shared(dims, ctx, groups, block_lists=lists, split_tokens=split).upload()
    out = decode(dims, q, kc, vc, plan, d ** -0.5)
    ref, a = reference(q, kc, vc, lists, ctx, bs, d ** -0.5)
    for b, n in enumerate(ctx):
        if n == 0:
            assert (out[b] == 0).all()
    assert_within(out, ref, a, f"{case[:2]} split {split}")
    again = decode(dims, q, kc, vc, plan, d ** -0.5)
    assert torch.equal(out, again)  # no order of arrival enters the result


@pytest.mark.parametrize("split", [0, 128, 384])
@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_parity_int8(case, split):
    sizes, sh, tails, bs, hq, hkv, d = case
    ctx, lists, groups, nb = make_batch(15, sizes, sh, tails, bs)
    cache, dense = int8_pool(nb, bs, hkv, d, 150, ctx, lists)
    q = values((len(ctx), hq, d), 152)
    dims = pa.make_dims(nb, bs, hq, hkv, d)
    plan = pa.pa_pack_decode_shared(dims, ctx, groups, block_lists=lists, split_tokens=split).upload()
    out = decode8(dims, q, cache, plan, d ** -0.5)
    ref, a = reference(q, *dense, lists, ctx, bs, d ** -0.5)
    for b, n in enumerate(ctx):
        if n == 0:
            assert (out[b] == 0).all()
    assert_within(out, ref, a, f"int8 {case[:2]} split {split}")
    assert torch.equal(out, decode8(dims, q, cache, plan, d ** -0.5))


def test_int8_every_code():
    """All 255 codes in keys and values, with scales whose products fp16 holds exactly."""
    bs, hq, hkv, d = 256, 4, 1, 128
    ctx, lists = [256, 256], [[0], [0]]
    k = torch.zeros(2, bs, hkv, d, dtype=torch.int8, device="cuda")
    v = ((torch.arange(bs, device="cuda")[:, None] + torch.arange(d, device="cuda")) % 255 - 127).to(torch.int8)
    k[0, :, 0, :] = v.roll(5, 0)
    cache = [k, torch.stack([v, v])[:, :, None, :].contiguous()] + [
        torch.full((2, hkv, bs), s, dtype=torch.float16, device="cuda") for s in (0.0625, 0.25)]
    q = values((2, hq, d), 155)
    dims = pa.make_dims(2, bs, hq, hkv, d)
    plan = pa.pa_pack_decode_shared(dims, ctx, block_lists=lists, split_tokens=128).upload()
    assert plan.meta.num_shared_items > 0 and plan.meta.num_single_items == 0
    out = decode8(dims, q, cache, plan, 0.5)
    dense = [c.double() * s for c, s in zip(cache[:2], (0.0625, 0.25))]
    ref, a = reference(q, *dense, lists, ctx, bs, 0.5)
    assert_within(out, ref, a, "every code")


@pytest.mark.parametrize("split", [0, 128])
def test_int8_block_ids_outside_the_pool_read_as_zeros(split):
    bs, hq, hkv, d = 16, 4, 2, 64
    ctx, lists, groups, nb = make_batch(9, [2], [8], [20, 40], bs)
    cache, dense = int8_pool(nb, bs, hkv, d, 90, ctx, lists)
    q = values((2, hq, d), 92)
    dims = pa.make_dims(nb, bs, hq, hkv, d)
    width = max(len(x) for x in lists)
    table = np.full((4, width), -1, np.int32)
    for b, r in enumerate((3, 1)):
        table[r, :len(lists[b])] = lists[b]
    table[[1, 3], 3], table[1, 9] = -5, nb + 100
    plan = pa.pa_pack_decode_shared(dims, ctx, shared_lens=[8 * bs], table_rows=[3, 1], max_blocks=width,
                                    split_tokens=split).upload()
    out = decode8(dims, q, cache, plan, d ** -0.5, block_tables=torch.tensor(table, device="cuda"))
    torch.cuda.synchronize()
    assert pa.pa_read_device_error() == 1 << 6
    kz, vz = (torch.cat([c, torch.zeros_like(c[:1])]) for c in dense)
    zeroed = [[x if 0 <= x < nb else nb for x in table[r, :len(lists[b])].tolist()] for b, r in enumerate((3, 1))]
    ref, a = reference(q, kz, vz, zeroed, ctx, bs, d ** -0.5)
    assert_within(out, ref, a, "bad ids int8")


def test_int8_equals_pa_decode_int8_and_replays():
    bs, hq, hkv, d = 16, 28, 4, 128
    ctx, lists, groups, nb = make_batch(17, [40, 9], [40, 17], [1 + 13 * i for i in range(49)], bs)
    cache, dense = int8_pool(nb, bs, hkv, d, 170, ctx, lists)
    q = values((49, hq, d), 172)
    dims = pa.make_dims(nb, bs, hq, hkv, d)
    plan = pa.pa_pack_decode_shared(dims, ctx, groups, block_lists=lists).upload()
    ws, out = pa.shared_workspace(plan), torch.empty_like(q)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        pa.pa_decode_shared_int8(dims, q, *cache, plan, d ** -0.5, out, ws)
    p2 = pa.pa_pack_decode(dims, ctx, lists).upload()
    for rep in range(3):
        q.copy_(values((49, hq, d), 172 + rep))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        ref, a = reference(q, *dense, lists, ctx, bs, d ** -0.5)
        assert_within(out, ref, a, f"replay {rep}")
        plain = torch.empty_like(q)
        pa.pa_decode_int8(dims, q, *cache, p2, d ** -0.5, plain, pa.decode_workspace(p2))
        assert ((out.double() - plain.double()).abs() <= 2 * (U * (a + ref.abs()) + 2e-4 * a)).all()


def test_large_scores_and_scale():
    """Scores of several hundred and a prefix far above the suffix (and below it): the merge neither overflows nor
    loses the smaller part's weight."""
    bs, hq, hkv, d = 16, 8, 2, 128
    ctx, lists, groups, nb = make_batch(6, [6], [12], [9, 20, 33, 1, 64, 100], bs)
    for up in (True, False):
        kc, vc = pool(nb, bs, hkv, d, 60, ctx, lists)
        shared = torch.tensor([int(x) for x in lists[0][:12]], device="cuda")
        kc[shared] *= 6.0 if up else 0.25
        q = values((6, hq, d), 62) * 4
        dims = pa.make_dims(nb, bs, hq, hkv, d)
        plan = pa.pa_pack_decode_shared(dims, ctx, block_lists=lists, split_tokens=128).upload()
        out = decode(dims, q, kc, vc, plan, 0.25)
        ref, a = reference(q, kc, vc, lists, ctx, bs, 0.25)
        # scores reach 6 * 4 * 128 * 0.25 = 768 at the most here: 2^-24 of that per score, in log2 units 7e-5
        assert_within(out, ref, a, f"large scores {up}")


def test_equals_pa_decode():
    """The same batch through pa_decode: both within their roundings of the same sums."""
    bs, hq, hkv, d = 16, 28, 4, 128
    ctx, lists, groups, nb = make_batch(7, [24, 9], [40, 17], [1 + 13 * i for i in range(33)], bs)
    kc, vc = pool(nb, bs, hkv, d, 70, ctx, lists)
    q = values((33, hq, d), 72)
    dims = pa.make_dims(nb, bs, hq, hkv, d)
    out = decode(dims, q, kc, vc, pa.pa_pack_decode_shared(dims, ctx, groups, block_lists=lists).upload(), d ** -0.5)
    plain = torch.empty_like(q)
    plan = pa.pa_pack_decode(dims, ctx, lists).upload()
    pa.pa_decode(dims, q, kc, vc, plan, d ** -0.5, plain, pa.decode_workspace(plan))
    ref, a = reference(q, kc, vc, lists, ctx, bs, d ** -0.5)
    assert ((out.double() - plain.double()).abs() <= 2 * (U * (a + ref.abs()) + 2e-4 * a)).all()


@pytest.mark.parametrize("split", [0, 128])
def test_device_table_and_rows(split):
    """A plan for a table on the device whose rows are in another order."""
    bs, hq, hkv, d = 32, 8, 2, 64
    ctx, lists, groups, nb = make_batch(8, [3, 2], [4, 2], [5, 60, 33, 1, 2], bs)
    kc, vc = pool(nb, bs, hkv, d, 80, ctx, lists)
    q = values((5, hq, d), 82)
    dims = pa.make_dims(nb, bs, hq, hkv, d)
    rows = [7, 2, 5, 0, 3]
    table = np.full((9, 8), -1, np.int32)
    for b, r in enumerate(rows):
        table[r, :len(lists[b])] = lists[b]
    plan = pa.pa_pack_decode_shared(dims, ctx, groups, shared_lens=[4 * bs, 2 * bs], table_rows=rows, max_blocks=8,
                                    split_tokens=split).upload()
    out = decode(dims, q, kc, vc, plan, d ** -0.5, block_tables=torch.tensor(table, device="cuda"))
    ref, a = reference(q, kc, vc, lists, ctx, bs, d ** -0.5)
    assert_within(out, ref, a, "device table")
    with pytest.raises(ValueError):
        decode(dims, q, kc, vc, plan, d ** -0.5)
    with pytest.raises(ValueError):
        decode(dims, q, kc, vc, plan, d ** -0.5, block_tables=torch.tensor(table[:, :7].copy(), device="cuda"))


def test_tensors_of_the_host_are_refused():
    dims = pa.make_dims(4, 16, 2, 1, 64)
    kc, q = values((4, 16, 1, 64), 1), values((2, 2, 64), 2)
    plan = pa.pa_pack_decode_shared(dims, [20, 30], block_lists=[[0, 1], [0, 2]], split_tokens=128).upload()
    ws, out = pa.shared_workspace(plan), torch.empty_like(q)
    for args in ((q.cpu(), kc, kc, out, ws), (q, kc.cpu(), kc, out, ws), (q, kc, kc, out.cpu(), ws),
                 (q, kc, kc, out, ws.cpu())):
        with pytest.raises(ValueError):
            pa.pa_decode_shared(dims, args[0], args[1], args[2], plan, 0.1, args[3], args[4])
    wide = values((2, 3, 64), 2)[:, :2]                       # heads of a larger tensor
    for args in ((wide, kc, kc, out), (q, kc.transpose(0, 1), kc, out), (q, kc, kc, wide)):
        with pytest.raises(ValueError, match="contiguous"):
            pa.pa_decode_shared(dims, *args[:3], plan, 0.1, args[3], ws)


@pytest.mark.parametrize("split", [0, 128])
def test_block_ids_outside_the_pool_read_as_zeros(split):
    bs, hq, hkv, d = 16, 4, 2, 64
    ctx, lists, groups, nb = make_batch(9, [2], [8], [20, 40], bs)
    kc, vc = pool(nb, bs, hkv, d, 90, ctx, lists)
    q = values((2, hq, d), 92)
    dims = pa.make_dims(nb, bs, hq, hkv, d)
    width = max(len(x) for x in lists)
    table = np.full((2, width), -1, np.int32)
    for b in range(2):
        table[b, :len(lists[b])] = lists[b]
    table[:, 3], table[1, 9] = -5, nb + 100
    plan = pa.pa_pack_decode_shared(dims, ctx, shared_lens=[8 * bs], max_blocks=width, split_tokens=split).upload()
    assert plan.meta.direct == (3 if split == 0 else 0)
    out = decode(dims, q, kc, vc, plan, d ** -0.5, block_tables=torch.tensor(table, device="cuda"))
    torch.cuda.synchronize()
    assert pa.pa_read_device_error() == 1 << 6
    kz, vz = (torch.cat([c, torch.zeros_like(c[:1])]) for c in (kc, vc))  # block nb: zeros
    zeroed = [[x if 0 <= x < nb else nb for x in table[b, :len(lists[b])].tolist()] for b in range(2)]
    ref, a = reference(q, kz, vz, zeroed, ctx, bs, d ** -0.5)
    assert_within(out, ref, a, "bad ids")


def test_offsets_past_32_bits():
    """Blocks at the end of a cache of more than 2^32 elements."""
    bs, hq, hkv, d = 1024, 16, 8, 128
    nb = (1 << 32) // (bs * hkv * d) + 6
    kc = torch.zeros(nb, bs, hkv, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    lists = [[nb - 1, 0, nb - 3], [nb - 1, 0, nb - 2]]
    ctx = [2 * bs + 77, 2 * bs + 1000]
    for i, x in enumerate((nb - 1, 0, nb - 3, nb - 2)):
        kc[x], vc[x] = values((bs, hkv, d), 100 + i), values((bs, hkv, d), 110 + i)
    q = values((2, hq, d), 120)
    dims = pa.make_dims(nb, bs, hq, hkv, d)
    plan = pa.pa_pack_decode_shared(dims, ctx, block_lists=lists).upload()
    assert plan.meta.tokens_saved == 2 * bs
    out = decode(dims, q, kc, vc, plan, d ** -0.5)
    ref, a = reference(q, kc, vc, lists, ctx, bs, d ** -0.5)
    assert_within(out, ref, a, "past 32 bits")


def test_two_streams_and_a_captured_call():
    """Two calls at once with workspaces of their own, and replays of a captured one over new queries."""
    bs, hq, hkv, d = 16, 28, 4, 128
    ctx, lists, groups, nb = make_batch(10, [20], [30], [1 + 17 * i for i in range(20)], bs)
    kc, vc = pool(nb, bs, hkv, d, 130, ctx, lists)
    dims = pa.make_dims(nb, bs, hq, hkv, d)
    qs = [values((20, hq, d), 132 + i) for i in range(4)]
    refs = [reference(q, kc, vc, lists, ctx, bs, d ** -0.5) for q in qs]
    plans = [pa.pa_pack_decode_shared(dims, ctx, block_lists=lists, split_tokens=s).upload() for s in (128, 512)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(qs[0]) for _ in range(2)]
    wss = [pa.shared_workspace(p) for p in plans]
    for _ in range(5):
        for i in range(2):
            pa.pa_decode_shared(dims, qs[i], kc, vc, plans[i], d ** -0.5, outs[i], wss[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert_within(outs[i], *refs[i], f"stream {i}")

    q, out = qs[0].clone(), torch.empty_like(qs[0])
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        pa.pa_decode_shared(dims, q, kc, vc, plans[0], d ** -0.5, out, wss[0])
    for i in (2, 3):
        q.copy_(qs[i])
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert_within(out, *refs[i], f"replay {i}")


def test_store_then_shared_decode():
    """The serving step: the new tokens' rows go to the plan's slots, then the batch decodes."""
    bs, hq, hkv, d = 16, 8, 2, 128
    ctx, lists, groups, nb = make_batch(11, [7], [6], [1, 16, 17, 32, 5, 48, 33], bs)
    kc, vc = pool(nb, bs, hkv, d, 140, [c - 1 for c in ctx], lists)
    k, v, q = values((7, hkv, d), 142), values((7, hkv, d), 143), values((7, hq, d), 144)
    dims = pa.make_dims(nb, bs, hq, hkv, d)
    plan = pa.pa_pack_decode_shared(dims, ctx, block_lists=lists).upload()
    pa.pa_store_kvcache(dims, k, v, kc, vc, plan.slot_mapping, 7)
    out = decode(dims, q, kc, vc, plan, d ** -0.5)
    for b in range(7):
        blk, off = int(lists[b][(ctx[b] - 1) // bs]), (ctx[b] - 1) % bs
        assert torch.equal(kc[blk, off], k[b]) and torch.equal(vc[blk, off], v[b])
    ref, a = reference(q, kc, vc, lists, ctx, bs, d ** -0.5)
    assert_within(out, ref, a, "store then decode")


APART = [  # sizes, shared blocks, tails, bs, hq, hkv, d: more items than the lanes of 152 CTAs at 128 keys each
    ([90], [30], [1 + 7 * i for i in range(90)], 16, 28, 4, 128),     # pairs
    ([12, 30, 1], [9, 0, 2], [3 + 37 * i for i in range(43)], 64, 16, 8, 64),  # a tile, no sharing, a group of one
    ([1] * 100, [3] * 100, [5 + i for i in range(100)], 128, 8, 4, 128),  # nothing shared: the decode kernels only
    ([400], [8], [0, 9, 200, None] * 100, 16, 16, 1, 64),             # contexts that are all prefix, and empty ones
]


@pytest.mark.parametrize("case", APART, ids=range(len(APART)))
def test_more_items_than_lanes(case):
    """The parts of single sequences run beside the others; the results of both caches stay what they are."""
    sizes, sh, tails, bs, hq, hkv, d = case
    ctx, lists, groups, nb = make_batch(12, sizes, sh, tails, bs)
    q = values((len(ctx), hq, d), 150)
    dims = pa.make_dims(nb, bs, hq, hkv, d)
    plan = pa.pa_pack_decode_shared(dims, ctx, groups, block_lists=lists, split_tokens=128).upload()
    m = plan.meta
    assert m.apart == 1 and m.num_items == m.num_shared_items and (m.num_items > 0) == (max(sizes) > 1)
    kc, vc = pool(nb, bs, hkv, d, 151, ctx, lists)
    out = decode(dims, q, kc, vc, plan, d ** -0.5)
    assert_within(out, *reference(q, kc, vc, lists, ctx, bs, d ** -0.5), f"apart {case[:2]}")
    assert all((out[b] == 0).all() for b, n in enumerate(ctx) if n == 0)
    assert torch.equal(out, decode(dims, q, kc, vc, plan, d ** -0.5))
    cache, dense = int8_pool(nb, bs, hkv, d, 152, ctx, lists)
    out = decode8(dims, q, cache, plan, d ** -0.5)
    assert_within(out, *reference(q, *dense, lists, ctx, bs, d ** -0.5), f"apart int8 {case[:2]}")
    assert torch.equal(out, decode8(dims, q, cache, plan, d ** -0.5))


def test_more_items_than_lanes_on_two_streams_and_replayed():
    """Calls of three launches at once, with workspaces of their own, and a captured chain of them: each call's
    queries are the last one's result, so a launch that began too early would be seen."""
    sizes, sh, tails, bs, hq, hkv, d = APART[0]
    ctx, lists, groups, nb = make_batch(13, sizes, sh, tails, bs)
    kc, vc = pool(nb, bs, hkv, d, 160, ctx, lists)
    dims = pa.make_dims(nb, bs, hq, hkv, d)
    plan = pa.pa_pack_decode_shared(dims, ctx, groups, block_lists=lists, split_tokens=128).upload()
    assert plan.meta.apart == 1
    qs = [values((len(ctx), hq, d), 162 + i) for i in range(2)]
    want = [decode(dims, q, kc, vc, plan, d ** -0.5) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    wss, outs = [pa.shared_workspace(plan) for _ in range(2)], [torch.empty_like(qs[0]) for _ in range(2)]
    for _ in range(5):
        for i in range(2):
            pa.pa_decode_shared(dims, qs[i], kc, vc, plan, d ** -0.5, outs[i], wss[i], stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(outs[i], want[i]) for i in range(2))

    chain = [qs[0]]
    for _ in range(4):
        chain.append(decode(dims, chain[-1], kc, vc, plan, d ** -0.5))
        torch.cuda.synchronize()
    x, y = qs[0].clone(), torch.empty_like(qs[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):  # the result becomes the queries, in place of the ones before
            pa.pa_decode_shared(dims, x, kc, vc, plan, d ** -0.5, y, wss[0])
            pa.pa_decode_shared(dims, y, kc, vc, plan, d ** -0.5, x, wss[0])
    x.copy_(qs[0])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(x, chain[4]) and torch.equal(y, chain[3])


def test_more_items_than_lanes_with_ids_outside_the_pool():
    sizes, sh, tails, bs, hq, hkv, d = APART[0]
    ctx, lists, groups, nb = make_batch(14, sizes, sh, tails, bs)
    kc, vc = pool(nb, bs, hkv, d, 170, ctx, lists)
    q = values((len(ctx), hq, d), 172)
    dims = pa.make_dims(nb, bs, hq, hkv, d)
    width = max(len(x) for x in lists)
    table = np.full((len(ctx), width), -1, np.int32)
    for b, x in enumerate(lists):
        table[b, :len(x)] = x
    table[:, 3], table[80, 31], table[7, 30] = -5, nb, 1 << 30  # a shared block, two of single sequences
    plan = pa.pa_pack_decode_shared(dims, ctx, groups, shared_lens=[sh[0] * bs], max_blocks=width, split_tokens=128).upload()
    assert plan.meta.apart == 1
    out = decode(dims, q, kc, vc, plan, d ** -0.5, block_tables=torch.tensor(table, device="cuda"))
    torch.cuda.synchronize()
    assert pa.pa_read_device_error() == 1 << 6
    kz, vz = (torch.cat([c, torch.zeros_like(c[:1])]) for c in (kc, vc))  # block nb: zeros
    zeroed = [[x if 0 <= x < nb else nb for x in table[b, :len(lists[b])].tolist()] for b in range(len(ctx))]
    assert_within(out, *reference(q, kz, vz, zeroed, ctx, bs, d ** -0.5), "apart bad ids")


@pytest.mark.parametrize("n, hq, hkv, d", [(4, 28, 4, 128), (60, 28, 4, 128), (9, 16, 1, 64), (200, 4, 1, 64), (19, 16, 8, 128),
                                           (20, 16, 8, 128)])
def test_short_contexts_few_and_many(n, hq, hkv, d):
    """Contexts decoded whole, with fewer and with more (context, KV head) pairs than SMs."""
    bs = 16
    ctx, lists, groups, nb = make_batch(15, [n], [2], [1 + 5 * i % 90 for i in range(n)], bs)
    q = values((n, hq, d), 180)
    dims = pa.make_dims(nb, bs, hq, hkv, d)
    plan = pa.pa_pack_decode_shared(dims, ctx, groups, block_lists=lists).upload()
    assert plan.meta.direct == 3
    kc, vc = pool(nb, bs, hkv, d, 181, ctx, lists)
    out = decode(dims, q, kc, vc, plan, d ** -0.5)
    assert_within(out, *reference(q, kc, vc, lists, ctx, bs, d ** -0.5), f"direct {n}")
    cache, dense = int8_pool(nb, bs, hkv, d, 182, ctx, lists)
    out = decode8(dims, q, cache, plan, d ** -0.5)
    assert_within(out, *reference(q, *dense, lists, ctx, bs, d ** -0.5), f"direct int8 {n}")


CHAINS = [  # group size, shared blocks, tails: decoded whole, in one launch, in launches side by side
    (6, 2, [1 + 9 * i for i in range(6)], 0),
    (5, 70, [1 + 40 * i for i in range(5)], 128),
    (90, 30, [1 + 7 * i for i in range(90)], 128),
]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("case", CHAINS, ids=range(len(CHAINS)))
def test_order_with_the_launches_before(case, int8):
    """The launches may be set up during the one before: queries, keys and the plan itself, changed right before a
    call by a kernel and by a copy, are the ones it reads; in a captured graph too, also behind another stream."""
    n, sh, tails, split = case
    bs, hq, hkv, d = 16, 28, 4, 128
    dims, batches = None, []
    for seed in (20, 21):  # the same lengths in other blocks
        ctx, lists, groups, nb = make_batch(seed, [n], [sh], tails, bs)
        dims = pa.make_dims(nb, bs, hq, hkv, d)
        batches.append(pa.pa_pack_decode_shared(dims, ctx, groups, block_lists=lists, split_tokens=split))
    if int8:
        g = torch.Generator(device="cuda").manual_seed(190)
        src = [[torch.randint(-127, 128, (nb, bs, hkv, d), generator=g, device="cuda", dtype=torch.int8) for _ in range(2)]
               for _ in range(2)]
        scales = [(torch.rand(nb, hkv, bs, generator=g, device="cuda") * 0.03 + 0.002).to(torch.float16) for _ in range(2)]
    else:
        src, scales = [[values((nb, bs, hkv, d), 191 + 2 * i + j) for j in range(2)] for i in range(2)], []
    qs = [values((n, hq, d), 196 + i) for i in range(2)]
    call = pa.pa_decode_shared_int8 if int8 else pa.pa_decode_shared
    assert {bool(p.meta.direct) for p in batches} == {split == 0} and {p.meta.apart for p in batches} == {int(n == 90)}

    image = torch.empty(int(max(p.meta.total_bytes for p in batches)), dtype=torch.uint8, device="cuda")
    for p in batches:
        p.dev = image
    q, kv, out = torch.empty_like(qs[0]), [torch.empty_like(x) for x in src[0]], torch.empty_like(qs[0])
    wss = [pa.shared_workspace(p) for p in batches]

    def step(i, sync):
        p, c = batches[i & 1], src[i >> 1 & 1]
        for x, y in zip(kv, c):
            torch.add(y, 0, out=x)  # kernels
        torch.mul(qs[i >> 2 & 1], 1, out=q)
        p.upload()                  # a copy
        if i & 1:
            torch.add(c[0], 0, out=kv[0])  # and a kernel between the two
        if sync:
            torch.cuda.synchronize()
        call(dims, q, *kv, *scales, p, d ** -0.5, out, wss[i & 1])
        return out.clone()

    want = [step(i, True) for i in range(8)]
    assert len({w.double().sum().item() for w in want}) == 8
    torch.cuda.synchronize()
    got = [step(i, False) for i in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))

    # captured: behind a copy, behind a kernel, behind another stream's work
    batches[0].upload()
    pinned = [x.cpu().pin_memory() for x in qs]
    host_q = torch.empty_like(pinned[0]).pin_memory()
    side, graph, results = torch.cuda.Stream(), torch.cuda.CUDAGraph(), [torch.empty_like(out) for _ in range(3)]
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        q.copy_(host_q, non_blocking=True)
        call(dims, q, *kv, *scales, batches[0], d ** -0.5, results[0], wss[0])
        torch.neg(q, out=q)
        call(dims, q, *kv, *scales, batches[0], d ** -0.5, results[1], wss[0])
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            q.copy_(host_q, non_blocking=True)
        torch.cuda.current_stream().wait_stream(side)
        call(dims, q, *kv, *scales, batches[0], d ** -0.5, results[2], wss[0])
    for x, y in zip(kv, src[0]):
        x.copy_(y)
    for i in range(2):
        host_q.copy_(pinned[i])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(results[0], want[4 * i]) and torch.equal(results[2], want[4 * i])
        q.copy_(-qs[i])
        call(dims, q, *kv, *scales, batches[0], d ** -0.5, out, wss[0])
        torch.cuda.synchronize()
        assert torch.equal(results[1], out)


@pytest.mark.parametrize("case", CHAINS, ids=range(len(CHAINS)))
def test_padded_batch_and_a_row_named_twice(case):
    """Rows of q and out behind the last sequence are neither read nor written; sequences may name one table row."""
    n, sh, tails, split = case
    bs, hq, hkv, d = 16, 28, 4, 128
    ctx, lists, groups, nb = make_batch(30, [n], [sh], tails, bs)
    dims = pa.make_dims(nb, bs, hq, hkv, d)
    kc, vc = pool(nb, bs, hkv, d, 200, ctx, lists)
    cache, dense = int8_pool(nb, bs, hkv, d, 201, ctx, lists)
    width = max(len(x) for x in lists) + 1
    table = torch.full((n + 2, width), -1, dtype=torch.int32)
    for b, x in enumerate(lists):
        table[b + 1, :len(x)] = torch.tensor(np.asarray(x, np.int32))
    rows = [b + 1 for b in range(n)]
    rows[n - 2], ctx[n - 2], lists[n - 2] = rows[n - 1], ctx[n - 1] - 1, lists[n - 1]  # one token behind its twin
    plan = pa.pa_pack_decode_shared(dims, ctx, groups, shared_lens=[sh * bs], table_rows=rows, max_blocks=width,
                                    split_tokens=split).upload()
    q = values((n + 3, hq, d), 202)
    q[n:] = float("nan")
    ws, bt = pa.shared_workspace(plan), table.cuda()
    for int8 in (False, True):
        out = torch.full_like(q, 7.0)
        if int8:
            pa.pa_decode_shared_int8(dims, q, *cache, plan, d ** -0.5, out, ws, block_tables=bt)
        else:
            pa.pa_decode_shared(dims, q, kc, vc, plan, d ** -0.5, out, ws, block_tables=bt)
        ref, a = reference(q[:n], *(dense if int8 else (kc, vc)), lists, ctx, bs, d ** -0.5)
        assert_within(out[:n], ref, a, f"padded {case[:2]} int8 {int8}")
        assert (out[n:] == 7.0).all()


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("case", CHAINS, ids=range(len(CHAINS)))
def test_plan_uploaded_on_another_stream(case, int8):
    """A plan that a copy stream brings late: the call waits for it, although it may be set up during a kernel."""
    n, sh, tails, split = case
    bs, hq, hkv, d = 16, 28, 4, 128
    plans = []
    for seed in (40, 41):
        ctx, lists, groups, nb = make_batch(seed, [n], [sh], tails, bs)
        dims = pa.make_dims(nb, bs, hq, hkv, d)
        plans.append(pa.pa_pack_decode_shared(dims, ctx, groups, block_lists=lists, split_tokens=split))
    image = torch.empty(int(max(p.meta.total_bytes for p in plans)), dtype=torch.uint8, device="cuda")
    for p in plans:
        p.dev = image
    if int8:
        cache, _ = int8_pool(nb, bs, hkv, d, 210, [nb * bs], [list(range(nb))])
        call = lambda q, p, out, ws: pa.pa_decode_shared_int8(dims, q, *cache, p, d ** -0.5, out, ws)
    else:
        kc, vc = values((nb, bs, hkv, d), 211), values((nb, bs, hkv, d), 212)
        call = lambda q, p, out, ws: pa.pa_decode_shared(dims, q, kc, vc, p, d ** -0.5, out, ws)
    q0, ws = values((n, hq, d), 213), pa.shared_workspace(plans[0])
    q, out, want = torch.empty_like(q0), torch.empty_like(q0), []
    for p in plans:
        p.upload()
        torch.cuda.synchronize()
        call(q0, p, out, ws)
        want.append(out.clone())
    assert not torch.equal(*want)
    side, main = torch.cuda.Stream(), torch.cuda.current_stream()
    for i in range(4):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(400_000)  # a few hundred microseconds
            plans[i & 1].upload(stream=side)
        q.zero_()
        torch.mul(q0, 1, out=q)         # the kernel right before the call, done long before the copy
        main.wait_stream(side)
        call(q, plans[i & 1], out, ws)
        torch.cuda.synchronize()
        assert torch.equal(out, want[i & 1]), i
