"""pa_decode_window(_int8) and pa_decode_weights(_int8) against their formulas in 64 bits.

The cache holds NaN and infinities wherever no query looks, and the tables no ids for pages without visible keys."""
import numpy as np
import pytest
import torch

from paged_kv_cache_kvcache_gb300 import pagedattn as pa
from tests.bounded_model import Case, attend, near

pytestmark = pytest.mark.gpu

EVERYTHING = 2 ** 31 - 1
HEADS = [(16, 8, 128), (28, 4, 128), (12, 1, 64), (7, 1, 128), (8, 8, 128), (4, 2, 64), (16, 1, 128)]
WINDOWS = [  # lengths, window, sinks, block size
    ([1, 2, 15, 16, 17, 0, 31, 33], 1, 0, 16),
    ([1, 40, 64, 65, 100, 129], 16, 4, 16),
    ([300, 77, 1000, 5], 100, 1, 32),
    ([513, 512, 511, 700, 3], 512, 100, 256),
    ([2000, 1900], 333, 16, 64),
    ([4100], 4000, 17, 16),
    ([900, 40, 0, 2500], EVERYTHING, 0, 16),
    ([257] * 40, 31, 300, 16),
    ([1024] * 3, 5, 5, 1024),
    ([70000, 2, 65537], 1000, 30, 16),
]


def run(c, q, **kw):
    out = torch.full((len(c.lens) if "table_rows" not in kw else kw["table_rows"].numel(), c.hq, c.d), 9.0,
                     dtype=torch.bfloat16, device="cuda")
    call = pa.pa_decode_window_int8 if c.int8 else pa.pa_decode_window
    call(c.dims, q.cuda(), *c.gpu, c.bt, c.ctx, c.window, c.sinks, c.scale, out, **kw)
    return out


def queries(c, n, seed=1):
    return torch.randn(n, c.hq, c.d, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


@pytest.mark.parametrize("int8", [False, True], ids=["bf16", "int8"])
@pytest.mark.parametrize("w", range(len(WINDOWS)))
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "-".join(map(str, h)))
def test_window(heads, w, int8):
    lens, window, sinks, bs = WINDOWS[w]
    c = Case(lens, *heads, bs, window, sinks, int8, seed=w)
    q = queries(c, len(lens))
    want, size, _ = c.decode(q)
    near(run(c, q), want, size)


@pytest.mark.parametrize("int8", [False, True], ids=["bf16", "int8"])
def test_rows_of_a_larger_table(int8):
    c = Case([100, 0, 700, 33, 256], 8, 2, 128, 16, 64, 4, int8)
    rows = [2, 2, 4, 0, 1, 3, 2]
    q = queries(c, len(rows))
    pick = [c.decode(q[i:i + 1].expand(5, -1, -1)) for i in range(len(rows))]
    want, size = (np.stack([p[x][r] for p, r in zip(pick, rows)]) for x in (0, 1))
    near(run(c, q, table_rows=torch.tensor(rows, dtype=torch.int32, device="cuda")), want, size)


@pytest.mark.parametrize("int8", [False, True], ids=["bf16", "int8"])
def test_many_sequences_run_without_clusters(int8):
    c = Case([int(x) for x in np.random.default_rng(5).integers(1, 200, 400)], 8, 4, 64, 16, 90, 4, int8)
    q = queries(c, 400)
    want, size, _ = c.decode(q)
    near(run(c, q), want, size)


@pytest.mark.parametrize("int8", [False, True], ids=["bf16", "int8"])
def test_bad_ids_rows_and_lengths(int8):
    c = Case([100, 60, 40], 8, 2, 64, 16, 50, 20, int8)
    q = queries(c, 3)
    c.bt[0, 0], c.bt[0, 5] = -1, c.blocks  # keys 0..15 (sinks) and 80..95 of row 0 read as zeros
    for x in (c.kd, c.vd):
        x[c.slots[0][:16]] = 0
        x[c.slots[0][80:96]] = 0
    want, size, _ = c.decode(q)
    near(run(c, q), want, size)
    assert pa.pa_read_device_error() == 1 << 6
    # a row outside the table, and one of a negative length, are empty
    c.ctx[2] = -5
    out = run(c, q, table_rows=torch.tensor([1, 3, 2], dtype=torch.int32, device="cuda"))
    assert pa.pa_read_device_error() == 1 << 6
    assert not out[1].any() and not out[2].any()
    # a context longer than its table row is cut there
    d = Case([64], 8, 2, 64, 16, 30, 0, int8)
    d.width, d.bt, d.ctx = 4, d.bt[:, :4].contiguous(), d.ctx + 1000
    want, size, _ = d.decode(q[:1])
    near(run(d, q[:1]), want, size)
    assert pa.pa_read_device_error() == 1 << 6


def test_nan_and_infinite_scores_go_through():
    c = Case([80, 80, 80, 40], 4, 2, 64, 16, 40, 4, False)
    q = queries(c, 4)
    kc, vc = c.gpu
    flat = kc.view(-1, 2, 64)
    flat[int(c.slots[0][50]), 0, 0] = float("nan")   # a visible key of KV head 0: heads 0 and 1
    vc.view(-1, 2, 64)[int(c.slots[1][79]), 1, 5] = float("nan")  # a visible value: component 5 of heads 2 and 3
    q[3] = 0
    for t in c.slots[3]:
        flat[int(t)] = 0
        flat[int(t), :, 0] = float("-inf")  # 0 * -inf: every score NaN
    out = run(c, q).float().cpu()
    assert out[0, :2].isnan().all() and not out[0, 2:].isnan().any()
    assert out[1, 2:, 5].isnan().all() and out[1].isnan().sum() == 2
    assert not out[2].isnan().any() and out[3].isnan().all()
    q[3, :, 0] = 1.0
    assert not run(c, q)[3].any()  # every score -inf: no weight at all


@pytest.mark.parametrize("int8", [False, True], ids=["bf16", "int8"])
def test_captured_call_follows_the_tables_on_the_device(int8):
    c = Case([100, 700, 33], 28, 4, 128, 16, 128, 4, int8)
    q = queries(c, 3).cuda()
    out = torch.empty_like(q)
    call = pa.pa_decode_window_int8 if int8 else pa.pa_decode_window
    args = (c.dims, q, *c.gpu, c.bt, c.ctx, c.window, c.sinks, c.scale, out)
    call(*args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(*args)
        call(*args)
    other = Case([90, 1, 600], 28, 4, 128, 16, 128, 4, int8, seed=9)  # other lengths, pages, values
    for to, x in zip(c.gpu, other.gpu):
        to.zero_()
        to[:x.shape[0]] = x[:to.shape[0]]
    assert other.blocks <= c.blocks
    c.bt.fill_(-1)
    c.bt[:, :other.width] = other.bt
    c.ctx.copy_(other.ctx)
    q.copy_(queries(c, 3, seed=7))
    graph.replay()
    want, size, _ = other.decode(q.cpu())
    near(out, want, size)


def test_two_streams_at_once():
    cs = [Case([1500] * 6, 16, 8, 128, 16, 700, 4, False, seed=s) for s in (1, 2)]
    qs = [queries(c, 6, seed=3).cuda() for c in cs]
    outs = [torch.empty_like(q) for q in qs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, q, o, st in zip(cs, qs, outs, streams):
            pa.pa_decode_window(c.dims, q, *c.gpu, c.bt, c.ctx, c.window, c.sinks, c.scale, o, stream=st)
    torch.cuda.synchronize()
    for c, q, o in zip(cs, qs, outs):
        want, size, _ = c.decode(q.cpu())
        near(o, want, size)


# ---------------------------------------------------------------- weights

LENGTHS = [([1, 2, 15, 16, 17, 0, 31, 33], 16), ([300, 77, 1000, 5], 32), ([2500, 600], 256), ([40] * 90, 16), ([5000], 64)]


@pytest.mark.parametrize("int8", [False, True], ids=["bf16", "int8"])
@pytest.mark.parametrize("n", range(len(LENGTHS)))
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "-".join(map(str, h)))
def test_weights(heads, n, int8):
    """A weight's fp32 error: of its score (at most 128 products of a few units, each sum rounded by 2^-24: under 2^-14 of
    a log2 unit) and of the exponent and the sum (2^-21): under 1e-4 of itself; its sum with the old score 2^-22."""
    lens, bs = LENGTHS[n]
    c = Case(lens, *heads, bs, EVERYTHING, 0, int8, seed=n)
    q = queries(c, len(lens))
    want, size, w = c.decode(q)
    g = torch.Generator().manual_seed(3)
    shape = (len(lens), c.hkv, c.width * bs)
    old = torch.rand(shape, generator=g)
    for b, x in enumerate(lens):
        old[b, :, x:] = float("nan")  # not looked at
    for decay, apart in ((1.0, False), (0.75, True), (0.0, True)):
        scores = old.clone().cuda()
        if decay == 0.0:
            scores.fill_(float("nan"))
        to = torch.full(shape, 5.0, device="cuda") if apart else scores
        out = torch.empty(len(lens), c.hq, c.d, dtype=torch.bfloat16, device="cuda")
        ws = pa.weights_workspace(c.dims, len(lens), c.width)
        ws.fill_(255)
        call = pa.pa_decode_weights_int8 if int8 else pa.pa_decode_weights
        call(c.dims, q.cuda(), *c.gpu, c.bt, c.ctx, c.scale, out, scores, ws, decay=decay,
             scores_out=to if apart else None)
        near(out, want, size)
        got = to.double().cpu().numpy()
        for b, x in enumerate(lens):
            base = decay * old[b, :, :x].double().numpy() if decay else 0.0
            assert (np.abs(got[b, :, :x] - base - w[b]) <= 1e-4 * w[b] + 2.0 ** -22 * (base + w[b]) + 1e-30).all()
            rest = got[b, :, x:]
            assert (rest == 5).all() if apart else np.isnan(rest).all()


def test_weights_of_other_rows_stay():
    c = Case([100, 50, 70], 8, 2, 64, 16, EVERYTHING, 0, False)
    q = queries(c, 2)
    scores = torch.zeros(3, 2, c.width * 16, device="cuda")
    out = torch.empty(2, 8, 64, dtype=torch.bfloat16, device="cuda")
    ws = pa.weights_workspace(c.dims, 2, c.width)
    rows = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    for _ in range(3):
        pa.pa_decode_weights(c.dims, q.cuda(), *c.gpu, c.bt, c.ctx, c.scale, out, scores, ws, table_rows=rows)
    a, b = (c.decode(q[i:i + 1].expand(3, -1, -1))[2] for i in (0, 1))
    got = scores.cpu().numpy()
    assert not got[1].any()
    for row, w in ((2, a[2]), (0, b[0])):
        assert np.abs(got[row][:, :w.shape[1]] - 3 * w).max() <= 4e-4
        assert abs(got[row].sum() - 3 * 8) <= 1e-3


def test_two_captured_graphs_share_a_workspace():
    cs = [Case([700, 90, 333], 8, 2, 128, 16, EVERYTHING, 0, int8, seed=4 + int8) for int8 in (False, True)]
    ws = pa.weights_workspace(cs[0].dims, 3, cs[0].width)
    runs = []
    for c in cs:
        q = queries(c, 3).cuda()
        scores, out = torch.zeros(3, 2, c.width * 16, device="cuda"), torch.empty_like(q)
        call = pa.pa_decode_weights_int8 if c.int8 else pa.pa_decode_weights
        args = (c.dims, q, *c.gpu, c.bt, c.ctx, c.scale, out, scores, ws)
        call(*args)
        scores.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(*args)
        runs.append((graph, c, q, scores, out))
    for _ in range(3):
        for r in runs:
            r[0].replay()
    for _, c, q, scores, out in runs:
        want, size, w = c.decode(q.cpu())
        near(out, want, size)
        for b, x in enumerate(w):
            assert np.abs(scores[b, :, :x.shape[1]].cpu().numpy() - 3 * x).max() <= 5e-4


@pytest.mark.parametrize("int8", [False, True], ids=["bf16", "int8"])
def test_offsets_past_32_bits(int8):
    """Pages behind 2^32 bytes of a pool, rotated and stored there and decoded from there."""
    nb, bs, hq, hkv, d = (80000 if int8 else 40000), 32, 8, 8, 128  # 2.6 GB a plane
    dims = pa.make_dims(nb, bs, hq, hkv, d)
    if int8:
        caches = pa.int8_cache(dims)
    else:
        caches = tuple(torch.zeros(nb, bs, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(100, 8, d, generator=g).to(torch.bfloat16) for _ in range(3))
    cs = torch.zeros(4, d)
    cs[:, :d // 2] = 1  # no turn
    rope = pa.Rope(dims, cs.cuda())
    pages = nb - 1 - np.arange(4)
    slots = torch.tensor(pages[np.arange(100) // bs] * bs + np.arange(100) % bs, dtype=torch.int32, device="cuda")
    out = torch.empty(100, hq, d, dtype=torch.bfloat16, device="cuda")
    store = pa.pa_rope_store_int8 if int8 else pa.pa_rope_store
    store(dims, rope, q.cuda(), k.cuda(), v.cuda(), torch.zeros(100, dtype=torch.int32, device="cuda"), slots, out, *caches)
    assert torch.equal(out.cpu(), q)
    bt = torch.tensor(pages[None], dtype=torch.int32, device="cuda")
    ctx = torch.tensor([100], dtype=torch.int32, device="cuda")
    got = torch.empty(1, hq, d, dtype=torch.bfloat16, device="cuda")
    look = pa.pa_decode_window_int8 if int8 else pa.pa_decode_window
    look(dims, q[:1].cuda(), *caches, bt, ctx, 60, 5, d ** -0.5, got)
    mask = np.r_[np.ones(5, bool), np.zeros(35, bool), np.ones(60, bool)]
    kd, vd = k.double().numpy(), v.double().numpy()
    want, size = (x[None] for x in attend(q[0].double().numpy(), kd, vd, mask, d ** -0.5)[:2])
    if int8:  # codes: within half a step of max|x| / 127 of the values, and scores of those of the keys
        size = size + 2.0 ** 8 * 0.02
    near(got, want, size)
