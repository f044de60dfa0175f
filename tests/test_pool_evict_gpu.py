"""pa_pool_evict against the plain model, bit for bit, and a run of the operators of a bounded cache together."""
import numpy as np
import pytest
import torch

from paged_kv_cache_kvcache_gb300 import pagedattn as pa
from tests import evict_model, rope_model
from tests.bounded_model import attend, near, seen
from tests.test_pool_gpu import append, assert_same, both, i32

pytestmark = pytest.mark.gpu

MALFORMED = 1 << 8


def fork(dims, pool, model, parents, children):
    pa.pa_pool_fork(dims, pool, i32(parents), i32(children))
    assert model.fork(parents, children)


def score(pool, model, hkv, seed, kind="random"):
    """Scores of every row; behind a context NaN, which nobody looks at."""
    r = np.random.default_rng(seed)
    rows, width = model.tables.shape
    shape = (rows, hkv, width * model.bs)
    x = r.exponential(size=shape).astype(np.float32) ** 2
    if kind == "ties":
        x = r.integers(0, 3, shape).astype(np.float32)
    elif kind == "odd":  # what no softmax gives, too
        x = r.standard_normal(shape).astype(np.float32) * 10.0 ** r.integers(-30, 30, shape)
        for v in (np.nan, np.inf, -np.inf, 0.0, -0.0):
            x[r.random(shape) < 0.05] = v
        x = x.astype(np.float32)
    elif kind == "equal":
        x[:] = 0
    for row, n in zip(x, model.ctx):
        row[:, max(int(n), 0):] = np.nan
    return x


def evict(dims, pool, model, rows, scores, budget, first, last, apart=False, stream=None):
    """One call on both sides; returns the scores afterwards."""
    dev = torch.tensor(scores, device="cuda")
    to = torch.full_like(dev, 7.0) if apart else dev
    kept = torch.full((len(rows), budget), -9, dtype=torch.int32, device="cuda")
    pa.pa_pool_evict(dims, pool, i32(rows), dev, budget, kept, first=first, last=last, scores_out=to if apart else None,
                     stream=stream)
    torch.cuda.synchronize()
    before = np.full_like(scores, 7.0) if apart else scores
    want = evict_model.evict(model, list(rows), scores, budget, first, last, before if apart else None)
    if want is None:
        assert pa.pa_read_device_error() == MALFORMED
        assert (kept == -1).all()
        assert np.array_equal(to.cpu().numpy(), before, equal_nan=True)
    else:
        assert pa.pa_read_device_error() == 0
        assert np.array_equal(kept.cpu().numpy(), want[0])
        assert np.array_equal(to.cpu().numpy().view(np.int32), want[1].view(np.int32)) or \
            np.array_equal(to.cpu().numpy(), want[1], equal_nan=True)
    assert_same(pool, model)
    return want


SHAPES = [  # layers, hkv, d, bs, gap, lengths, budget, first, last
    (1, 2, 64, 16, 0, [40, 33, 16, 1], 16, 0, 0),
    (2, 4, 128, 16, 3, [200, 90, 0, 333], 100, 4, 20),
    (3, 1, 64, 32, 0, [500, 64, 65, 129], 65, 1, 64),
    (1, 8, 128, 64, 1, [1000, 700], 333, 64, 100),
    (2, 7, 128, 16, 0, [300, 301, 17], 299, 0, 1),
    (1, 3, 64, 128, 0, [2500], 1, 0, 0),
    (1, 1, 128, 16, 0, [5000, 4097, 1025], 1024, 0, 1000),
    (28, 2, 64, 16, 0, [150] * 8, 64, 4, 32),
    (1, 2, 64, 16, 0, [100, 50], 60, 60, 0),
    (1, 2, 64, 16, 0, [100, 50], 60, 0, 60),
    (28, 3, 64, 16, 2, [90, 130] * 6, 70, 3, 9),  # (of INT8, scales of three heads move together, of four and one)
    (16, 5, 64, 16, 0, [130, 40] * 5, 33, 0, 4),
]


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("how", ["random", "ties", "odd", "equal"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_evict(shape, how, kind):
    layers, hkv, d, bs, gap, lens, budget, first, last = SHAPES[shape]
    pages = sum(-(-n // bs) for n in lens)
    dims, pool, model = both(kind, layers, pages + 3, bs, hkv, d, len(lens) + 2, max(-(-n // bs) for n in lens) + 1,
                             seed=shape, gap=gap)
    rows = list(np.random.default_rng(shape).permutation(len(lens) + 2)[:len(lens)])
    append(dims, pool, model, rows, lens)
    want = evict(dims, pool, model, rows[::-1], score(pool, model, hkv, shape, how), budget, first, last,
                 apart=shape % 2 == 1)
    assert want is not None
    # again: nothing is left to do; then the rows grow into what was given back, and shrink once more
    s = score(pool, model, hkv, shape + 50, how)
    evict(dims, pool, model, rows, s, budget, first, last, apart=shape % 2 == 0)
    append(dims, pool, model, rows, [max(0, n - budget) for n in lens])
    evict(dims, pool, model, rows[:1], score(pool, model, hkv, shape + 99, how), max(1, budget - 1), 0, 0)


def test_more_tokens_than_the_choice_keeps_in_shared_memory():
    for how in ("random", "ties"):
        dims, pool, model = both("bf16", 1, 130, 1024, 1, 64, 3, 65)
        append(dims, pool, model, [2, 0], [60000, 49153])
        assert evict(dims, pool, model, [0, 2], score(pool, model, 1, 4, how), 20000, 100, 500) is not None


def test_shared_pages():
    dims, pool, model = both("bf16", 2, 60, 16, 2, 64, 8, 10)
    append(dims, pool, model, [0], [70])
    fork(dims, pool, model, [0, 0], [1, 2])  # four full pages shared by three, a fifth of each one's own
    append(dims, pool, model, [1, 2], [50, 60])
    s = score(pool, model, 2, 1)
    s[1:3, :, :64] += 1000  # the prefix outweighs the rest: it stays where it is, and shared
    assert evict(dims, pool, model, [1, 2], s, 90, 0, 8) is not None
    s = score(pool, model, 2, 2)
    s[1, :, :64] += 1000
    s[1, :, 20] = 0  # token 20 would go: the shared page behind it would be written
    assert evict(dims, pool, model, [1], s, 80, 0, 8) is None
    s[1, :, :64] += 1000
    assert evict(dims, pool, model, [0], score(pool, model, 2, 3), 48, 48, 0) is not None  # shared pages given back
    model.check()
    assert evict(dims, pool, model, [1, 2], s, 64, 64, 0) is not None


@pytest.mark.parametrize("what", ["row outside", "negative row", "row twice", "page outside", "page of count 0",
                                  "length beyond the table", "negative length", "page used twice"])
def test_refused_calls_change_nothing(what):
    dims, pool, model = both("int8", 2, 40, 16, 2, 64, 6, 6)
    append(dims, pool, model, [0, 1, 2], [50, 60, 40])
    rows = [0, 1, 2]
    if what == "row outside":
        rows = [0, 6, 2]
    elif what == "negative row":
        rows = [0, 1, -1]
    elif what == "row twice":
        rows = [0, 1, 0]
    elif what == "page outside":
        model.tables[1, 2] = 40
    elif what == "page of count 0":
        model.refs[model.tables[2, 1]] = 0
    elif what == "length beyond the table":
        model.ctx[1] = 97
    elif what == "negative length":
        model.ctx[2] = -3
    else:
        model.refs[model.tables[0, 1]] = 2
    pool.block_tables.copy_(i32(model.tables))
    pool.context_lens.copy_(i32(model.ctx))
    pool.ref_counts.copy_(i32(model.refs))
    s = score(pool, model, 2, 1)
    for apart in (False, True):
        assert evict(dims, pool, model, rows, s, 30, 2, 3, apart=apart) is None


def test_wrong_tensors_are_refused():
    dims, pool, model = both()
    append(dims, pool, model, [0], [30])
    s = torch.zeros(12, 2, 96, device="cuda")
    kept = torch.zeros(1, 20, dtype=torch.int32, device="cuda")
    for kw in (dict(scores=s[:, :1]), dict(scores=s.double()), dict(scores=s.cpu()), dict(kept=kept[:, :19]),
               dict(kept=kept.long()), dict(kept=kept.cpu()), dict(rows=i32([0]).long()), dict(scores_out=s[:11])):
        args = dict(rows=i32([0]), scores=s, kept=kept) | kw
        with pytest.raises(ValueError):
            pa.pa_pool_evict(dims, pool, args["rows"], args["scores"], 20, args["kept"], scores_out=args.get("scores_out"))
    for kw in (dict(budget=0), dict(budget=20, first=15, last=6), dict(budget=20, first=-1), dict(budget=20, last=-1)):
        with pytest.raises((pa.PagedAttnError, ValueError)):
            pa.pa_pool_evict(dims, pool, i32([0]), s, kept=kept, **kw)
    assert_same(pool, model)


def test_captured_and_on_another_stream():
    dims, pool, model = both("bf16", 3, 60, 16, 2, 128, 5, 12)
    append(dims, pool, model, [0, 1, 2], [150, 70, 120])
    s = score(pool, model, 2, 8)
    state = [x.clone() for x in (pool.block_tables, pool.context_lens, pool.ref_counts, pool.k_cache, pool.v_cache)]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    evict(dims, pool, model, [2, 0, 1], s, 64, 4, 16, apart=True, stream=st)
    dev, to = torch.tensor(s, device="cuda"), torch.full(s.shape, 7.0, device="cuda")
    kept, rows = torch.empty(3, 64, dtype=torch.int32, device="cuda"), i32([2, 0, 1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_pool_evict(dims, pool, rows, dev, 64, kept, first=4, last=16, scores_out=to)
    for x, y in zip((pool.block_tables, pool.context_lens, pool.ref_counts, pool.k_cache, pool.v_cache), state):
        x.copy_(y)
    graph.replay()
    assert_same(pool, model)  # as the first time


def test_offsets_past_32_bits():
    """A layer far behind 2^32 bytes, and slots in the pool's last pages."""
    nb, bs, hkv, d = 40000, 32, 8, 128  # 2.6 GB a layer and plane
    k, v = (torch.zeros(2, nb, bs, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dims = pa.make_dims(nb, bs, hkv, hkv, d)
    pool = pa.page_pool(dims, k, v, 2, 6)
    pages = list(range(nb - 4, nb))
    pool.block_tables[1, :4] = i32(pages)
    pool.context_lens[1] = 128
    pool.ref_counts[nb - 4:] = 1
    x = torch.randn(2, 128, hkv, d, device="cuda").to(torch.bfloat16)
    k[:, nb - 4:], v[:, nb - 4:] = x.view(2, 4, bs, hkv, d), -x.view(2, 4, bs, hkv, d)
    s = torch.zeros(2, hkv, 192, device="cuda")
    s[1, :, 1:128:2] = 1
    kept = torch.empty(1, 64, dtype=torch.int32, device="cuda")
    pa.pa_pool_evict(dims, pool, i32([1]), s, 64, kept)
    assert torch.equal(kept[0].cpu(), torch.arange(1, 128, 2, dtype=torch.int32))
    assert torch.equal(k[:, nb - 4:nb - 2].reshape(2, 64, hkv, d), x[:, 1::2])
    assert torch.equal(v[:, nb - 4:nb - 2].reshape(2, 64, hkv, d), -x[:, 1::2])
    assert pool.context_lens.tolist() == [0, 64] and pool.ref_counts[nb - 4:].tolist() == [1, 1, 0, 0]
    assert pool.block_tables[1].tolist() == pages[:2] + [-1] * 4


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_serving_run(kind):
    """Prompts, then decode steps of a layer that keeps account of the weights and one with a window, with rows shrunk on
    the way: append, rotation and store, both decodes, eviction; against 64-bit arithmetic on the cache's own values."""
    int8 = kind == "int8"
    hq, hkv, d, bs, nb, rows, width = 8, 2, 64, 16, 90, 5, 16
    dims = pa.make_dims(nb, bs, hq, hkv, d)
    if int8:
        caches = pa.int8_cache(dims)
        pool = pa.page_pool(dims, *caches[:2], rows, width, *caches[2:])
    else:
        caches = tuple(torch.zeros(nb, bs, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        pool = pa.page_pool(dims, *caches, rows, width)
    rope = pa.Rope(dims, rope_model.table(2000, d).cuda(), q_weight=torch.ones(d, dtype=torch.bfloat16, device="cuda"),
                   k_weight=torch.ones(d, dtype=torch.bfloat16, device="cuda"))
    store = pa.pa_rope_store_int8 if int8 else pa.pa_rope_store
    weigh = pa.pa_decode_weights_int8 if int8 else pa.pa_decode_weights
    look = pa.pa_decode_window_int8 if int8 else pa.pa_decode_window
    g = torch.Generator().manual_seed(5)
    live = [3, 0, 4]
    lrows = i32(live)
    scores = torch.zeros(rows, hkv, width * bs, device="cuda")
    ws = pa.weights_workspace(dims, 3, width)
    pos = np.array([0, 0, 0])  # next position of each row's next token
    lens = np.array([0, 0, 0])
    scale, budget = d ** -0.5, 40

    def step(new):
        """The rows' next tokens through append and store; returns the last token's queries."""
        nonlocal pos, lens
        n = int(sum(new))
        slots = torch.empty(n, dtype=torch.int32, device="cuda")
        pa.pa_pool_append(dims, pool, lrows, i32(np.cumsum([0] + list(new))), slots)
        qkv = torch.randn(n, hq + 2 * hkv, d, generator=g).to(torch.bfloat16).cuda()
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        at = np.concatenate([p + np.arange(m) for p, m in zip(pos, new)])
        out = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
        store(dims, rope, q, k, v, i32(at), slots, out, *caches)
        want = rope_model.turned(q, rope.q_weight, rope.cos_sin, at[None], [0] * (d // 2), False, 1e-6)
        assert (np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * np.abs(want).max()).all()
        pos, lens = pos + new, lens + new
        return out[torch.as_tensor(np.cumsum(new) - 1)].contiguous()

    step([30, 7, 21])
    for i in range(60):
        q = step([1, 1, 1])
        out, out2 = torch.empty_like(q), torch.empty_like(q)
        weigh(dims, q, *caches, pool.block_tables, pool.context_lens, scale, out, scores, ws, table_rows=lrows)
        look(dims, q, *caches, pool.block_tables, pool.context_lens, 10, 3, scale, out2, table_rows=lrows)
        assert pool.context_lens[lrows.long()].tolist() == list(lens)
        if i % 7 == 0 or i > 55:  # the model on what the cache holds
            kv = [x.flatten(0, 1).double().cpu().numpy() for x in caches[:2]]
            if int8:
                kv = [x * s.transpose(1, 2).flatten(0, 1).double().cpu().numpy()[..., None] for x, s in zip(kv, caches[2:])]
            table = pool.block_tables.cpu().numpy()
            for b, (r, n) in enumerate(zip(live, lens)):
                at = (table[r, np.arange(n) // bs] * bs + np.arange(n) % bs).astype(int)
                x = q[b].double().cpu().numpy()
                for o, win, sinks in ((out, 2 ** 31 - 1, 0), (out2, 10, 3)):
                    want, size, w = attend(x, kv[0][at], kv[1][at], seen(n, n - 1, win, sinks), scale)
                    near(o[b], want, size)
        if (lens >= budget + 8).any():
            kept = torch.empty(3, budget, dtype=torch.int32, device="cuda")
            before = [scores[r, :, :n].cpu().numpy() for r, n in zip(live, lens)]
            pa.pa_pool_evict(dims, pool, lrows, scores, budget, kept, first=2, last=8)
            for b, n in enumerate(lens):
                want = evict_model.choose(before[b], int(n), budget, 2, 8)
                assert kept[b, :len(want)].tolist() == list(want)
            lens = np.minimum(lens, budget)
    assert (pool.ref_counts.sum().item() == sum(-(-int(n) // bs) for n in lens)) and (lens >= budget).all()
    assert pa.pa_read_device_error() == 0
