"""The page pool's calls on the GPU against the plain model: integers and copied pages are compared bit for bit."""
import numpy as np
import pytest
import torch

from paged_kv_cache_kvcache_gb300 import pagedattn as pa
from tests.pool_model import PoolModel
from tests.test_shared_decode_gpu import assert_within, reference, values

pytestmark = pytest.mark.gpu

NO_ROOM, MALFORMED = 1 << 7, 1 << 8


def i32(x, device="cuda"):
    return torch.tensor(np.asarray(x, np.int32), device=device)


def caches(kind, layers, nb, bs, hkv, d, seed, gap=0):
    """(k, v, ks, vs) on the GPU with `gap` pages of another owner between the layers."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "bf16":
        return [torch.randn(layers, nb + gap, bs, hkv, d, generator=g, device="cuda").to(torch.bfloat16)[:, :nb]
                for _ in range(2)] + [None, None]
    kv = [torch.randint(-127, 128, (layers, nb + gap, bs, hkv, d), generator=g, device="cuda", dtype=torch.int8)[:, :nb]
          for _ in range(2)]
    sc = [torch.rand(layers, nb + gap, hkv, bs, generator=g, device="cuda").to(torch.float16)[:, :nb] for _ in range(2)]
    return kv + sc


def host(x):
    return x.cpu().view(torch.int16).numpy().copy() if x.dtype in (torch.bfloat16, torch.float16) else x.cpu().numpy().copy()


def both(kind="bf16", layers=2, nb=40, bs=16, hkv=2, d=64, rows=12, width=6, seed=1, gap=0):
    """(dims, pool, model) over the same pages."""
    k, v, ks, vs = caches(kind, layers, nb, bs, hkv, d, seed, gap)
    dims = pa.make_dims(nb, bs, hkv, hkv, d)
    pool = pa.page_pool(dims, k, v, rows, width, ks, vs)
    model = PoolModel(rows, width, nb, bs, [host(k), host(v)], [host(x) for x in (ks, vs) if x is not None])
    return dims, pool, model


def assert_same(pool, model, what=""):
    torch.cuda.synchronize()
    assert np.array_equal(pool.block_tables.cpu().numpy(), model.tables), what
    assert np.array_equal(pool.context_lens.cpu().numpy(), model.ctx), what
    assert np.array_equal(pool.ref_counts.cpu().numpy(), model.refs), what
    for got, want in zip((pool.k_cache, pool.v_cache), model.pages):
        assert np.array_equal(host(got), want), what
    for got, want in zip((pool.k_scale, pool.v_scale), model.scales):
        assert np.array_equal(host(got), want), what


def append(dims, pool, model, rows, counts, stream=None):
    cu = np.cumsum([0] + list(counts))
    slots = torch.full((max(int(cu[-1]), 0),), -7, dtype=torch.int32, device="cuda")
    pa.pa_pool_append(dims, pool, i32(rows), i32(cu), slots, stream=stream)
    want = model.append(list(rows), list(counts))
    torch.cuda.synchronize()
    assert slots.cpu().tolist() == (want if want is not None else [-1] * slots.numel())
    return want is not None


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_worked_example(kind):
    dims, pool, m = both(kind, gap=3)
    assert append(dims, pool, m, [7], [37])
    pa.pa_pool_fork(dims, pool, i32([7, 7, 7]), i32([0, 11, 3]))
    assert m.fork([7, 7, 7], [0, 11, 3])
    assert_same(pool, m, "fork")
    assert append(dims, pool, m, [0, 3, 7, 11], [1, 20, 0, 11])
    assert_same(pool, m, "append")
    pa.pa_pool_free(dims, pool, i32([7, 11]))
    m.free([7, 11])
    assert_same(pool, m, "free")
    remap = torch.empty(40, dtype=torch.int32, device="cuda")
    pa.pa_pool_compact(dims, pool, remap)
    assert np.array_equal(remap.cpu().numpy(), m.compact())
    assert_same(pool, m, "compact")
    m.check()


@pytest.mark.parametrize("kind,layers,nb,bs,hkv,d,gap", [
    ("bf16", 1, 40, 16, 1, 64, 0), ("bf16", 3, 70, 32, 2, 128, 1), ("int8", 2, 50, 16, 4, 64, 0),
    ("int8", 1, 37, 256, 3, 128, 2), ("bf16", 2, 45, 1024, 1, 64, 0), ("int8", 3, 41, 64, 1, 64, 5)])
def test_random_sequences_of_calls(kind, layers, nb, bs, hkv, d, gap):
    """Two hundred random calls, refused ones among them."""
    rng = np.random.default_rng(layers * 100 + nb)
    rows, width = 14, 5
    dims, pool, m = both(kind, layers, nb, bs, hkv, d, rows, width, seed=nb, gap=gap)
    refused = 0
    for step in range(200):
        op = rng.integers(5)
        some = rng.permutation(rows)[:rng.integers(1, 6)]
        if op <= 1:
            ok = append(dims, pool, m, some, rng.integers(0, 2 * bs + 2, len(some)))
        elif op == 2:
            parents = rng.integers(0, rows, len(some))
            pa.pa_pool_fork(dims, pool, i32(parents), i32(some))
            ok = m.fork(parents.tolist(), some.tolist())
        elif op == 3:
            pa.pa_pool_free(dims, pool, i32(some))
            m.free(some)
            ok = True
        else:
            remap = torch.empty(nb, dtype=torch.int32, device="cuda")
            if step % 2:
                tables, refs = torch.full_like(pool.block_tables, 99), torch.full_like(pool.ref_counts, 99)
                pa.pa_pool_compact(dims, pool, remap, tables, refs)
                pool.block_tables.copy_(tables)
                pool.ref_counts.copy_(refs)
            else:
                pa.pa_pool_compact(dims, pool, remap)
            assert np.array_equal(remap.cpu().numpy(), m.compact())
            ok = True
        torch.cuda.synchronize()
        code = pa.pa_read_device_error()
        assert (code & (NO_ROOM | MALFORMED) != 0) == (not ok) and code & ~(NO_ROOM | MALFORMED) == 0, (step, op, code)
        refused += not ok
        if step % 20 == 0 or not ok:
            assert_same(pool, m, f"step {step}")
    assert_same(pool, m, "end")
    m.check()
    assert 10 < refused < 150


REFUSALS = {
    "no free pages": (NO_ROOM, lambda d, p, o: append_only(d, p, [4], [31 * 16 + 1])),
    "table too narrow": (NO_ROOM, lambda d, p, o: append_only(d, p, [0], [40 * 16])),
    "a row outside": (MALFORMED, lambda d, p, o: append_only(d, p, [12], [1])),
    "a negative row": (MALFORMED, lambda d, p, o: append_only(d, p, [-1], [1])),
    "a row twice": (MALFORMED, lambda d, p, o: append_only(d, p, [4, 0, 4], [1, 1, 1])),
    "a negative count": (MALFORMED, lambda d, p, o: append_only(d, p, [4, 5], [3, -1])),
    "counts beside the slots": (MALFORMED, lambda d, p, o: pa.pa_pool_append(d, p, i32([4]), i32([0, 3]), o[:2])),
    "counts from 1": (MALFORMED, lambda d, p, o: pa.pa_pool_append(d, p, i32([4]), i32([1, 3]), o[:3])),
    "fork without pages": (NO_ROOM, lambda d, p, o: pa.pa_pool_fork(d, p, i32([0] * 10), i32(list(range(2, 12))))),
    "child in use": (MALFORMED, lambda d, p, o: pa.pa_pool_fork(d, p, i32([0]), i32([1]))),
    "child twice": (MALFORMED, lambda d, p, o: pa.pa_pool_fork(d, p, i32([0, 1]), i32([5, 5]))),
    "child and parent": (MALFORMED, lambda d, p, o: pa.pa_pool_fork(d, p, i32([0, 5]), i32([5, 6]))),
    "parent outside": (MALFORMED, lambda d, p, o: pa.pa_pool_fork(d, p, i32([12]), i32([5]))),
    "child outside": (MALFORMED, lambda d, p, o: pa.pa_pool_fork(d, p, i32([0]), i32([99]))),
}


def append_only(dims, pool, rows, counts):
    cu = np.cumsum([0] + list(counts))
    pa.pa_pool_append(dims, pool, i32(rows), i32(cu), torch.empty(max(int(cu[-1]), 0), dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("name", REFUSALS)
def test_refused_calls_change_nothing(name):
    """33 pages in use, 9 left: a prompt of 500 tokens and one of 25."""
    bit, call = REFUSALS[name]
    dims, pool, m = both(nb=42, width=35)
    assert append(dims, pool, m, [0, 1], [500, 10])
    out = torch.zeros(8, dtype=torch.int32, device="cuda")
    call(dims, pool, out)
    torch.cuda.synchronize()
    assert pa.pa_read_device_error() == bit
    assert_same(pool, m, name)
    if "counts" in name:
        assert (out[:2] == -1).all() and (out[3:] == 0).all()
    assert append(dims, pool, m, [1], [16 * 9])      # the pool goes on
    assert_same(pool, m, name)


def test_shared_partly_filled_page_is_not_written():
    """A table that shares its last, partly filled page (not a fork's doing) cannot grow into it."""
    dims, pool, m = both()
    assert append(dims, pool, m, [0], [20])
    pool.block_tables[1, :2] = pool.block_tables[0, :2]
    pool.context_lens[1] = 20
    pool.ref_counts[:2] += 1
    before = [x.clone() for x in (pool.block_tables, pool.context_lens, pool.ref_counts)]
    append_only(dims, pool, [1], [1])
    torch.cuda.synchronize()
    assert pa.pa_read_device_error() == MALFORMED
    assert all(torch.equal(a, b) for a, b in zip(before, (pool.block_tables, pool.context_lens, pool.ref_counts)))


def test_rows_of_nearly_2_to_31_tokens():
    """A table wide enough for more tokens than an int32 counts: the row is refused before its length wraps."""
    dims, pool, m = both(layers=1, nb=8, bs=1024, hkv=1, d=64, rows=2, width=(1 << 21) + 4, seed=6)
    pool.context_lens[1] = (1 << 31) - 1 - 1024 - 5          # (its pages do not matter here)
    for count in (6, 1024, 5000):
        append_only(dims, pool, [1], [count])
        torch.cuda.synchronize()
        assert pa.pa_read_device_error() & NO_ROOM
    assert int(pool.context_lens[1]) == (1 << 31) - 1 - 1024 - 5 and int(pool.ref_counts.sum()) == 0


def test_tensors_of_the_host_are_refused():
    dims, pool, m = both()
    rows, cu, slots = i32([1]), i32([0, 1]), torch.empty(1, dtype=torch.int32, device="cuda")
    for bad in (lambda: pa.pa_pool_append(dims, pool, rows.cpu(), cu, slots),
                lambda: pa.pa_pool_append(dims, pool, rows, cu, slots.cpu()),
                lambda: pa.pa_pool_fork(dims, pool, rows, rows.cpu()), lambda: pa.pa_pool_free(dims, pool, rows.cpu()),
                lambda: pa.pa_pool_compact(dims, pool, torch.empty(40, dtype=torch.int32))):
        with pytest.raises(ValueError):
            bad()
    assert_same(pool, m)


def test_free_twice_empty_and_outside():
    dims, pool, m = both()
    assert append(dims, pool, m, [0, 1, 2], [20, 33, 1])
    pa.pa_pool_free(dims, pool, i32([1, 5, 1, 1, 2]))
    m.free([1, 2])
    assert_same(pool, m)
    assert pa.pa_read_device_error() == 0
    pa.pa_pool_free(dims, pool, i32([-1, 0, 12]))
    m.free([0])
    assert_same(pool, m)
    assert pa.pa_read_device_error() == MALFORMED


@pytest.mark.parametrize("nb,bs,n,most", [(5000, 16, 300, 200), (140000, 16, 700, 1500), (4096, 16, 1, 30000),
                                          (9001, 32, 1500, 3)])
def test_large_pools(nb, bs, n, most):
    """Pools and batches over several planning CTAs and several rounds of ids; append, fork, free and compact."""
    rng = np.random.default_rng(nb)
    rows = 2 * n + 5
    width = max(-(-most // bs) + 1, 4)
    dims, pool, m = both(layers=1, nb=nb, bs=bs, hkv=1, d=64, rows=rows, width=width, seed=3)
    perm = rng.permutation(rows)
    counts = rng.integers(most // 2, most + 1, n)
    while sum(-(-int(c) // bs) for c in counts) > nb * 0.7:
        counts = counts // 2
    assert append(dims, pool, m, perm[:n], counts)
    assert_same(pool, m, "append")
    gone = perm[:n][rng.random(n) < 0.4][:n - 1]
    if len(gone):
        pa.pa_pool_free(dims, pool, i32(gone))
        m.free(gone)
    kept = [r for r in perm[:n] if m.ctx[r]]
    parents = rng.choice(kept, min(n, 200))
    children = perm[n:n + len(parents)]
    pa.pa_pool_fork(dims, pool, i32(parents), i32(children))
    assert m.fork(parents.tolist(), children.tolist())
    assert_same(pool, m, "fork")
    assert append(dims, pool, m, kept, [1] * len(kept))
    remap = torch.empty(nb, dtype=torch.int32, device="cuda")
    pa.pa_pool_compact(dims, pool, remap)
    assert np.array_equal(remap.cpu().numpy(), m.compact())
    assert_same(pool, m, "compact")
    m.check()


@pytest.mark.parametrize("nb", [900, 60000])
def test_very_many_rows(nb):
    """More rows than the bitmap of a call's rows holds."""
    rows = 70000
    dims, pool, m = both(layers=1, nb=nb, bs=16, hkv=1, d=64, rows=rows, width=3, seed=4)
    some = [69999, 0, 65536, 65535, 40000]
    assert append(dims, pool, m, some, [5, 16, 30, 1, 0])
    for rows_, counts in (([1, 69999, 1], [1, 1, 1]), ([65536 + 7, 9, 65536 + 7], [1, 1, 1])):
        assert not append(dims, pool, m, rows_, counts)
        assert pa.pa_read_device_error() == MALFORMED
    for parents, children in (([0, 69999], [68000, 68000]), ([69999, 5], [5, 68000]), ([69998], [69999])):
        pa.pa_pool_fork(dims, pool, i32(parents), i32(children))
        assert not m.fork(parents, children)
        assert pa.pa_read_device_error() == MALFORMED
    pa.pa_pool_fork(dims, pool, i32([69999, 65536, 65536]), i32([69998, 1, 66000]))
    assert m.fork([69999, 65536, 65536], [69998, 1, 66000])
    pa.pa_pool_free(dims, pool, i32([0, 65536]))
    m.free([0, 65536])
    remap = torch.empty(nb, dtype=torch.int32, device="cuda")
    pa.pa_pool_compact(dims, pool, remap)
    assert np.array_equal(remap.cpu().numpy(), m.compact())
    assert_same(pool, m)


def test_fragmented_pools():
    """Used and free pages in random places, over one and over several rounds of ids."""
    for nb, used in ((1, 1), (15, 7), (17, 16), (4097, 2000), (16384, 16000), (50001, 20000), (300007, 150000)):
        dims, pool, m = both(layers=1, nb=nb, bs=16, hkv=1, d=64, rows=3, width=max(used // 2 + 1, 6000), seed=5)
        rng = np.random.default_rng(nb)
        ids = rng.permutation(nb)[:used].astype(np.int32)
        half = used // 2
        for r, part in ((0, ids[:half]), (2, ids[half:])):
            m.tables[r, :len(part)], m.ctx[r] = part, 16 * len(part)
        m.refs[ids] = 1
        m.check()
        pool.block_tables.copy_(i32(m.tables)), pool.context_lens.copy_(i32(m.ctx)), pool.ref_counts.copy_(i32(m.refs))
        n = min(nb - used, 5000)
        assert append(dims, pool, m, [1], [16 * n])     # the lowest free ids, wherever they are
        assert_same(pool, m, f"append {nb}")
        pa.pa_pool_free(dims, pool, i32([0]))
        m.free([0])
        remap = torch.empty(nb, dtype=torch.int32, device="cuda")
        tables, refs = torch.full_like(pool.block_tables, 99), torch.full_like(pool.ref_counts, 99)
        pa.pa_pool_compact(dims, pool, remap, tables, refs)
        assert np.array_equal(remap.cpu().numpy(), m.compact())
        pool.block_tables.copy_(tables), pool.ref_counts.copy_(refs)
        assert_same(pool, m, f"compact {nb}")


def test_full_and_empty_pools():
    dims, pool, m = both(nb=9, rows=4, width=9)
    remap = torch.empty(9, dtype=torch.int32, device="cuda")
    pa.pa_pool_compact(dims, pool, remap)
    assert (remap == -1).all()
    assert append(dims, pool, m, [2], [9 * 16])
    pa.pa_pool_compact(dims, pool, remap)
    assert remap.tolist() == list(range(9))
    assert not append(dims, pool, m, [1], [1])
    assert pa.pa_read_device_error() == NO_ROOM
    assert append(dims, pool, m, [1, 2], [0, 0])     # nothing asked for, nothing taken
    pa.pa_pool_fork(dims, pool, i32([2]), i32([0]))  # whole pages only: a full pool can still share them
    assert m.fork([2], [0])
    assert_same(pool, m)


def test_captured_step():
    """One decode step's append, replayed until the rows outgrow their pages, and a fork and a free in a graph."""
    dims, pool, m = both(nb=40)
    assert append(dims, pool, m, [3, 4, 5], [10, 31, 16])
    rows, cu, slots = i32([3, 4, 5]), i32([0, 1, 2, 3]), torch.empty(3, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        pa.pa_pool_append(dims, pool, rows, cu, slots)
    for _ in range(40):
        graph.replay()
        want = m.append([3, 4, 5], [1, 1, 1])
        torch.cuda.synchronize()
        assert slots.tolist() == want
    assert_same(pool, m)
    parents, children = i32([3, 4, 4]), i32([0, 1, 2])
    graph2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph2, stream=s):
        pa.pa_pool_fork(dims, pool, parents, children)
        pa.pa_pool_append(dims, pool, children, cu, slots)
        pa.pa_pool_free(dims, pool, children)
    for _ in range(3):
        graph2.replay()
        assert m.fork([3, 4, 4], [0, 1, 2])
        want = m.append([0, 1, 2], [1, 1, 1])
        m.free([0, 1, 2])
        torch.cuda.synchronize()
        assert slots.tolist() == want
    assert_same(pool, m)


def test_offsets_past_32_bits():
    """Pages whose byte and element offsets within the layers pass 2^32."""
    bs, hkv, d, layers = 1024, 8, 128, 2
    nb = (1 << 32) // (bs * hkv * d) + 4
    k = torch.zeros(layers, nb, bs, hkv, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    dims = pa.make_dims(nb, bs, hkv, hkv, d)
    pool = pa.page_pool(dims, k, v, 3, 4)
    pool.ref_counts.fill_(1)                          # all taken but one
    pool.ref_counts[nb - 2] = 0
    pool.ref_counts[0] = 0
    pool.block_tables[0, 0], pool.context_lens[0] = nb - 1, 1000
    k[:, nb - 1], v[:, nb - 1] = values((layers, bs, hkv, d), 5), values((layers, bs, hkv, d), 6)
    pa.pa_pool_fork(dims, pool, i32([0, 0]), i32([1, 2]))
    torch.cuda.synchronize()
    assert pool.block_tables[:, 0].tolist() == [nb - 1, 0, nb - 2]
    for page in (0, nb - 2):
        assert torch.equal(k[:, page, :1000], k[:, nb - 1, :1000]) and torch.equal(v[:, page, :1000], v[:, nb - 1, :1000])
        assert (k[:, page, 1000:] == 0).all()


@pytest.mark.parametrize("kind", ["bf16"])
def test_serving_run(kind):
    """A prompt, three samples of it, two steps of shared decode on the pool's own tables, one sample leaves, the
    pool is compacted: every step's output is the formula's over the keys stored so far."""
    bs, hq, hkv, d, layers = 16, 8, 2, 64, 2
    nb, rows, width = 40, 8, 8
    k, v, _, _ = caches("bf16", layers, nb, bs, hkv, d, 9)
    dims = pa.make_dims(nb, bs, hq, hkv, d)
    pool = pa.page_pool(dims, k, v, rows, width)
    other = torch.empty(24, dtype=torch.int32, device="cuda")
    pa.pa_pool_append(dims, pool, i32([6]), i32([0, 24]), other)   # somebody else's pages come first
    n = 53
    slots = torch.empty(n, dtype=torch.int32, device="cuda")
    pa.pa_pool_append(dims, pool, i32([2]), i32([0, n]), slots)
    keys = {r: [[], []] for r in (2, 3, 4)}                         # what each row holds, K then V, per token
    new = [values((n, hkv, d), 20 + i) for i in range(2 * layers)]
    for layer in range(layers):
        pa.pa_store_kvcache(dims, new[2 * layer], new[2 * layer + 1], k[layer], v[layer], slots, n)
    for r in keys:
        keys[r] = [x.clone() for x in new]
    pa.pa_pool_fork(dims, pool, i32([2, 2]), i32([3, 4]))
    pa.pa_pool_free(dims, pool, i32([6]))
    live, ctx = [2, 3, 4], n
    for step in range(3):
        if step == 2:                                               # row 3 leaves, the others move together
            pa.pa_pool_free(dims, pool, i32([3]))
            live = [2, 4]
            pa.pa_pool_compact(dims, pool, torch.empty(nb, dtype=torch.int32, device="cuda"))
        B = len(live)
        one = torch.empty(B, dtype=torch.int32, device="cuda")
        pa.pa_pool_append(dims, pool, i32(live), i32(range(B + 1)), one)
        ctx += 1
        plan = pa.pa_pack_decode_shared(dims, [ctx] * B, shared_lens=[n // bs * bs], table_rows=live,
                                        max_blocks=width, split_tokens=128).upload()
        for layer in range(layers):
            kn, vn, q = (values((B, h, d), 50 + 10 * step + 3 * layer + i) for i, h in enumerate((hkv, hkv, hq)))
            pa.pa_store_kvcache(dims, kn, vn, k[layer], v[layer], one, B)
            out = torch.empty_like(q)
            pa.pa_decode_shared(dims, q, k[layer], v[layer], plan, d ** -0.5, out, pa.shared_workspace(plan),
                                block_tables=pool.block_tables)
            for i, r in enumerate(live):
                keys[r][2 * layer] = torch.cat([keys[r][2 * layer], kn[i:i + 1]])
                keys[r][2 * layer + 1] = torch.cat([keys[r][2 * layer + 1], vn[i:i + 1]])
            dense = [torch.stack([keys[r][2 * layer + j] for r in live]).reshape(B * ctx, 1, hkv, d) for j in (0, 1)]
            ref, a = reference(q, *dense, [range(i * ctx, (i + 1) * ctx) for i in range(B)], [ctx] * B, 1, d ** -0.5)
            assert_within(out, ref, a, f"step {step} layer {layer}")
    assert int((pool.ref_counts > 0).sum()) == n // bs + 2 and (pool.ref_counts[:n // bs + 2] > 0).all()


def test_order_with_the_launches_before():
    """A call may be set up during the launch before it: rows and counts that a kernel or a copy changes right
    before the call, and the state that the call before leaves, are the ones it reads."""
    dims, pool, m = both("bf16", layers=2, nb=200, rows=24, width=6, seed=77)
    rows, cu, slots = i32([0] * 4), i32([0] * 5), torch.zeros(4 * 37, dtype=torch.int32, device="cuda")
    remap = torch.empty(200, dtype=torch.int32, device="cuda")
    pinned = torch.zeros(4, dtype=torch.int32).pin_memory()
    rng = np.random.default_rng(78)
    torch.cuda.synchronize()
    for step in range(40):
        some = [int(x) for x in rng.permutation(12)[:4]]
        want = i32(some)
        if step % 2:
            rows.copy_(want)
        else:
            torch.cuda.synchronize()  # (the copy before has read the pinned words)
            pinned.copy_(torch.tensor(some, dtype=torch.int32))
            rows.copy_(pinned, non_blocking=True)
        pa.pa_pool_free(dims, pool, rows)
        m.free(some)
        torch.mul(torch.arange(5, dtype=torch.int32, device="cuda"), 1 + step % 37, out=cu)
        n = 4 * (1 + step % 37)
        pa.pa_pool_append(dims, pool, rows, cu, slots[:n])
        m.append(some, [1 + step % 37] * 4)
        parents = rows.clone()
        torch.add(rows, 12, out=rows)
        pa.pa_pool_free(dims, pool, rows)
        m.free([x + 12 for x in some])
        pa.pa_pool_fork(dims, pool, parents, rows)
        assert m.fork(some, [x + 12 for x in some])
        if step % 5 == 4:
            pa.pa_pool_compact(dims, pool, remap)
            m.compact()
    torch.cuda.synchronize()
    assert pa.pa_read_device_error() == 0
    assert_same(pool, m, "end")
    m.check()


@pytest.mark.parametrize("nb", [31, 32, 33, 1023, 1024, 1025, 2049, 8193, 16383, 16384, 16385, 32768, 32769, 131072, 131073])
def test_sizes_around_the_words_and_rounds_of_ids(nb):
    """A search and a compaction where warps, CTAs and rounds end, with the border between kept and moved pages at
    and beside a word's ends."""
    for used in sorted({1, min(32, nb), min(33, nb), nb // 2 // 32 * 32 or 1, nb // 2 + 1, nb - 1, nb}):
        dims, pool, m = both(layers=1, nb=nb, bs=16, hkv=1, d=64, rows=3, width=max(nb, 4), seed=6)
        rng = np.random.default_rng(nb * 7 + used)
        ids = np.sort(rng.permutation(nb)[:used]).astype(np.int32)
        m.tables[0, :used], m.ctx[0], m.refs[ids] = ids, 16 * used, 1
        pool.block_tables.copy_(i32(m.tables)), pool.context_lens.copy_(i32(m.ctx)), pool.ref_counts.copy_(i32(m.refs))
        n = min(nb - used, 70)
        assert append(dims, pool, m, [1], [16 * n])
        assert np.array_equal(pool.block_tables[1].cpu().numpy(), m.tables[1])
        pa.pa_pool_free(dims, pool, i32([1]))
        m.free([1])
        if used < nb:  # one page too many is refused
            assert not append(dims, pool, m, [1], [16 * (nb - used) + 1])
            assert pa.pa_read_device_error() == NO_ROOM
        remap = torch.empty(nb, dtype=torch.int32, device="cuda")
        pa.pa_pool_compact(dims, pool, remap)
        assert np.array_equal(remap.cpu().numpy(), m.compact())
        assert_same(pool, m, f"compact {nb} {used}")
