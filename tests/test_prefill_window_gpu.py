"""pa_prefill_window(_int8) against its formula in 64 bits.

The cache holds NaN and infinities wherever no query looks; the plan names such a page where a table entry is not needed."""
import numpy as np
import pytest
import torch

from paged_kv_cache_kvcache_gb300 import pagedattn as pa
from tests.bounded_model import Case, near, seen

pytestmark = pytest.mark.gpu

EVERYTHING = 2 ** 31 - 1
HEADS = [(16, 8, 128), (28, 4, 128), (12, 1, 64), (7, 1, 128), (8, 8, 128), (4, 2, 64), (16, 1, 128)]
CASES = [  # (length, new tokens) of each sequence, window, sinks, block size
    ([(1, 1), (2, 2), (17, 17), (5, 0), (130, 1)], 1, 0, 16),
    ([(300, 300), (129, 128)], 16, 4, 16),
    ([(700, 50), (400, 400), (33, 33)], 100, 130, 32),
    ([(1000, 1), (777, 3)], 128, 1, 256),
    ([(600, 600)], 255, 257, 64),
    ([(500, 200)], EVERYTHING, 0, 16),
    ([(900, 100), (20, 20)], 300, EVERYTHING, 128),
    ([(1400, 300)], 1000, 200, 1024),
]
MANY = [([(1600, 1600)], 200, 4, 16), ([(900, 700), (1200, 500)], 333, 150, 128)]  # more work items than SMs


def model(c, q, new):
    """(out, size) of the packed queries."""
    out, size, at = np.zeros(q.shape), np.zeros(q.shape), 0
    x, g = q.double().numpy(), c.hq // c.hkv
    for n, lq, slots in zip(c.lens, new, c.slots):
        mask = np.stack([seen(n, n - lq + i, c.window, c.sinks) for i in range(lq)]) if lq else np.zeros((0, n), bool)
        for h in range(c.hq):
            k, v = c.kd[slots, h // g], c.vd[slots, h // g]
            cols = mask.any(0)
            s = np.where(mask[:, cols], x[at:at + lq, h] @ k[cols].T * c.scale, -np.inf)
            if lq:
                p = np.exp(s - s.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                out[at:at + lq, h], size[at:at + lq, h] = p @ v[cols], p @ np.abs(v[cols])
        at += lq
    return out, size


def run(seqs, window, sinks, bs, heads, int8, seed):
    lens, new = [n for n, _ in seqs], [m for _, m in seqs]
    c = Case(lens, *heads, bs, window, sinks, int8, seed=seed, first_new=[n - m for n, m in seqs])
    if int8:  # a prompt reads code * scale as bf16
        c.kd, c.vd = (torch.tensor(x).to(torch.bfloat16).double().numpy() for x in (c.kd, c.vd))
    unseen = np.setdiff1d(np.arange(c.blocks), c.table[c.table >= 0])
    lists = [np.where(t[:-(-n // bs)] < 0, unseen[0], t[:-(-n // bs)]) for t, n in zip(c.table, lens)]
    q = torch.randn(sum(new), c.hq, c.d, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)
    plan = pa.pa_pack_prefill(c.dims, lens, new, lists).upload()
    out = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device="cuda")
    if int8:
        ws = pa.prefill_workspace(plan).fill_(255)  # NaN wherever nothing is written
        pa.pa_prefill_window_int8(c.dims, q.cuda(), *c.gpu, plan, window, sinks, c.scale, out, ws)
    else:
        pa.pa_prefill_window(c.dims, q.cuda(), *c.gpu, plan, window, sinks, c.scale, out)
    near(out, *model(c, q, new))
    return c, q, plan, out


@pytest.mark.parametrize("int8", [False, True], ids=["bf16", "int8"])
@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "-".join(map(str, h)))
def test_prefill_window(heads, case, int8):
    run(*CASES[case], heads, int8, seed=case)


@pytest.mark.parametrize("int8", [False, True], ids=["bf16", "int8"])
@pytest.mark.parametrize("case", range(len(MANY)))
@pytest.mark.parametrize("heads", [(28, 4, 128), (16, 2, 64)], ids=lambda h: "-".join(map(str, h)))
def test_many_work_items(heads, case, int8):
    run(*MANY[case], heads, int8, seed=case)


def test_a_wide_window_is_the_prefill_without_one_and_a_plan_serves_both():
    c, q, plan, out = run([(1100, 900), (300, 300)], EVERYTHING, 0, 16, (28, 4, 128), False, 3)
    plain = torch.empty_like(out)
    pa.pa_prefill_varlen(c.dims, q.cuda(), *c.gpu, plan, c.scale, plain)
    assert torch.equal(out, plain)
    pa.pa_prefill_window(c.dims, q.cuda(), *c.gpu, plan, 5, EVERYTHING, c.scale, out)  # everything is a first token
    assert torch.equal(out, plain)
    pa.pa_prefill_window(c.dims, q.cuda(), *c.gpu, plan, 1, 0, c.scale, out)  # only itself
    own = np.concatenate([c.vd[s[-m:]] for s, m in zip(c.slots, (900, 300))]).repeat(7, 1)
    near(out, own, np.abs(own))


def test_captured_and_on_another_stream():
    c, q, plan, out = run([(800, 800)], 100, 4, 16, (16, 8, 128), False, 4)
    want = out.clone()
    qc, st, graph = q.cuda(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    out.zero_()
    torch.cuda.synchronize()
    pa.pa_prefill_window(c.dims, qc, *c.gpu, plan, 100, 4, c.scale, out, stream=st)
    st.synchronize()
    assert torch.equal(out, want)
    with torch.cuda.graph(graph):
        for _ in range(3):
            pa.pa_prefill_window(c.dims, qc, *c.gpu, plan, 100, 4, c.scale, out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("int8", [False, True], ids=["bf16", "int8"])
def test_a_few_queries_far_into_long_sequences(int8):
    run([(70000, 40), (33000, 200), (65537, 1)], 300, 10, 16, (4, 1, 64), int8, 7)


@pytest.mark.parametrize("int8", [False, True], ids=["bf16", "int8"])
@pytest.mark.parametrize("heads", [(16, 8, 128), (4, 2, 64)], ids=lambda h: "-".join(map(str, h)))
def test_behind_the_launch_that_writes_its_queries_and_keys(heads, int8):
    """Rotation and store, prefill and a step of decode without a pause, many times over: as with one after each call."""
    (hq, hkv, d), bs, lens, window, sinks = heads, 16, [700, 33, 1200], 300, 20
    blocks = sum(-(-n // bs) for n in lens)
    dims = pa.make_dims(blocks, bs, hq, hkv, d)
    g = np.random.default_rng(3)
    ids = np.split(g.permutation(blocks), np.cumsum([-(-n // bs) for n in lens])[:-1])
    at = [i[np.arange(n) // bs] * bs + np.arange(n) % bs for i, n in zip(ids, lens)]
    slots = torch.tensor(np.concatenate(at), dtype=torch.int32, device="cuda")
    pos = torch.tensor(np.concatenate([np.arange(n) for n in lens]), dtype=torch.int32, device="cuda")
    table = np.zeros((len(lens), max(map(len, ids))), np.int32)
    for row, i in zip(table, ids):
        row[:len(i)] = i
    table, ctx = torch.tensor(table, device="cuda"), torch.tensor(lens, dtype=torch.int32, device="cuda")
    plan = pa.pa_pack_prefill(dims, lens, lens, [list(i) for i in ids]).upload()
    ws = pa.prefill_workspace(plan) if int8 else None
    angle = torch.arange(2000)[:, None] * 1e4 ** (-torch.arange(d // 2) / (d // 2))
    rope = pa.Rope(dims, torch.cat([angle.cos(), angle.sin()], 1).float().contiguous().cuda())
    caches = pa.int8_cache(dims) if int8 else tuple(torch.zeros(blocks, bs, hkv, d, dtype=torch.bfloat16, device="cuda")
                                                    for _ in range(2))
    store, prefill, decode = ((pa.pa_rope_store_int8, pa.pa_prefill_window_int8, pa.pa_decode_window_int8) if int8 else
                              (pa.pa_rope_store, pa.pa_prefill_window, pa.pa_decode_window))
    scale = d ** -0.5
    gen = torch.Generator("cuda").manual_seed(1)
    rounds = [torch.randn(sum(lens), hq + 2 * hkv, d, device="cuda", generator=gen).to(torch.bfloat16) for _ in range(12)]

    def go(pause):
        outs = []
        for x in rounds:
            q, out = (torch.empty(sum(lens), hq, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            step = torch.empty(len(lens), hq, d, dtype=torch.bfloat16, device="cuda")
            pause()
            store(dims, rope, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], pos, slots, q, *caches)
            pause()
            prefill(dims, q, *caches, plan, window, sinks, scale, out, *([ws] if int8 else []))
            pause()
            decode(dims, x[:len(lens), :hq].contiguous(), *caches, table, ctx, window, sinks, scale, step)
            pause()
            outs += [q, out, step]
        torch.cuda.synchronize()
        return outs

    want = go(torch.cuda.synchronize)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(go(lambda: None), want))
    # the last round against the formula, on what the cache holds
    kv = [c.flatten(0, 1).double().cpu().numpy() for c in caches[:2]]
    if int8:  # code * scale: as bf16 for the prompts
        kv = [c * s.transpose(1, 2).flatten(0, 1).double().cpu().numpy()[..., None] for c, s in zip(kv, caches[2:])]
        kv = [torch.tensor(c).to(torch.bfloat16).double().numpy() for c in kv]
    c = Case.__new__(Case)
    c.hq, c.hkv, c.lens, c.slots, c.window, c.sinks, c.scale, c.kd, c.vd = hq, hkv, lens, at, window, sinks, scale, *kv
    out, size = model(c, want[-3].cpu(), lens)
    near(want[-2], out, size)
