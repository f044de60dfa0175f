"""The word by which own parts that run beside the products learn that the launches before them have ended."""
import numpy as np
import pytest
import torch

from paged_kv_cache_kvcache_gb300 import pagedattn as pa
from tests.test_shared_pack import make_batch

BS, HEADS = 16, (28, 4, 128)
PLANS = {  # group sizes, shared blocks, tails: is there a word?
    "beside": (([90], [30], [1 + 7 * i for i in range(90)]), True),
    # contexts that are all prefix, and short ones that share nothing: nothing to merge
    "beside, one part each": (([400] + [1] * 100, [8] + [0] * 100, [0] * 400 + [20 + i for i in range(100)]), True),
    "nothing shared": (([300], [0], [200 + i for i in range(300)]), False),
    "prefix only": (([400], [8], [0] * 400), False),
    "in the lanes": (([4], [40], [60, 200, 33, 1]), False),
}


def make(name, **kw):
    (sizes, sh, tails), word = PLANS[name]
    ctx, lists, groups, nb = make_batch(71, sizes, sh, tails, BS)
    dims = pa.make_dims(nb, BS, *HEADS)
    plan = pa.pa_pack_decode_shared(dims, ctx, groups, block_lists=lists, split_tokens=128, **kw)
    assert plan.meta.merge == (name not in ("beside, one part each", "prefix only"))
    return dims, plan, ctx, lists, nb, word


def results_bytes(m):
    up = lambda x: (x + 255) // 256 * 256
    return up(m.num_partials * HEADS[0] * HEADS[2] * 4) + up(m.num_partials * HEADS[0] * 4)


@pytest.mark.parametrize("name", PLANS)
def test_a_workspace_holds_the_word_where_there_is_a_launch_beside(name):
    _, plan, _, _, _, word = make(name, pin=False)
    m = plan.meta
    assert word == (m.apart == 1 and m.num_items > 0 and m.num_single_items > 0)
    assert m.workspace_bytes == results_bytes(m) + (256 if word else 0)
    scratch = m.num_scratch_tiles * 128 * HEADS[1] * HEADS[2] * 4
    scratch += (m.num_seqs * HEADS[0] * HEADS[2] * 2 + 255) // 256 * 256 if scratch else 0
    assert m.workspace_bytes_int8 == m.workspace_bytes + scratch


@pytest.mark.gpu
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("name", ["beside", "beside, one part each"])
def test_the_word_is_taken_back(name, int8):
    """A call leaves the word at 0, whatever the workspace held, so that a replayed call, which gives the same word
    again, waits for it again; calls that share a workspace one after another, two graphs among them, and calls on two
    streams with one each keep their results."""
    from tests.test_shared_decode_gpu import assert_within, int8_pool, pool, reference, values
    dims, plan, ctx, lists, nb, _ = make(name)
    plan.upload()
    hq, hkv, d = HEADS
    n = len(ctx)
    if int8:
        cache, dense = int8_pool(nb, BS, hkv, d, 72, ctx, lists)
    else:
        cache = dense = pool(nb, BS, hkv, d, 72, ctx, lists)
    call = pa.pa_decode_shared_int8 if int8 else pa.pa_decode_shared
    qs = [values((n, hq, d), 73 + i) for i in range(2)]
    at = results_bytes(plan.meta)
    want = []
    for i, fill in enumerate((0xFF, 0)):
        ws = pa.shared_workspace(plan)
        ws.fill_(fill)
        out = torch.full_like(qs[0], 7.0)
        call(dims, qs[i], *cache, plan, d ** -0.5, out, ws)
        torch.cuda.synchronize()
        assert (ws[at:at + 8] == 0).all()
        assert_within(out, *reference(qs[i], *dense, lists, ctx, BS, d ** -0.5), f"{name} {fill}")
        want.append(out)
    q, graphs, outs = qs[0].clone(), [], [torch.empty_like(qs[0]) for _ in range(2)]
    for out in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(dims, q, *cache, plan, d ** -0.5, out, ws)
            call(dims, q, *cache, plan, d ** -0.5, out, ws)
        graphs.append(g)
    for step in range(6):
        q.copy_(qs[step & 1])
        for g, out in zip(graphs, outs):
            out.fill_(7.0)
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, want[step & 1]) for out in outs) and (ws[at:at + 8] == 0).all()
    streams, wss = [torch.cuda.Stream() for _ in range(2)], [pa.shared_workspace(plan) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(8):
        for i in range(2):
            call(dims, qs[i], *cache, plan, d ** -0.5, outs[i], wss[i], stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(outs[i], want[i]) for i in range(2))
    assert pa.pa_read_device_error() == 0
