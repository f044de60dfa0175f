"""A windowed prefill right behind the launch that writes its work list and block table."""
import numpy as np
import pytest
import torch

from paged_kv_cache_kvcache_gb300 import pagedattn as pa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("int8", [False, True], ids=["bf16", "int8"])
@pytest.mark.parametrize("lens", [[700, 33, 1200], [900] * 40], ids=["few", "many"])
def test_a_plan_that_the_launch_ahead_writes(lens, int8):
    """Plans of two orders of the pages and of the sequences come in turn into the one that the calls read; each call
    gives what it gives with a pause on both sides, bit for bit."""
    hq, hkv, d, bs, new = 8, 2, 64, 16, [min(n, 300) for n in lens]
    pages = [-(-n // bs) for n in lens]
    dims = pa.make_dims(sum(pages) + 3, bs, hq, hkv, d)
    r = np.random.default_rng(2)
    plans = []
    for _ in range(2):
        lists = np.split(r.permutation(dims.num_blocks)[:sum(pages)], np.cumsum(pages)[:-1])
        plans.append(pa.pa_pack_prefill(dims, lens, new, [list(x) for x in lists]).upload())
    to = pa.pa_pack_prefill(dims, lens, new, [list(x) for x in lists]).upload()
    shape = (dims.num_blocks, bs, hkv, d)
    if int8:
        caches = [torch.randint(-127, 128, shape, dtype=torch.int8, device="cuda") for _ in range(2)] + \
            [torch.full((dims.num_blocks, hkv, bs), 0.02, dtype=torch.float16, device="cuda") for _ in range(2)]
        ws = [pa.prefill_workspace(to)]
        call = pa.pa_prefill_window_int8
    else:
        caches = [torch.randn(shape, device="cuda").to(torch.bfloat16) for _ in range(2)]
        ws, call = [], pa.pa_prefill_window
    q = torch.randn(sum(new), hq, d, device="cuda").to(torch.bfloat16)

    def go(pause):
        outs = []
        for i in range(20):
            out = torch.empty_like(q)
            pause()
            torch.bitwise_or(plans[i % 2].dev, 0, out=to.dev)  # a kernel, not a copy
            pause()
            call(dims, q, *caches, to, 100, 4, d ** -0.5, out, *ws)
            pause()
            outs.append(out)
        torch.cuda.synchronize()
        return outs

    want = go(torch.cuda.synchronize)
    assert not torch.equal(want[0], want[1])
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(go(lambda: None), want))
