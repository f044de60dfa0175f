"""CPU tests of arguments of the calls over a bounded cache that the bindings pass on, in 32 bits, or refuse."""
import pytest
import torch

from paged_kv_cache_kvcache_gb300 import pagedattn as pa
from tests import rope_model

DIMS = (6, 16, 4, 2, 64)
BF = torch.bfloat16
MOST = 2 ** 31 - 1


class Recorder:
    """In the library's place: notes the calls that get through."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args)) or pa.PA_OK


@pytest.fixture
def calls(monkeypatch):
    recorder = Recorder()
    monkeypatch.setattr(pa, "_lib", recorder)
    monkeypatch.setattr(pa, "_device", lambda: -1)  # where the host's tensors are
    return recorder.calls


def cache(int8):
    nb, bs, _, hkv, d = DIMS
    pages = [torch.zeros(nb, bs, hkv, d, dtype=torch.int8 if int8 else BF) for _ in range(2)]
    return pages + [torch.zeros(nb, hkv, bs, dtype=torch.float16) for _ in range(2 if int8 else 0)]


@pytest.mark.parametrize("int8", [False, True])
def test_positions_of_other_shapes_are_refused(calls, int8):
    dims, n = pa.make_dims(*DIMS), 3
    q, k, v, out = (torch.zeros(n, h, 64, dtype=BF) for h in (4, 2, 2, 4))
    slots = torch.zeros(n, dtype=torch.int32)

    def call(axes, *shape):
        rope = pa.Rope(dims, rope_model.table(10, 64), axes=axes, pair_axis=[i % axes for i in range(32)])
        f = pa.pa_rope_store_int8 if int8 else pa.pa_rope_store
        f(dims, rope, q, k, v, torch.zeros(shape, dtype=torch.int32), slots, out, *cache(int8), stream=0)

    for good in ((1, n), (1, 1, n), (1, n, 1), (2, 2, n), (2, 2 * n), (4, 4, n), (4, 2, 2, n)):
        call(*good)  # the tokens of an axis lie side by side
    assert len(calls) == 7
    for bad in ((2, n, 2), (4, n, 4), (4, n, 2, 2), (2, n), (1, n + 1), (2, 2, n + 1)):
        with pytest.raises(ValueError):
            call(*bad)
    assert len(calls) == 7


@pytest.mark.parametrize("int8", [False, True])
def test_windows_past_32_bits_are_everything(calls, int8):
    """An int of C takes the low 32 bits of what it is given: 2^32 + 5 was a window of 5."""
    dims, n = pa.make_dims(*DIMS), 3
    q, table, ctx = torch.zeros(n, 4, 64, dtype=BF), torch.zeros(n, 2, dtype=torch.int32), torch.zeros(n, dtype=torch.int32)
    f = pa.pa_decode_window_int8 if int8 else pa.pa_decode_window
    for x, want in ((8, 8), (MOST, MOST), (2 ** 31, MOST), (2 ** 32 + 5, MOST), (2 ** 63, MOST)):
        f(dims, q, *cache(int8), table, ctx, x, x, 0.1, torch.zeros_like(q), stream=0)
        assert calls[-1][1][-5:-3] == (want, want)
    f(dims, q, *cache(int8), table, ctx, 5 - 2 ** 32, -2 ** 40, 0.1, torch.zeros_like(q), stream=0)
    assert all(x < 0 for x in calls[-1][1][-5:-3])  # which the library refuses


def test_first_and_last_tokens_past_32_bits_are_refused(calls):
    """first = 2^32 + 4 was 4."""
    dims, n = pa.make_dims(*DIMS), 2
    table, ctx, refs = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32), torch.zeros(6, dtype=torch.int32)
    pool = object.__new__(pa.PagePool)
    pool.dims, pool.dims_ref, pool.ref, pool.ws, pool.device, pool.block_tables = dims, 1, 1, (256, 1), -1, table
    pool.check = lambda dims: None
    rows, kept = torch.zeros(n, dtype=torch.int32), torch.zeros(n, 8, dtype=torch.int32)
    scores = torch.zeros(4, 2, 32)

    def call(first, last):
        pa.pa_pool_evict(dims, pool, rows, scores, 8, kept, first=first, last=last, stream=0)
        return calls[-1][1][7:9]

    assert call(3, 2) == (3, 2)
    assert call(2 ** 32 + 4, 2 ** 40) == (MOST, MOST)  # more than the budget: refused
    assert all(x < 0 for x in call(4 - 2 ** 32, -2 ** 40))


@pytest.mark.parametrize("int8", [False, True])
def test_prefill_window_refuses_wrong_tensors_and_dims(monkeypatch, int8):
    """What it took for the plan's tensors, whatever their type, shape, strides and device."""
    dims = pa.make_dims(*DIMS)
    plan = pa.pa_pack_prefill(dims, [20, 5], [7, 5], [[0, 1], [2]], pin=False)
    plan.dev = torch.zeros(int(plan.meta.total_bytes), dtype=torch.uint8)
    recorder = Recorder()
    monkeypatch.setattr(pa, "_lib", recorder)
    monkeypatch.setattr(pa, "_device", lambda: -1)
    calls, f = recorder.calls, pa.pa_prefill_window_int8 if int8 else pa.pa_prefill_window
    good = {"q": torch.zeros(12, 4, 64, dtype=BF), "out": torch.zeros(12, 4, 64, dtype=BF)}
    good.update(zip(("k", "v", "ks", "vs"), cache(int8)))
    ws = [torch.zeros(max(256, int(plan.meta.workspace_bytes)), dtype=torch.uint8)] if int8 else []

    def call(dims=dims, plan=plan, ws=ws, **kw):
        t = {**good, **kw}
        f(dims, t["q"], t["k"], t["v"], *((t["ks"], t["vs"]) if int8 else ()), plan, 8, 2, 0.1, t["out"], *ws, stream=0)

    call()
    nb, bs, hq, hkv, d = DIMS
    call(k=torch.zeros(8, bs, hkv, d, dtype=good["k"].dtype))  # more pages than the dims name
    call(q=torch.zeros(12, 256, dtype=BF), out=torch.zeros(16, 4, 64, dtype=BF))  # a bucket's rows
    call(dims=pa.make_dims(nb + 1, bs, hq, hkv, d), k=torch.zeros(7, bs, hkv, d, dtype=good["k"].dtype),
         v=torch.zeros(7, bs, hkv, d, dtype=good["k"].dtype), **({x: torch.zeros(7, hkv, bs, dtype=torch.float16)
                                                                 for x in ("ks", "vs")} if int8 else {}))
    assert len(calls) == 4
    bad = [dict(q=good["q"].float()), dict(q=good["q"].half()), dict(q=good["q"][:11]),
           dict(q=torch.zeros(12, 64, 4, dtype=BF).transpose(1, 2)), dict(out=good["out"].float()),
           dict(out=torch.zeros(24, 4, 64, dtype=BF)[::2]), dict(out=good["out"][:11]), dict(k=good["k"][:5]),
           dict(v=good["v"].float()), dict(v=good["v"].transpose(1, 2)),
           dict(dims=pa.make_dims(nb + 1, bs, hq, hkv, d)), dict(dims=pa.make_dims(nb - 1, bs, hq, hkv, d)),
           dict(dims=pa.make_dims(nb, 32, hq, hkv, d)),
           dict(dims=pa.make_dims(nb, bs, hkv, hq, d)), dict(dims=pa.make_dims(nb, bs, 2 * hq, 2 * hkv, d))]
    if int8:
        bad += [dict(ks=good["ks"].float()), dict(vs=good["vs"][:5]), dict(ws=[torch.zeros(1 << 20, dtype=torch.uint8)[::2]])]
    for kw in bad:
        with pytest.raises(ValueError):
            call(**kw)
    monkeypatch.setattr(pa, "_device", lambda: 0)  # the tensors and the plan are elsewhere
    with pytest.raises(ValueError):
        call()
    assert len(calls) == 4
