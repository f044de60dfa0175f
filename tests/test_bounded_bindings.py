"""CPU tests of what the decodes over a bounded cache refuse: the binding (shapes, types) and the library (arguments)."""
import ctypes

import pytest
import torch

from paged_kv_cache_kvcache_gb300 import pagedattn as pa

DIMS = (6, 16, 4, 2, 64)
BF = torch.bfloat16


class Recorder:
    """In the library's place: notes the calls that get through."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append(name) or pa.PA_OK


@pytest.fixture
def calls(monkeypatch):
    recorder = Recorder()
    monkeypatch.setattr(pa, "_lib", recorder)
    monkeypatch.setattr(pa, "_device", lambda: -1)  # where the host's tensors are
    return recorder.calls


def tensors(int8):
    nb, bs, hq, hkv, d = DIMS
    cache = torch.int8 if int8 else BF
    t = {"q": torch.zeros(3, hq, d, dtype=BF), "k": torch.zeros(nb, bs, hkv, d, dtype=cache),
         "v": torch.zeros(nb, bs, hkv, d, dtype=cache)}
    if int8:
        t.update(ks=torch.zeros(nb, hkv, bs, dtype=torch.float16), vs=torch.zeros(nb, hkv, bs, dtype=torch.float16))
    t.update(table=torch.zeros(3, 2, dtype=torch.int32), ctx=torch.zeros(3, dtype=torch.int32))
    return t


def window(t, out=None, **kw):
    f = pa.pa_decode_window_int8 if "ks" in t else pa.pa_decode_window
    f(pa.make_dims(*DIMS), *t.values(), 8, 2, 0.1, torch.zeros_like(t["q"]) if out is None else out, stream=0, **kw)


def weights(t, out=None, scores=None, **kw):
    f = pa.pa_decode_weights_int8 if "ks" in t else pa.pa_decode_weights
    scores = torch.zeros(3, 2, 32) if scores is None else scores
    f(pa.make_dims(*DIMS), *t.values(), 0.1, torch.zeros_like(t["q"]) if out is None else out, scores,
      torch.empty(4096, dtype=torch.uint8), stream=0, **kw)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("call", [window, weights])
def test_wrong_tensors_are_refused(calls, call, int8):
    good = tensors(int8)
    call(good)
    call(good, table_rows=torch.zeros(3, dtype=torch.int32))
    assert len(calls) == 2
    bad = {"q": good["q"].float(), "k": good["k"][:5], "v": good["v"].half(), "table": good["table"].long(),
           "ctx": good["ctx"][:2]}
    if int8:
        bad.update(ks=good["ks"].float(), vs=good["vs"][:2])
    for name, x in bad.items():
        with pytest.raises(ValueError):
            call({**good, name: x})
    with pytest.raises(ValueError):
        call({**good, "q": torch.zeros(3, 64, 4, dtype=BF).transpose(1, 2)})
    with pytest.raises(ValueError):
        call({**good, "table": torch.zeros(2, 3, dtype=torch.int32).t()})
    with pytest.raises(ValueError):
        call(good, out=torch.zeros(3, 4, 64))
    with pytest.raises(ValueError):
        call(good, out=torch.zeros(2, 4, 64, dtype=BF))
    with pytest.raises(ValueError):  # more sequences than rows, and no rows named
        call({**good, "q": torch.zeros(4, 4, 64, dtype=BF)})
    with pytest.raises(ValueError):
        call(good, table_rows=torch.zeros(2, dtype=torch.int32))
    assert len(calls) == 2


def test_wrong_scores_are_refused(calls):
    good = tensors(False)
    for bad in (torch.zeros(3, 2, 31), torch.zeros(3, 2, 32, dtype=torch.float64), torch.zeros(2, 2, 32),
                torch.zeros(3, 32, 2).transpose(1, 2)):
        with pytest.raises(ValueError):
            weights(good, scores=bad)
        with pytest.raises(ValueError):
            weights(good, scores_out=bad)
    assert calls == []


def test_library_refusals():
    L = pa.lib()

    def rc(fn="window", seqs=1, rows=1, width=2, w=8, sinks=0, scale=0.1, decay=1.0, q=64, out=64, scores=64, table=None,
           blocks=6, ws=256, ws_bytes=1 << 20, bs=16, ks=64, int8=False):
        d = ctypes.byref(pa.make_dims(blocks, bs, *DIMS[2:]))
        f = ctypes.c_float
        head = (d, q, 64, 64, *((ks, 64) if int8 else ()), 64, 64, table, seqs, rows, width)
        i8 = "_int8" if int8 else ""
        if fn == "window":
            return getattr(L, "pa_decode_window" + i8)(*head, w, sinks, f(scale), out, None)
        return getattr(L, "pa_decode_weights" + i8)(*head, f(scale), f(decay), scores, 64, out, ws, ws_bytes, None)

    bad, no = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED
    for fn in ("window", "weights"):
        for int8 in (False, True):
            assert rc(fn, seqs=0, int8=int8) == pa.PA_OK
            for kw in (dict(seqs=-1), dict(rows=0), dict(width=0), dict(seqs=2), dict(scale=0.0), dict(scale=float("nan")),
                       dict(scale=float("inf")), dict(q=None), dict(q=72), dict(out=8), dict(blocks=0)):
                assert rc(fn, int8=int8, **kw) == bad, (fn, kw)
            assert rc(fn, width=2 ** 27, int8=int8) == no
            assert rc(fn, seqs=2 ** 28, rows=2 ** 28, int8=int8) == no
            assert rc(fn, bs=24, int8=int8) == no
        assert rc(fn, int8=True, ks=None) == bad and rc(fn, int8=True, ks=40) == bad
    assert rc(w=0) == bad and rc(sinks=-1) == bad
    for kw in (dict(decay=-0.1), dict(decay=1.5), dict(decay=float("nan")), dict(scores=None), dict(ws=None), dict(ws=64)):
        assert rc("weights", **kw) == bad, kw
    need = ctypes.c_uint64()
    d = pa.make_dims(*DIMS)
    assert L.pa_decode_weights_workspace(ctypes.byref(d), 3, 2, ctypes.byref(need)) == pa.PA_OK
    assert need.value == 3 * 2 * 32 * 4 * 4
    assert rc("weights", ws_bytes=2 * 32 * 4 * 4 - 1) == pa.PA_ERR_WORKSPACE
    assert L.pa_decode_weights_workspace(ctypes.byref(d), -1, 2, ctypes.byref(need)) == bad
    assert L.pa_decode_weights_workspace(ctypes.byref(d), 1, 2, None) == bad


@pytest.mark.parametrize("int8", [False, True])
def test_prefill_window_refusals(int8):
    L = pa.lib()
    dims = pa.make_dims(*DIMS)
    plan = pa.pa_pack_prefill(dims, [20, 5], [20, 5], [[0, 1], [2]], pin=False)

    def rc(window=8, sinks=0, scale=0.1, q=64, ws_bytes=1 << 30, meta=True):
        m = ctypes.byref(plan.meta) if meta else None
        head = (ctypes.byref(dims), q, 64, 64, *((64, 64) if int8 else ()), 64, 64, 64, *((64, 64) if int8 else ()), window,
                sinks, ctypes.c_float(scale), 64, m, 64)
        return L.pa_prefill_window_int8(*head, 64, ws_bytes, None) if int8 else L.pa_prefill_window(*head, None)

    for kw in (dict(window=0), dict(window=-1), dict(sinks=-1), dict(scale=0.0), dict(q=None), dict(q=8), dict(meta=False)):
        assert rc(**kw) == pa.PA_ERR_INVALID_ARG, kw
    if int8:
        assert rc(ws_bytes=16) == pa.PA_ERR_WORKSPACE
    empty = pa.pa_pack_prefill(dims, [5], [0], [[0]], pin=False)
    plan.meta = empty.meta
    assert rc() == pa.PA_OK


def test_evict_library_refusals():
    L = pa.lib()
    need = ctypes.c_uint64()
    d0 = pa.make_dims(*DIMS)
    assert L.pa_pool_workspace(ctypes.byref(d0), ctypes.byref(pa.pa_pool(5, 4, 1)), ctypes.byref(need)) == pa.PA_OK

    def rc(n=1, budget=8, first=0, last=0, rows=64, scores=64, out=64, kept=64, ws=256, ws_bytes=need.value, dims=DIMS,
           **pool):
        fields = dict(num_rows=5, max_blocks=4, num_layers=1, block_tables=64, context_lens=64, ref_counts=64, k_cache=64,
                      v_cache=64) | pool
        d, p = pa.make_dims(*dims), pa.pa_pool(**fields)
        return L.pa_pool_evict(ctypes.byref(d), ctypes.byref(p), rows, n, scores, out, budget, first, last, kept, ws, ws_bytes,
                               None)

    bad = pa.PA_ERR_INVALID_ARG
    assert rc(n=0) == pa.PA_OK
    for kw in (dict(n=-1), dict(n=6), dict(budget=0), dict(budget=-3), dict(first=-1), dict(last=-1), dict(first=5, last=4),
               dict(first=2 ** 31 - 1, last=2 ** 31 - 1), dict(rows=None), dict(scores=None), dict(out=None), dict(kept=None),
               dict(ws=None), dict(ws=64), dict(k_cache=None), dict(v_cache=8), dict(k_scale=64), dict(ref_counts=4),
               dict(num_rows=0), dict(num_layers=2, layer_stride=8)):
        assert rc(**kw) == bad, kw
    assert rc(ws_bytes=need.value - 1) == pa.PA_ERR_WORKSPACE
    assert rc(max_blocks=2 ** 28, dims=(6, 16, 4, 2, 64)) == pa.PA_ERR_UNSUPPORTED
    assert rc(max_blocks=2 ** 27 - 1, dims=(6, 16, 4, 2, 64)) == pa.PA_ERR_UNSUPPORTED  # a row of nearly 2^31 tokens
    assert rc(dims=(6, 24, 4, 2, 64)) == pa.PA_ERR_UNSUPPORTED
