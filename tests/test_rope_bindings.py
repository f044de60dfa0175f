"""CPU tests of pa_rope_store's refusals: by the binding (shapes, types, strides) and by the library (arguments)."""
import ctypes

import pytest
import torch

from paged_kv_cache_kvcache_gb300 import pagedattn as pa
from tests import rope_model

DIMS = (6, 16, 4, 2, 64)
BF = torch.bfloat16


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


def tensors(int8, n=3):
    nb, bs, hq, hkv, d = DIMS
    cache = torch.int8 if int8 else BF
    t = {"q": torch.zeros(n, hq, d, dtype=BF), "k": torch.zeros(n, hkv, d, dtype=BF), "v": torch.zeros(n, hkv, d, dtype=BF),
         "positions": torch.zeros(n, dtype=torch.int32), "slots": torch.zeros(n, dtype=torch.int32),
         "out": torch.zeros(n, hq, d, dtype=BF), "kc": torch.zeros(nb, bs, hkv, d, dtype=cache),
         "vc": torch.zeros(nb, bs, hkv, d, dtype=cache)}
    if int8:
        t.update(ks=torch.zeros(nb, hkv, bs, dtype=torch.float16), vs=torch.zeros(nb, hkv, bs, dtype=torch.float16))
    return t


def call(t, rope=None):
    dims = pa.make_dims(*DIMS)
    rope = rope or pa.Rope(dims, rope_model.table(10, 64))
    (pa.pa_rope_store_int8 if "ks" in t else pa.pa_rope_store)(dims, rope, *t.values(), stream=0)


@pytest.mark.parametrize("int8", [False, True])
def test_wrong_tensors_are_refused(calls, int8):
    call(tensors(int8))
    qkv = torch.zeros(3, 8, 64, dtype=BF)
    call({**tensors(int8), "q": qkv[:, :4], "k": qkv[:, 4:6], "v": qkv[:, 6:]})
    assert [c[0] for c in calls] == ["pa_rope_store_int8" if int8 else "pa_rope_store"] * 2
    assert calls[1][1][5:8] == (512, 512, 512)
    calls.clear()
    good = tensors(int8)
    bad = {"q": good["q"].float(), "k": good["k"][:2], "v": good["v"].half(), "positions": good["positions"].long(),
           "slots": good["slots"][:2], "out": torch.zeros(3, 4, 128, dtype=BF)[..., :64], "kc": good["kc"][:5],
           "vc": good["vc"].float()}
    if int8:
        bad.update(ks=good["ks"].float(), vs=good["vs"][:2])
    for name, x in bad.items():
        with pytest.raises(ValueError):
            call({**good, name: x})
    for name in ("q", "k", "v"):  # a token's heads apart
        wide = torch.zeros(*good[name].shape[:2], 128, dtype=BF)[..., :64]
        with pytest.raises(ValueError):
            call({**good, name: wide})
    with pytest.raises(ValueError):
        call({**good, "positions": torch.zeros(2, 3, dtype=torch.int32)})
    assert calls == []


def test_wrong_ropes_are_refused():
    dims = pa.make_dims(*DIMS)
    t = rope_model.table(10, 64)
    for kw in (dict(cos_sin=t.double()), dict(cos_sin=t[:, :62].contiguous(), pair_axis=[0] * 32), dict(cos_sin=t.t()),
               dict(cos_sin=t, axes=2, pair_axis=[2] * 32), dict(cos_sin=t, q_weight=torch.ones(64)),
               dict(cos_sin=t, k_weight=torch.ones(32, dtype=BF)), dict(cos_sin=t, pair_axis=[0] * 31)):
        with pytest.raises(ValueError):
            pa.Rope(dims, **kw)


def test_library_refusals():
    dims, L = pa.make_dims(*DIMS), pa.lib()
    t = rope_model.table(10, 64)

    def rc(change=(), n=1, strides=(256, 128, 128), q=64, out=4096, k=64, blocks=6, v=64):
        s = pa.Rope(dims, t).struct
        s.cos_sin = 64
        for name, x in change:
            if name == "axis":
                s.pair_axis[31] = x
            else:
                setattr(s, name, x)
        d = pa.make_dims(blocks, *DIMS[1:])
        return L.pa_rope_store(ctypes.byref(d), ctypes.byref(s), q, k, v, *strides, 64, 64, n, out, 64, 64, None)

    assert rc(n=0) == pa.PA_OK
    for change in ([("rotary_dim", 0)], [("rotary_dim", 24)], [("rotary_dim", 80)], [("num_axes", 0)], [("num_axes", 5)]):
        assert rc(change, n=0) == pa.PA_ERR_UNSUPPORTED, change
    for change in ([("axis", 1)], [("eps", -1.0)], [("eps", float("nan"))], [("interleaved", 2)], [("max_position", 0)],
                   [("cos_sin", None)], [("cos_sin", 72)], [("q_weight", 8)], [("k_weight", 8)]):
        assert rc(change) == pa.PA_ERR_INVALID_ARG, change
    assert rc(n=-1) == pa.PA_ERR_INVALID_ARG
    for strides in ((255, 128, 128), (248, 128, 128), (256, 120, 128), (256, 128, 124)):
        assert rc(strides=strides) == pa.PA_ERR_INVALID_ARG, strides
    assert rc(q=72) == pa.PA_ERR_INVALID_ARG and rc(out=8) == pa.PA_ERR_INVALID_ARG and rc(k=None) == pa.PA_ERR_INVALID_ARG
    assert rc(out=64, strides=(512, 128, 128)) == pa.PA_ERR_INVALID_ARG  # in place, tokens apart
    assert rc(blocks=0) == pa.PA_ERR_INVALID_ARG
    assert rc(n=2 ** 31 - 1) == pa.PA_ERR_UNSUPPORTED
    assert L.pa_rope_store(ctypes.byref(dims), None, *[64] * 3, 256, 128, 128, 64, 64, 1, 64, 64, 64, None) == \
        pa.PA_ERR_INVALID_ARG
