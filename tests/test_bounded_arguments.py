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

    for good in ((1, n), (1, 1, n), (2, 2, n), (4, 4, n)):
        call(*good)
    assert len(calls) == 4
    for bad in ((1, n, 1), (2, n, 2), (2, 2 * n), (4, n, 4), (4, 2, 2, n), (2, n), (1, n + 1)):
        with pytest.raises(ValueError):
            call(*bad)
    assert len(calls) == 4
