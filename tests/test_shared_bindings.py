"""CPU tests of the shared decode's Python calls: tensors that are too small or of another type are refused before the
library is called (which sees addresses only)."""
import pytest
import torch

from paged_kv_cache_kvcache_gb300 import pagedattn as pa

DIMS = (6, 16, 4, 2, 64)


class Recorder:
    """In the library's place: notes the calls that get through."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append(name) or pa.PA_OK


@pytest.fixture
def plan_and_calls(monkeypatch):
    plan = pa.pa_pack_decode_shared(pa.make_dims(*DIMS), [40, 33, 0], shared_lens=[32], table_rows=[0, 2, 1], max_blocks=3,
                                    split_tokens=128, pin=False)
    recorder = Recorder()
    monkeypatch.setattr(pa, "_lib", recorder)
    monkeypatch.setattr(pa, "_device", lambda: -1)  # where the host's tensors are
    plan.upload(device="cpu", stream=0)
    recorder.calls.clear()
    return plan, recorder.calls


def tensors(int8):
    nb, bs, hq, hkv, d = DIMS
    cache = torch.int8 if int8 else torch.bfloat16
    t = {"q": torch.zeros(3, hq, d, dtype=torch.bfloat16), "k": torch.zeros(nb, bs, hkv, d, dtype=cache),
         "v": torch.zeros(nb, bs, hkv, d, dtype=cache), "out": torch.zeros(3, hq, d, dtype=torch.bfloat16)}
    if int8:
        t.update(ks=torch.zeros(nb, hkv, bs, dtype=torch.float16), vs=torch.zeros(nb, hkv, bs, dtype=torch.float16))
    return t


def call(plan, t, dims=DIMS):
    bt = torch.zeros(3, 3, dtype=torch.int32)
    ws = pa.shared_workspace(plan, device="cpu")
    if "ks" in t:
        pa.pa_decode_shared_int8(pa.make_dims(*dims), t["q"], t["k"], t["v"], t["ks"], t["vs"], plan, 0.1, t["out"], ws,
                                 block_tables=bt, stream=0)
    else:
        pa.pa_decode_shared(pa.make_dims(*dims), t["q"], t["k"], t["v"], plan, 0.1, t["out"], ws, block_tables=bt, stream=0)


@pytest.mark.parametrize("int8", [False, True])
def test_small_and_wrongly_typed_tensors_are_refused(plan_and_calls, int8):
    plan, calls = plan_and_calls
    name = "pa_decode_shared_int8" if int8 else "pa_decode_shared"
    good = tensors(int8)
    call(plan, good)
    more = {k: torch.cat([x, x[:1]]) for k, x in good.items()}  # padded batches and larger caches are fine
    call(plan, more)
    assert calls == [name] * 2
    for key, x in good.items():
        for bad in (x[:-1], x.flatten()[:-1], x[:0]):
            with pytest.raises(ValueError, match="values"):
                call(plan, {**good, key: bad})
        for dtype in (torch.float16, torch.bfloat16, torch.float32, torch.int8, torch.uint8):
            if dtype is not x.dtype:
                with pytest.raises(ValueError, match="must be"):
                    call(plan, {**good, key: x.to(dtype)})
    larger = (DIMS[0] + 1,) + DIMS[1:]  # dims of a pool that the caches do not hold
    with pytest.raises(ValueError, match="values"):
        call(plan, good, larger)
    assert calls == [name] * 2
    call(plan, more, larger)
    assert calls == [name] * 3


def test_an_empty_batch_needs_nothing(monkeypatch):
    plan = pa.pa_pack_decode_shared(pa.make_dims(*DIMS), [], block_lists=[], pin=False)
    recorder = Recorder()
    monkeypatch.setattr(pa, "_lib", recorder)
    monkeypatch.setattr(pa, "_device", lambda: -1)
    plan.upload(device="cpu", stream=0)
    t = tensors(False)
    pa.pa_decode_shared(pa.make_dims(*DIMS), t["q"][:0], t["k"], t["v"], plan, 0.1, t["out"][:0], stream=0)
    assert recorder.calls[-1] == "pa_decode_shared"


def test_a_plan_packed_again_counts_from_its_upload_on(plan_and_calls, monkeypatch):
    """Until it is uploaded again, calls run the plan on the device: what they need goes by that one."""
    plan, calls = plan_and_calls  # rows 0, 2 and 1 of a table 3 wide
    recorder = pa._lib
    monkeypatch.setattr(pa, "_lib", None)  # the packer is the library's
    again = pa.pa_pack_decode_shared(pa.make_dims(*DIMS), [10], shared_lens=[0], table_rows=[0], max_blocks=2,
                                     split_tokens=128, into=plan)
    assert again is plan and plan.num_rows == 1
    monkeypatch.setattr(pa, "_lib", recorder)
    t = tensors(False)
    for shape in ((1, 2), (2, 3), (3, 2)):
        with pytest.raises(ValueError, match="3 rows or more, 3"):
            pa.pa_decode_shared(pa.make_dims(*DIMS), t["q"], t["k"], t["v"], plan, 0.1, t["out"],
                                block_tables=torch.zeros(*shape, dtype=torch.int32), stream=0)
    with pytest.raises(ValueError, match="q has"):
        call(plan, {**t, "q": t["q"][:1]})
    call(plan, t)
    plan.upload(device="cpu", stream=0)
    calls.clear()
    pa.pa_decode_shared(pa.make_dims(*DIMS), t["q"][:1], t["k"], t["v"], plan, 0.1, t["out"][:1],
                        block_tables=torch.zeros(1, 2, dtype=torch.int32), stream=0)
    assert calls == ["pa_decode_shared"]
