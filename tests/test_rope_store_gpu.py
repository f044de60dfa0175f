"""pa_rope_store(_int8) against its formulas in 64 bits.

Tolerance of a bf16 result: half a step, 2^-8 of the value, and for what fp32 rounds before it (a mean of squares, a
reciprocal root, two products and a sum: under 32 roundings of 2^-24 of the row's largest value) 2^-19 of that.
An INT8 code is within half a step of the value, plus the 2^-11 that fp16 rounds its scale by and as much again for
fp32: amax / 127 (1/2 + 127 2^-11 + 2^-7).
"""
import numpy as np
import pytest
import torch

from paged_kv_cache_kvcache_gb300 import pagedattn as pa
from tests import rope_model

pytestmark = pytest.mark.gpu

CASES = [  # tokens, hq, hkv, d, bs, rot, axes, interleaved, norm, packed
    (1, 16, 8, 128, 256, 128, 1, False, "qk", True),
    (7, 28, 4, 128, 16, 128, 1, False, None, True),
    (33, 4, 2, 64, 16, 64, 3, False, "qk", False),
    (65, 7, 1, 128, 32, 64, 2, True, "q", True),
    (130, 12, 1, 64, 16, 16, 1, True, "k", False),
    (257, 16, 16, 128, 64, 112, 4, False, None, False),
    (2500, 28, 4, 128, 16, 128, 1, False, "qk", True),  # many: four rows per group
    (4001, 8, 8, 64, 16, 32, 3, True, "qk", True),
    (3000, 16, 8, 128, 128, 48, 2, False, "k", False),
]


def make(case, seed=0, far=3000):
    n, hq, hkv, d, bs, rot, axes, inter, norm, packed = case
    g = torch.Generator().manual_seed(seed)
    draw = lambda *shape: torch.randn(*shape, generator=g).to(torch.bfloat16).cuda()
    if packed:
        qkv = draw(n, hq + 2 * hkv, d)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        q, k, v = draw(n, hq, d), draw(n, hkv, d), draw(n, hkv, d)
    blocks = -(-n // bs) + 2
    r = np.random.default_rng(seed)
    slots = r.permutation(blocks * bs)[:n].astype(np.int32)
    slots[r.random(n) < 0.05] = -1
    pos = r.integers(0, far, (axes, n)).astype(np.int32)
    axis = r.integers(0, axes, rot // 2) if inter else np.arange(rot // 2) * axes // (rot // 2)
    dims = pa.make_dims(blocks, bs, hq, hkv, d)
    cs = rope_model.table(far, rot).cuda()
    w = lambda on: (1 + 0.5 * torch.randn(d, generator=g)).to(torch.bfloat16).cuda() if on else None
    qw, kw = w(norm and "q" in norm), w(norm and "k" in norm)
    rope = pa.Rope(dims, cs, axes=axes, pair_axis=axis, interleaved=inter, q_weight=qw, k_weight=kw, eps=1e-6)
    want = [rope_model.turned(x, xw, cs, pos, axis, inter, 1e-6) for x, xw in ((q, qw), (k, kw))]
    return dict(dims=dims, rope=rope, q=q, k=k, v=v, slots=slots, pos=pos, want=want, n=n)


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda()


def near(got, want):
    got = got.double().cpu().numpy()
    top = np.abs(want).max(-1, keepdims=True) if want.size else 0.0
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * top).all()


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_rope_store(case):
    c = make(case)
    d = c["dims"]
    kc = torch.full((d.num_blocks, d.block_size, d.num_kv_heads, d.head_dim), 7.0, dtype=torch.bfloat16, device="cuda")
    vc, out = kc.clone(), torch.empty_like(c["q"].contiguous())
    pa.pa_rope_store(d, c["rope"], c["q"], c["k"], c["v"], i32(c["pos"]), i32(c["slots"]), out, kc, vc)
    near(out, c["want"][0])
    live = c["slots"] >= 0
    rows = lambda x: x.flatten(0, 1).cpu()[c["slots"][live].astype(np.int64)]
    near(rows(kc), c["want"][1][live])
    assert torch.equal(rows(vc), c["v"].cpu()[torch.as_tensor(live)])
    untouched = np.ones(d.num_blocks * d.block_size, bool)
    untouched[c["slots"][live]] = False
    for x in (kc, vc):
        assert (x.flatten(0, 1).cpu()[torch.as_tensor(untouched)] == 7).all()


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_rope_store_int8(case):
    c = make(case, seed=1)
    d = c["dims"]
    kc, vc, ks, vs = pa.int8_cache(d)
    out = torch.empty_like(c["q"].contiguous())
    pa.pa_rope_store_int8(d, c["rope"], c["q"], c["k"], c["v"], i32(c["pos"]), i32(c["slots"]), out, kc, vc, ks, vs)
    near(out, c["want"][0])
    live, slots = c["slots"] >= 0, c["slots"][c["slots"] >= 0].astype(np.int64)
    codes = kc.flatten(0, 1).cpu()[slots].double().numpy()
    scale = ks.transpose(1, 2).flatten(0, 1).cpu()[slots].double().numpy()[..., None]
    want = c["want"][1][live]
    top = np.abs(want).max(-1, keepdims=True)
    assert (np.abs(codes * scale - want) <= top / 127 * (0.5 + 127 * 2.0 ** -11 + 2.0 ** -7)).all()
    # values: as the store quantises them, bit for bit; other slots as they were
    kr, vr, ksr, vsr = pa.int8_cache(d)
    pa.pa_store_kvcache_int8(d, c["k"].contiguous(), c["v"].contiguous(), kr, vr, ksr, vsr, i32(c["slots"]))
    assert torch.equal(vc, vr) and torch.equal(vs, vsr)
    gone = torch.ones(d.num_blocks * d.block_size, dtype=torch.bool)
    gone[slots] = False
    assert not kc.flatten(0, 1).cpu()[gone].any() and not ks.transpose(1, 2).flatten(0, 1).cpu()[gone].any()


def test_in_place_and_tiny_and_zero_rows():
    c = make(CASES[8])
    d, n = c["dims"], c["n"]
    q = c["q"].clone()
    q[5] = 0
    q[6] *= 1e-30  # the eps decides
    want = rope_model.turned(q, None, c["rope"].cos_sin, c["pos"], list(c["rope"].struct.pair_axis)[:24], False, 1e-6)
    kc, vc = (torch.zeros(d.num_blocks, d.block_size, d.num_kv_heads, d.head_dim, dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    pa.pa_rope_store(d, c["rope"], q, c["k"], c["v"], i32(c["pos"]), i32(c["slots"]), q, kc, vc)
    near(q, want)
    # no tokens: nothing happens
    e = torch.empty(0, d.num_heads, d.head_dim, dtype=torch.bfloat16, device="cuda")
    ek = torch.empty(0, d.num_kv_heads, d.head_dim, dtype=torch.bfloat16, device="cuda")
    one = torch.empty(0, dtype=torch.int32, device="cuda")
    pa.pa_rope_store(d, c["rope"], e, ek, ek, torch.empty(2, 0, dtype=torch.int32, device="cuda"), one, e.clone(), kc, vc)


@pytest.mark.parametrize("int8", [False, True])
def test_bad_positions_and_slots_are_skipped_and_flagged(int8):
    c = make((40, 8, 2, 64, 16, 64, 2, False, "qk", True), seed=3)
    d = c["dims"]
    pos, slots = c["pos"].copy(), np.arange(40, dtype=np.int32)
    pos[0, 3], pos[1, 4], pos[1, 39] = -1, 3000, 2 ** 31 - 1
    out = torch.full((40, 8, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    caches = pa.int8_cache(d) if int8 else tuple(
        torch.zeros(d.num_blocks, d.block_size, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    call = pa.pa_rope_store_int8 if int8 else pa.pa_rope_store
    call(d, c["rope"], c["q"], c["k"], c["v"], i32(pos), i32(slots), out, *caches)
    assert pa.pa_read_device_error() == 1 << 9
    bad = [3, 4, 39]
    assert (out[bad] == 5).all() and not caches[0].flatten(0, 1)[bad].any() and not caches[1].flatten(0, 1)[bad].any()
    good = [i for i in range(40) if i not in bad]
    near(out[good], c["want"][0][good])
    slots[[1, 2]] = [-2, d.num_blocks * d.block_size]
    call(d, c["rope"], c["q"], c["k"], c["v"], i32(c["pos"]), i32(slots), out, *caches)
    assert pa.pa_read_device_error() == 1
    near(out, c["want"][0])


def test_other_stream_and_captured():
    c = make(CASES[1], seed=5)
    d = c["dims"]
    kc, vc = (torch.zeros(d.num_blocks, d.block_size, d.num_kv_heads, d.head_dim, dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    out = torch.empty_like(c["q"].contiguous())
    pos, slots = i32(c["pos"]), i32(c["slots"])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    pa.pa_rope_store(d, c["rope"], c["q"], c["k"], c["v"], pos, slots, out, kc, vc, stream=st)
    st.synchronize()
    near(out, c["want"][0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            pa.pa_rope_store(d, c["rope"], c["q"], c["k"], c["v"], pos, slots, out, kc, vc)
    out.zero_()
    kc.zero_()
    graph.replay()
    torch.cuda.synchronize()
    near(out, c["want"][0])
    live = c["slots"] >= 0
    near(kc.flatten(0, 1).cpu()[c["slots"][live].astype(np.int64)], c["want"][1][live])
