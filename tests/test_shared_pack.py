"""CPU tests of pa_pack_decode_shared: every key of every context is covered once, shared keys
once per group, and malformed batches are refused."""
import ctypes

import numpy as np
import pytest
import torch

from paged_kv_cache_kvcache_gb300 import pagedattn as pa


def make_batch(seed, sizes, shared_blocks, tails, bs):
    """(contexts, block lists, group offsets, pool blocks): group i shares shared_blocks[i] whole blocks, each
    sequence continues for tails[b] tokens in blocks of its own; tails[b] None: an entry of context 0."""
    rng = np.random.default_rng(seed)
    need = sum(shared_blocks) + sum(-(-t // bs) for t in tails if t is not None)
    ids = list(rng.permutation(need + 3).astype(np.int32))
    ctx, lists, b = [], [], 0
    for n, sh in zip(sizes, shared_blocks):
        common = [ids.pop() for _ in range(sh)]
        for _ in range(n):
            t = tails[b]
            b += 1
            if t is None:
                ctx.append(0)
                lists.append([])
            else:
                ctx.append(sh * bs + t)
                lists.append(common + [ids.pop() for _ in range(-(-t // bs))])
    return ctx, lists, np.cumsum([0] + list(sizes)).tolist(), need + 3


def arrays(plan):
    m = plan.meta
    return (plan.host_array(m.off_items, 8 * m.num_items).reshape(-1, 8),
            plan.host_array(m.off_cta_items, 32 * m.num_ctas).reshape(-1, 32)[:, :4],
            plan.host_array(m.off_seq_parts, 2 * m.num_seqs).reshape(-1, 2))


CASES = [  # sizes, shared blocks, tails, bs, hq, hkv, d, split
    ([4], [3], [1, 5, 16, 40], 16, 8, 2, 64, 0),
    ([4], [3], [1, 0, 16, 40], 16, 8, 2, 64, 128),          # one context ends with the prefix
    ([3, 1, 2], [2, 4, 0], [7, 300, 1, 9, 33, 2], 32, 28, 4, 128, 0),
    ([20, 37], [9, 1], [1 + 3 * i for i in range(57)], 64, 28, 4, 128, 256),
    ([17], [5], [3] * 17, 16, 16, 1, 128, 128),             # 8 sequences per tile, 16 per item
    ([5], [2], [4, None, 6, None, 9], 16, 4, 4, 64, 0),     # padding entries inside a group
    ([2, 3], [1, 0], [None] * 5, 256, 8, 8, 128, 0),        # nothing but padding
    ([1], [0], [5000], 16, 7, 1, 128, 512),
]


@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_parts_cover_every_key_once(case):
    sizes, sh, tails, bs, hq, hkv, d, split = case
    ctx, lists, groups, nb = make_batch(1, sizes, sh, tails, bs)
    dims = pa.make_dims(nb, bs, hq, hkv, d)
    plan = pa.pa_pack_decode_shared(dims, ctx, groups, block_lists=lists, split_tokens=split, pin=False)
    m = plan.meta
    items, cta, parts = arrays(plan)
    B = len(ctx)
    P = 128 // (hq // hkv)
    assert m.rows_per_tile == P and m.num_seqs == B
    if m.num_items:  # CTA by CTA: pairs, first lane, second lane
        assert cta[0, 0] == 0 and cta[-1, 3] == m.num_items and (cta[1:, 0] == cta[:-1, 3]).all()
        assert (np.diff(cta, axis=1) >= 0).all() and (cta[:, 3] > cta[:, 0]).all()
        records = plan.host_array(m.off_cta_items, 32 * m.num_ctas).reshape(-1, 32)
        for (first, l0, l1, end), r in zip(cta.tolist(), records):
            assert (items[first:l0, 1] > P).all() and (items[l0:end, 1] <= P).all()
            # copies of the first items; zeros (no keys) where there is none
            assert r[8:16].tolist() == (items[first].tolist() if first < l1 else [0] * 8)
            assert r[16:24].tolist() == (items[l1].tolist() if l1 < end else [0] * 8)
    table = plan.host_array(m.off_block_tables, B * m.max_blocks_per_seq).reshape(B, -1)
    for b in range(B):
        n = -(-ctx[b] // bs)
        assert table[b, :n].tolist() == [int(x) for x in lists[b][:n]] and (table[b, n:] == -1).all()
    seen = [np.zeros((hkv, c), np.int32) for c in ctx]
    used = {}
    shared_reads = 0
    tiles = {tuple(x) for x in plan.host_array(m.off_scratch_tiles, 4 * m.num_scratch_tiles).reshape(-1, 4).tolist()}
    assert len({x[3] for x in tiles}) == m.num_scratch_tiles and all(x[3] % 128 == 0 and x[1] < x[2] for x in tiles)
    # the parts of single sequences, per (sequence, range) with their slots: instead of those in the CTAs' lists where
    # they run apart, beside them (for an INT8 cache) elsewhere
    ones = plan.host_array(m.off_single_items, 4 * m.num_single_items).reshape(-1, 4).tolist()
    everything = items.tolist()
    if m.apart:
        assert all(x[1] > 1 for x in everything)
        everything += [[b, 1, g, b, k0, k1, max(slot - parts[b, 0], 0) if slot >= 0 else 0, 0]
                       for b, k0, k1, slot in ones for g in range(hkv)]
        assert all((slot >= 0) == (parts[b, 1] > 1) for b, _, _, slot in ones)
    for s0, n, g, row, k0, k1, part, scratch in everything:
        if n > 1 or not m.apart:  # every key tile of the lists' items is in the scratch cache, at the item's row
            for k in range(k0, k1, 128):
                x, = [x for x in tiles if x[1] == k and x[3] == scratch + k]
                assert x[2] >= min(k1, k + 128) and table[x[0], :x[2] // bs].tolist() == table[row, :x[2] // bs].tolist()
        assert 1 <= n <= 2 * P and 0 <= k0 < k1 and 0 <= g < hkv
        assert k0 % min(bs, 128) == 0 and (split == 0 or k1 - k0 <= split)
        for b in range(s0, s0 + n):
            seen[b][g, k0:k1] += 1
            # the blocks read are this sequence's own list's
            assert table[row, k0 // bs:-(-k1 // bs)].tolist() == table[b, k0 // bs:-(-k1 // bs)].tolist()
            assert part < parts[b, 1]
            assert used.setdefault((b, part, g), (k0, k1)) == (k0, k1)
        shared_reads += (n - 1) * (k1 - k0) if g == 0 else 0
    for b in range(B):
        assert (seen[b] == 1).all()
    want = {(s0, k0, k1, parts[s0, 0] + part if parts[s0, 1] > 1 else -1)
            for s0, n, g, _, k0, k1, part, _ in everything if n == 1}
    assert len(ones) == len(want) and set(map(tuple, ones)) == want
    assert m.num_shared_items == sum(i[1] > 1 for i in items.tolist())
    assert plan.host_array(m.off_table_rows, B).tolist() == list(range(B))
    for _, l0, l1, end in cta.tolist():  # in each lane parts of several sequences come first
        for a, b in ((l0, l1), (l1, end)):
            assert (np.diff((items[a:b, 1] == 1).astype(int)) >= 0).all()
    slots = [s for b in range(B) if parts[b, 1] > 1 for s in range(parts[b, 0], parts[b, 0] + parts[b, 1])]
    assert slots == list(range(m.num_partials))
    assert all(parts[b, 1] == 0 for b in range(B) if ctx[b] == 0) and m.max_parts == max(parts[:, 1])
    assert m.merge == int(any(parts[:, 1] != 1))
    # what a group of n live sequences with s shared tokens saves
    saved, at = 0, 0
    for n, s in zip(sizes, sh):
        live = [c for c in ctx[at:at + n] if c]
        at += n
        runs = sum(1 for i in range(at - n, at) if ctx[i] and (i == at - n or not ctx[i - 1]))
        saved += s * bs * (len(live) - runs) if len(live) > 1 else 0
    assert m.tokens_saved == saved


def test_items_are_dealt_out_evenly():
    """No lane gets more than one item's worth of time above the mean; more items than lanes run in two launches."""
    ctx, lists, groups, nb = make_batch(2, [64], [40], [5 + 11 * i for i in range(64)], 64)
    dims = pa.make_dims(nb, 64, 28, 4, 128)
    plan = pa.pa_pack_decode_shared(dims, ctx, groups, block_lists=lists, split_tokens=256, pin=False)
    items, cta, _ = arrays(plan)
    assert plan.meta.apart and len(items) == plan.meta.num_shared_items
    cost = [(1.62 if n > 18 else 2.4) * -(-(k1 - k0) // 128) + (2.5 if n > 18 else 2.0) for _, n, _, _, k0, k1, _, _ in items.tolist()]
    load = [sum(cost[p:l0]) + sum(cost[a:b]) for p, l0, l1, end in cta.tolist() for a, b in ((l0, l1), (l1, end))]
    assert max(load) <= sum(load) / len(load) + max(cost)


def test_short_contexts_are_decoded_whole():
    """The plan decides by lengths; with a given split it never does.  Every sequence is in the list once."""
    dims = pa.make_dims(4000, 16, 28, 4, 128)

    def plan(n, shared, tail, split=0):
        ctx, lists, groups, nb = make_batch(3, [n], [shared // 16], [tail + i % 3 for i in range(n)], 16)
        return ctx, pa.pa_pack_decode_shared(dims, ctx, groups, block_lists=lists, split_tokens=split, pin=False)

    for n, shared, tail, direct in ((2, 64, 20, 3), (8, 256, 44, 3), (8, 8192, 44, 0), (64, 4096, 200, 0)):
        ctx, p = plan(n, shared, tail)
        m = p.meta
        assert m.direct == direct and plan(n, shared, tail, 128)[1].meta.direct == 0
        assert (m.workspace_bytes == 0) == bool(direct & 1) and (m.workspace_bytes_int8 == 0) == bool(direct & 2)
        whole = p.host_array(m.off_direct_items, 4 * n).reshape(-1, 4)
        assert sorted(whole[:, 0].tolist()) == list(range(n)) and (np.diff(whole[:, 2]) <= 0).all()
        assert all(x == [b, 0, ctx[b], -1] for x in whole.tolist() for b in x[:1])


def test_shared_length_is_found_and_checked():
    dims = pa.make_dims(64, 16, 4, 2, 64)
    ctx, lists = [100, 90, 70], [[1, 2, 3, 4, 5, 6, 7], [1, 2, 3, 9, 10, 11], [1, 2, 3, 4, 20]]
    find = lambda **k: pa.pa_pack_decode_shared(dims, ctx, block_lists=lists, pin=False, **k)
    assert find().meta.tokens_saved == 2 * 48
    assert find(shared_lens=[32]).meta.tokens_saved == 2 * 32
    assert find(shared_lens=[0]).meta.tokens_saved == 0
    for bad in ([64], [8], [-16], [4096]):   # not common, not whole blocks, negative, longer than a context
        with pytest.raises(pa.PagedAttnError) as e:
            find(shared_lens=bad)
        assert e.value.code == pa.PA_ERR_INVALID_ARG
    # the last block of a context counts only if the context fills it
    assert pa.pa_pack_decode_shared(dims, [40, 33], block_lists=[[1, 2, 3], [1, 2, 3]], pin=False).meta.tokens_saved == 32


def test_plan_for_a_device_table():
    dims = pa.make_dims(64, 16, 4, 2, 64)
    plan = pa.pa_pack_decode_shared(dims, [100, 0, 70], [0, 3], shared_lens=[48], table_rows=[5, 9, 2], max_blocks=7,
                                    pin=False)
    items, _, parts = arrays(plan)
    assert not plan.meta.tables_packed and plan.meta.max_blocks_per_seq == 7
    m = plan.meta  # the empty entry parts the two that share: the decode kernels only
    assert len(items) == 0 and m.apart == 1 and m.num_ctas == 0
    assert set(plan.host_array(m.off_single_items, 4 * m.num_single_items).reshape(-1, 4)[:, 0].tolist()) == {0, 2}
    plan2 = pa.pa_pack_decode_shared(dims, [100, 70, 0], [0, 3], shared_lens=[48], table_rows=[5, 2, 9], max_blocks=7,
                                     pin=False)
    items, _, _ = arrays(plan2)
    assert {(int(s), int(n), int(r)) for s, n, r in items[:, [0, 1, 3]]} == {(0, 2, 5), (0, 1, 5), (1, 1, 2)}
    with pytest.raises(AssertionError):
        plan.slot_mapping
    bad = [dict(shared_lens=None), dict(max_blocks=6), dict(max_blocks=0), dict(table_rows=[5, -1, 2]),
           dict(split_tokens=64), dict(split_tokens=-128), dict(group_offsets=[0, 2]), dict(group_offsets=[1, 3]),
           dict(group_offsets=[0, 2, 1, 3], shared_lens=[0, 0, 0]), dict(context_lens=[100, -1, 70])]
    for change in bad:
        args = dict(context_lens=[100, 0, 70], group_offsets=[0, 3], shared_lens=[48], table_rows=[5, 9, 2], max_blocks=7)
        args.update(change)
        with pytest.raises(pa.PagedAttnError) as e:
            pa.pa_pack_decode_shared(dims, pin=False, **args)
        assert e.value.code == pa.PA_ERR_INVALID_ARG, change
    for change in (dict(shared_lens=[1, 2]), dict(table_rows=[1])):
        with pytest.raises(ValueError):
            pa.pa_pack_decode_shared(dims, [100, 0, 70], [0, 3], **{**dict(shared_lens=[48], max_blocks=7), **change})
    with pytest.raises(pa.PagedAttnError):   # block lists and table rows
        pa.pa_pack_decode_shared(dims, [5], block_lists=[[1]], table_rows=[0], pin=False)
    with pytest.raises(pa.PagedAttnError):   # an id outside the pool
        pa.pa_pack_decode_shared(dims, [5], block_lists=[[64]], pin=False)


def test_empty_batch_and_small_buffer():
    dims = pa.make_dims(8, 16, 4, 2, 64)
    plan = pa.pa_pack_decode_shared(dims, [], block_lists=[], pin=False)
    assert plan.meta.num_items == 0 and plan.meta.workspace_bytes == 0 and plan.meta.workspace_bytes_int8 == 0
    meta = pa.pa_shared_meta()
    ctx, off, groups = (np.array(x, np.int32) for x in ([20], [0, 2], [0, 1]))
    ids, buf = np.array([1, 2], np.int32), np.zeros(64, np.uint8)
    p = lambda a: a.ctypes.data_as(ctypes.c_void_p)
    rc = pa.lib().pa_pack_decode_shared(ctypes.byref(dims), 1, p(ctx), 1, p(groups), None, p(off), p(ids), None, 0, 0,
                                        p(buf), 64, ctypes.byref(meta))
    assert rc == pa.PA_ERR_WORKSPACE and meta.total_bytes > 64


def test_shared_decode_rejects_bad_args_without_touching_the_gpu():
    dims = pa.make_dims(8, 16, 4, 2, 64)
    m = pa.pa_shared_meta()
    L = pa.lib()

    def call(scale=0.1, q=16, out=16, ws=None, nbytes=0, bt=16, items=16, whole=16, rows=16, ones=16, dims=dims):
        return L.pa_decode_shared(ctypes.byref(dims), q, 16, 16, bt, ctypes.c_float(scale), out, ctypes.byref(m), items,
                                  16, 16, whole, rows, ones, ws, nbytes, None)

    m.num_seqs, m.num_items, m.num_ctas, m.max_blocks_per_seq, m.rows_per_tile = 0, 0, 0, 1, 64
    assert call() == pa.PA_OK                                   # nothing to do
    m.num_seqs, m.num_items, m.num_ctas = 2, 4, 4
    m.num_heads, m.num_kv_heads, m.head_dim, m.block_size = 4, 2, 64, 16
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        assert call(scale=bad) == pa.PA_ERR_INVALID_ARG
    assert call(q=None) == pa.PA_ERR_INVALID_ARG
    assert call(out=8) == pa.PA_ERR_INVALID_ARG
    assert call(items=24) == pa.PA_ERR_INVALID_ARG
    assert call(bt=None) == call(whole=None) == call(whole=8) == call(rows=None) == call(rows=18) == call(ones=None) == call(ones=8) == pa.PA_ERR_INVALID_ARG
    assert call(dims=pa.make_dims(8, 16, 8, 2, 64)) == pa.PA_ERR_INVALID_ARG   # packed for group 2
    for other in ((8, 16, 2, 1, 64), (8, 16, 8, 4, 64), (8, 16, 4, 2, 128), (8, 32, 4, 2, 64)):  # or for other heads or blocks
        assert call(dims=pa.make_dims(*other)) == pa.PA_ERR_INVALID_ARG
    assert call(dims=pa.make_dims(0, 16, 4, 2, 64)) == pa.PA_ERR_INVALID_ARG   # empty pool
    m.num_partials, m.workspace_bytes, m.workspace_bytes_int8 = 3, 1024 * 3 + 256, 1024 * 3 + 256
    assert call(ws=256, nbytes=1024) == pa.PA_ERR_WORKSPACE
    assert call(ws=16, nbytes=4096) == pa.PA_ERR_INVALID_ARG                   # not 256-byte aligned
    assert call(ws=None, nbytes=4096) == pa.PA_ERR_INVALID_ARG
    m.workspace_bytes = 512                                                    # not this batch's size
    assert call(ws=256, nbytes=4096) == pa.PA_ERR_INVALID_ARG
    m.workspace_bytes, m.num_scratch_tiles = 1024 * 3 + 256, 2
    m.workspace_bytes_int8 = m.workspace_bytes + 2 * 128 * 2 * 64 * 4 + 2 * 4 * 64 * 2

    def call8(**change):
        a = dict(ks=16, vs=16, one=16, rows=16, tiles=16, nbytes=1 << 20)
        a.update(change)
        return L.pa_decode_shared_int8(ctypes.byref(dims), 16, 16, 16, a["ks"], a["vs"], 16, ctypes.c_float(0.1), 16,
                                       ctypes.byref(m), 16, 16, 16, 16, a["rows"], a["one"], a["tiles"], 256, a["nbytes"], None)

    m.num_shared_items = 5  # more than there are items
    assert call8() == pa.PA_ERR_INVALID_ARG
    m.num_shared_items = 2
    for bad in (dict(ks=None), dict(vs=None), dict(ks=24), dict(one=None), dict(one=8), dict(rows=None), dict(rows=18), dict(tiles=None),
                dict(tiles=8)):
        assert call8(**bad) == pa.PA_ERR_INVALID_ARG, bad
    assert call8(nbytes=m.workspace_bytes) == pa.PA_ERR_WORKSPACE  # bf16's would do
    m.num_scratch_tiles = 1
    assert call8() == pa.PA_ERR_INVALID_ARG
    m.num_scratch_tiles, m.direct = 2, 2  # INT8 would decode whole contexts: it needs no workspace
    assert call8() == pa.PA_ERR_INVALID_ARG
    m.num_ctas = 0
    assert call(ws=256, nbytes=4096) == pa.PA_ERR_INVALID_ARG


def test_a_plan_keeps_its_dims_and_its_rows():
    dims = pa.make_dims(64, 16, 4, 2, 64)
    plan = pa.pa_pack_decode_shared(dims, [100, 70], shared_lens=[48], table_rows=[5, 2], max_blocks=7, pin=False)
    m = plan.meta
    assert (m.num_heads, m.num_kv_heads, m.head_dim, m.block_size) == (4, 2, 64, 16) and plan.num_rows == 6
    assert pa.pa_pack_decode_shared(dims, [100, 70], shared_lens=[48], max_blocks=7, pin=False).num_rows == 2
    plan.dev = torch.zeros(1, dtype=torch.uint8)
    for bad in (torch.zeros(5, 7), torch.zeros(6, 8), torch.zeros(42)):
        with pytest.raises(ValueError):
            pa._shared_tables(plan, bad.int())
    assert pa._shared_tables(plan, torch.zeros(6, 7, dtype=torch.int32))
