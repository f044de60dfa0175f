"""Thin ctypes binding of libpagedattn (include/pagedattn.h), same entry-point names.

Argument marshalling only: every step of the path (metadata packing, KV
scatter, prefill, decode) runs in the native library; torch provides device
memory, pinned host memory and streams.  There is no fallback: if the CUDA
library cannot be built or loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from dataclasses import dataclass
from typing import Optional, Sequence

import numpy as np
import torch

from . import _build

PA_OK, PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_ERR_WORKSPACE, PA_ERR_CUDA = 0, 1, 2, 3, 4

EXPORTS = ("pa_pack_prefill", "pa_pack_decode", "pa_upload", "pa_store_kvcache", "pa_prefill_varlen",
           "pa_decode", "pa_decode_static", "pa_copy_blocks", "pa_store_kvcache_int8", "pa_decode_int8",
           "pa_prefill_varlen_int8", "pa_pack_decode_fixed", "pa_decode_fused", "pa_copy_blocks_int8",
           "pa_decode_int8_fused", "pa_prefill_varlen_fused", "pa_prefill_varlen_int8_fused",
           "pa_pack_decode_shared", "pa_decode_shared", "pa_decode_shared_int8", "pa_pool_workspace", "pa_pool_append",
           "pa_pool_fork", "pa_pool_free", "pa_pool_compact",
           "pa_last_error_string", "pa_read_device_error", "pa_selftest_bounded_wait", "pa_stream_read",
           "pa_version")

PA_DECODE_STATIC_SCRATCH_BYTES = 16 << 20


class pa_dims(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class pa_prefill_meta(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("total_q", ctypes.c_int32), ("max_seqlen_q", ctypes.c_int32),
                ("max_seqlen_k", ctypes.c_int32), ("max_blocks_per_seq", ctypes.c_int32),
                ("num_tiles", ctypes.c_int32), ("rows_per_tile", ctypes.c_int32), ("prefix_aligned", ctypes.c_int32),
                ("off_cu_seqlens_q", ctypes.c_uint64), ("off_cu_seqlens_k", ctypes.c_uint64),
                ("off_block_tables", ctypes.c_uint64), ("off_slot_mapping", ctypes.c_uint64),
                ("off_tiles", ctypes.c_uint64), ("total_bytes", ctypes.c_uint64),
                ("off_scratch_tables", ctypes.c_uint64), ("off_scratch_items", ctypes.c_uint64),
                ("workspace_bytes", ctypes.c_uint64), ("scratch_blocks", ctypes.c_int32),
                ("scratch_pitch", ctypes.c_int32)]


class pa_decode_meta(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("max_blocks_per_seq", ctypes.c_int32),
                ("num_items", ctypes.c_int32), ("split_tokens", ctypes.c_int32), ("max_splits", ctypes.c_int32),
                ("num_partials", ctypes.c_int32), ("off_context_lens", ctypes.c_uint64),
                ("off_block_tables", ctypes.c_uint64), ("off_slot_mapping", ctypes.c_uint64),
                ("off_items", ctypes.c_uint64), ("off_seq_items", ctypes.c_uint64),
                ("total_bytes", ctypes.c_uint64), ("workspace_bytes", ctypes.c_uint64)]


class pa_shared_meta(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("num_groups", ctypes.c_int32), ("max_blocks_per_seq", ctypes.c_int32),
                ("num_items", ctypes.c_int32), ("num_ctas", ctypes.c_int32), ("num_partials", ctypes.c_int32),
                ("max_parts", ctypes.c_int32), ("rows_per_tile", ctypes.c_int32), ("merge", ctypes.c_int32),
                ("split_tokens", ctypes.c_int32), ("tables_packed", ctypes.c_int32),
                ("num_single_items", ctypes.c_int32), ("num_shared_items", ctypes.c_int32),
                ("num_scratch_tiles", ctypes.c_int32), ("direct", ctypes.c_int32), ("apart", ctypes.c_int32),
                ("tokens_saved", ctypes.c_uint64), ("off_block_tables", ctypes.c_uint64),
                ("off_slot_mapping", ctypes.c_uint64), ("off_items", ctypes.c_uint64),
                ("off_cta_items", ctypes.c_uint64), ("off_seq_parts", ctypes.c_uint64),
                ("off_single_items", ctypes.c_uint64), ("off_table_rows", ctypes.c_uint64),
                ("off_direct_items", ctypes.c_uint64), ("off_scratch_tiles", ctypes.c_uint64),
                ("total_bytes", ctypes.c_uint64),
                ("workspace_bytes", ctypes.c_uint64), ("workspace_bytes_int8", ctypes.c_uint64),
                ("num_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("block_size", ctypes.c_int32)]


class pa_pool(ctypes.Structure):
    _fields_ = [("num_rows", ctypes.c_int32), ("max_blocks", ctypes.c_int32), ("num_layers", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("block_tables", ctypes.c_void_p), ("context_lens", ctypes.c_void_p),
                ("ref_counts", ctypes.c_void_p), ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("layer_stride", ctypes.c_uint64),
                ("scale_layer_stride", ctypes.c_uint64)]


class PagedAttnError(RuntimeError):
    def __init__(self, code: int, fn: str, msg: str):
        super().__init__(f"{fn} failed with code {code}: {msg}")
        self.code = code


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """Load libpagedattn (building it with nvcc first if it is missing or stale)."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.build()
            L = ctypes.CDLL(path)
            P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
            L.pa_pack_prefill.argtypes = [P, I32, P, P, P, P, P, SZ, P]
            L.pa_pack_decode.argtypes = [P, I32, P, P, P, I32, P, SZ, P]
            L.pa_pack_decode_fixed.argtypes = [P, I32, P, P, P, I32, I32, P, SZ, P]
            L.pa_decode_fused.argtypes = [P, P, P, P, P, P, P, P, P, ctypes.c_float, P, P, P, P, P, SZ, P]
            L.pa_upload.argtypes = [P, P, SZ, P]
            L.pa_store_kvcache.argtypes = [P, P, P, P, P, P, I32, P]
            L.pa_prefill_varlen.argtypes = [P, P, P, P, P, P, P, ctypes.c_float, P, P, P, P]
            L.pa_prefill_varlen_fused.argtypes = [P, P, P, P, P, P, P, P, P, P, ctypes.c_float, P, P, P, P]
            L.pa_decode.argtypes = [P, P, P, P, P, P, ctypes.c_float, P, P, P, P, P, SZ, P]
            L.pa_decode_static.argtypes = [P, P, P, P, P, P, ctypes.c_float, P, P, P, P, P]
            L.pa_copy_blocks.argtypes = [P, P, P, P, I32, P]
            L.pa_copy_blocks_int8.argtypes = [P, P, P, P, P, P, I32, P]
            L.pa_decode_int8_fused.argtypes = [P, P, P, P, P, P, P, P, P, P, P, ctypes.c_float, P, P, P, P, P, SZ,
                                               P]
            L.pa_store_kvcache_int8.argtypes = [P, P, P, P, P, P, P, P, I32, P]
            L.pa_decode_int8.argtypes = [P, P, P, P, P, P, P, P, ctypes.c_float, P, P, P, P, P, SZ, P]
            L.pa_prefill_varlen_int8.argtypes = [P] * 11 + [ctypes.c_float] + [P] * 4 + [SZ, P]
            L.pa_prefill_varlen_int8_fused.argtypes = [P] * 14 + [ctypes.c_float] + [P] * 4 + [SZ, P]
            L.pa_pack_decode_shared.argtypes = [P, I32, P, I32, P, P, P, P, P, I32, I32, P, SZ, P]
            L.pa_decode_shared.argtypes = [P] * 5 + [ctypes.c_float] + [P] * 9 + [SZ, P]
            L.pa_decode_shared_int8.argtypes = [P] * 7 + [ctypes.c_float] + [P] * 10 + [SZ, P]
            L.pa_pool_workspace.argtypes = [P, P, P]
            L.pa_pool_append.argtypes = [P, P, P, P, I32, P, I32, P, SZ, P]
            L.pa_pool_fork.argtypes = [P, P, P, P, I32, P, SZ, P]
            L.pa_pool_free.argtypes = [P, P, P, I32, P]
            L.pa_pool_compact.argtypes = [P, P, P, P, P, P, SZ, P]
            L.pa_last_error_string.argtypes = []
            L.pa_last_error_string.restype = ctypes.c_char_p
            L.pa_read_device_error.argtypes = [P, P]
            L.pa_selftest_bounded_wait.argtypes = [ctypes.c_uint32, ctypes.c_int, P]
            L.pa_stream_read.argtypes = [P, SZ, P, P]
            L.pa_version.argtypes = []
            for name in EXPORTS:
                if name not in ("pa_last_error_string",):
                    getattr(L, name).restype = ctypes.c_int
            _lib = L
    return _lib


def _check(rc: int, fn: str):
    if rc != PA_OK:
        raise PagedAttnError(rc, fn, pa_last_error_string())


def pa_last_error_string() -> str:
    return lib().pa_last_error_string().decode(errors="replace")


def pa_version() -> int:
    return int(lib().pa_version())


# torch's own lookup of the current stream without building a Stream object (3 us of a call's 10)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_cur_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream) -> Optional[int]:
    if stream is None:
        if _raw_stream is not None and _cur_device is not None and torch.cuda.is_initialized():
            return _raw_stream(_cur_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        return t.data_ptr() if t.numel() > 0 else None
    return int(t)


_BF16, _FP16, _INT8 = torch.bfloat16, torch.float16, torch.int8
_device = _cur_device if _cur_device is not None else torch.cuda.current_device


def _elsewhere(t, dev: int):
    return ValueError(f"tensor on {t.device}, the current device is cuda:{dev}")


def _refuse(plan_device: int, tensors, wanted) -> None:
    """Why a call's plan and tensors are refused (the calls test for it themselves: a loop here is 0.2 us a tensor).

    ``wanted``: (what, tensor, type, least number of values).
    """
    dev = _device()
    if plan_device != dev:
        raise ValueError(f"the plan is on cuda:{plan_device}, the current device is cuda:{dev}")
    for t in tensors:
        if t is not None and t.get_device() != dev:  # a kernel launched on this device could not read it
            raise _elsewhere(t, dev)
        if t is not None and not t.is_contiguous():
            raise ValueError(f"tensors must be contiguous, got strides {t.stride()}")
    for what, t, dtype, least in wanted:
        if t.dtype is not dtype:
            raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
        if t.numel() < least:
            raise ValueError(f"{what} has {t.numel()} values, the plan and dims need {least}")


def _stream_of(dev: int, stream) -> Optional[int]:
    """_stream on a device that is known and in use."""
    return _raw_stream(dev) if stream is None and _raw_stream is not None else _stream(stream)


def _int32(t, what: str, count: Optional[int] = None, dev: Optional[int] = None) -> int:
    """Address of a contiguous int32 tensor (of `count` values, on device `dev`)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or not t.is_contiguous() or \
            (count is not None and t.numel() != count):
        raise ValueError(f"{what} must be a contiguous int32 tensor" + ("" if count is None else f" of {count}"))
    if dev is not None and t.get_device() != dev:
        raise _elsewhere(t, dev)
    return t.data_ptr()


def make_dims(num_blocks: int, block_size: int, num_heads: int, num_kv_heads: int, head_dim: int) -> pa_dims:
    return pa_dims(num_blocks, block_size, num_heads, num_kv_heads, head_dim)


def _i32(x) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(x, dtype=np.int32))


def _np_ptr(a: np.ndarray):
    return a.ctypes.data_as(ctypes.c_void_p) if a.size else None


def _flatten(block_lists) -> tuple:
    """Per-sequence block lists -> (offsets [B+1], flat ids); an (offsets, ids) pair passes through."""
    if isinstance(block_lists, tuple) and len(block_lists) == 2 and isinstance(block_lists[0], np.ndarray):
        return block_lists
    off = np.zeros(len(block_lists) + 1, dtype=np.int32)
    for i, b in enumerate(block_lists):
        off[i + 1] = off[i] + len(b)
    ids = (np.concatenate([np.asarray(b, np.int32) for b in block_lists]) if len(block_lists)
           else np.zeros(0, np.int32))
    return off, _i32(ids)


@dataclass
class _Plan:
    meta: ctypes.Structure
    host: torch.Tensor                 # pinned uint8 image
    dev: Optional[torch.Tensor] = None  # device copy

    def upload(self, device="cuda", stream=None) -> "_Plan":
        """One asynchronous host-to-device copy of the packed image (pa_upload)."""
        n = int(self.meta.total_bytes)
        if self.dev is None or self.dev.numel() < n:
            self.dev = torch.empty(max(n, 256), dtype=torch.uint8, device=device)
        _check(lib().pa_upload(_ptr(self.dev), _ptr(self.host), n, _stream(stream)), "pa_upload")
        return self

    def dptr(self, off: int) -> int:
        assert self.dev is not None, "upload the plan first"
        return self.dev.data_ptr() + int(off)

    def host_array(self, off: int, count: int) -> np.ndarray:
        """Read back a packed int32 array from the host image (tests/debugging)."""
        buf = self.host.numpy()
        return np.frombuffer(buf, dtype=np.int32, count=count, offset=int(off)).copy()


class PrefillPlan(_Plan):
    @property
    def slot_mapping(self) -> int:
        return self.dptr(self.meta.off_slot_mapping)


class DecodePlan(_Plan):
    @property
    def slot_mapping(self) -> int:
        return self.dptr(self.meta.off_slot_mapping)


class SharedPlan(_Plan):
    num_rows = 0       # rows that the block table must have
    call_shape = None  # of the plan that was uploaded: those rows, and the table's width

    def upload(self, device="cuda", stream=None) -> "SharedPlan":
        super().upload(device, stream)
        m, base = self.meta, self.dev.data_ptr()
        self.device = self.dev.get_device()
        self.call_shape = (self.num_rows, m.max_blocks_per_seq)
        self.call_ref = ctypes.byref(m)
        self.call_tables = base + m.off_block_tables if m.tables_packed or m.num_seqs == 0 else None
        self.call_arrays = tuple(base + x for x in (m.off_items, m.off_cta_items, m.off_seq_parts, m.off_direct_items,
                                                   m.off_table_rows, m.off_single_items))
        self.call_tiles = base + m.off_scratch_tiles
        # what a call's tensors hold at least: q and out, a page of a cache, a page's scales
        self.call_rows = m.num_seqs * m.num_heads * m.head_dim
        self.call_scales = m.block_size * m.num_kv_heads
        self.call_page = self.call_scales * m.head_dim
        return self

    @property
    def slot_mapping(self) -> int:
        """Device address of each last token's slot (plans packed from block lists)."""
        assert self.meta.tables_packed, "the plan was packed for device tables: the slots are the caller's"
        return self.dptr(self.meta.off_slot_mapping)


def _pack(fn_name, meta, args, into, pin, cls):
    fn = getattr(lib(), fn_name)
    host = into.host if into is not None else None
    if host is None:
        _check(fn(*args, None, 0, ctypes.byref(meta)), fn_name)
        host = torch.empty(max(int(meta.total_bytes), 256), dtype=torch.uint8, pin_memory=pin)
    rc = fn(*args, _ptr(host), host.numel(), ctypes.byref(meta))
    if rc == PA_ERR_WORKSPACE:  # reused buffer too small: grow it
        host = torch.empty(int(meta.total_bytes), dtype=torch.uint8, pin_memory=pin)
        rc = fn(*args, _ptr(host), host.numel(), ctypes.byref(meta))
    _check(rc, fn_name)
    if into is not None:
        into.meta, into.host = meta, host
        return into
    return cls(meta, host)


def pa_pack_prefill(dims: pa_dims, seq_lens, query_lens, block_lists, pin: bool = True,
                    into: Optional["PrefillPlan"] = None) -> "PrefillPlan":
    """Pack cu_seqlens, block tables, slot mapping and the tile list on the CPU.

    ``into`` reuses an earlier plan's pinned buffer (the caller must make sure
    no copy from it is still in flight).
    """
    seq_lens, query_lens = _i32(seq_lens), _i32(query_lens)
    off, ids = _flatten(block_lists)
    args = (ctypes.byref(dims), len(seq_lens), _np_ptr(seq_lens), _np_ptr(query_lens), _np_ptr(off), _np_ptr(ids))
    return _pack("pa_pack_prefill", pa_prefill_meta(), args, into, pin, PrefillPlan)


def pa_pack_decode(dims: pa_dims, context_lens, block_lists, split_tokens: int = 0, pin: bool = True,
                   into: Optional["DecodePlan"] = None) -> "DecodePlan":
    """Pack context lens, block tables, slot mapping and the split plan on the CPU."""
    ctx = _i32(context_lens)
    off, ids = _flatten(block_lists)
    args = (ctypes.byref(dims), len(ctx), _np_ptr(ctx), _np_ptr(off), _np_ptr(ids), int(split_tokens))
    return _pack("pa_pack_decode", pa_decode_meta(), args, into, pin, DecodePlan)


def pa_pack_decode_fixed(dims: pa_dims, context_lens, block_lists, max_context: int, split_tokens: int = 0,
                         pin: bool = True, into: Optional["DecodePlan"] = None) -> "DecodePlan":
    """Decode plan whose shapes depend only on (dims, len(context_lens), max_context, split_tokens).

    Padding entries have context 0 and an empty block list.  With ``into`` the
    previous plan's pinned buffer (and, after ``upload``, its device buffer)
    is reused, so launches captured in a CUDA graph stay valid.
    """
    ctx = _i32(context_lens)
    off, ids = _flatten(block_lists)
    args = (ctypes.byref(dims), len(ctx), _np_ptr(ctx), _np_ptr(off), _np_ptr(ids), int(max_context),
            int(split_tokens))
    return _pack("pa_pack_decode_fixed", pa_decode_meta(), args, into, pin, DecodePlan)


def pa_pack_decode_shared(dims: pa_dims, context_lens, group_offsets=None, shared_lens=None, block_lists=None,
                          table_rows=None, max_blocks: int = 0, split_tokens: int = 0, pin: bool = True,
                          into: Optional["SharedPlan"] = None) -> "SharedPlan":
    """Plan of a decode batch whose sequences share prefixes within groups of consecutive ones.

    ``group_offsets`` None is one group of all.  With ``block_lists`` the tables are packed and the
    shared length of each group is found (or, with ``shared_lens``, checked); without, the plan is for
    a block table on the device (row ``table_rows[b]`` of it, ``max_blocks`` wide) and ``shared_lens``
    is needed.
    """
    ctx = _i32(context_lens)
    groups = _i32([0, len(ctx)] if group_offsets is None else group_offsets)
    shared = None if shared_lens is None else _i32(shared_lens)
    if shared is not None and len(shared) != len(groups) - 1:
        raise ValueError(f"shared_lens has {len(shared)} entries for {len(groups) - 1} groups")
    rows = None if table_rows is None else _i32(table_rows)
    if rows is not None and len(rows) != len(ctx):
        raise ValueError(f"table_rows has {len(rows)} entries for {len(ctx)} sequences")
    off, ids = (None, None) if block_lists is None else _flatten(block_lists)
    if off is not None and len(off) != len(ctx) + 1:
        raise ValueError(f"block_lists has {len(off) - 1} entries for {len(ctx)} sequences")
    opt = lambda a: None if a is None else _np_ptr(a)
    args = (ctypes.byref(dims), len(ctx), _np_ptr(ctx), len(groups) - 1, _np_ptr(groups), opt(shared), opt(off),
            opt(ids), opt(rows), int(max_blocks), int(split_tokens))
    plan = _pack("pa_pack_decode_shared", pa_shared_meta(), args, into, pin, SharedPlan)
    plan.num_rows = len(ctx) if rows is None or len(rows) == 0 else int(rows.max()) + 1
    return plan


def pa_upload(dev_dst, host_src, nbytes: int, stream=None):
    _check(lib().pa_upload(_ptr(dev_dst), _ptr(host_src), int(nbytes), _stream(stream)), "pa_upload")


def pa_store_kvcache(dims: pa_dims, k, v, k_cache, v_cache, slot_mapping, num_tokens: Optional[int] = None,
                     stream=None):
    n = int(k.shape[0]) if num_tokens is None else int(num_tokens)
    _check(lib().pa_store_kvcache(ctypes.byref(dims), _ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache),
                                  _ptr(slot_mapping), n, _stream(stream)), "pa_store_kvcache")


def pa_prefill_varlen(dims: pa_dims, q, k_cache, v_cache, plan: PrefillPlan, scale: float, out, stream=None):
    m = plan.meta
    _check(lib().pa_prefill_varlen(ctypes.byref(dims), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                   plan.dptr(m.off_cu_seqlens_q), plan.dptr(m.off_cu_seqlens_k),
                                   plan.dptr(m.off_block_tables), float(scale), _ptr(out), ctypes.byref(m),
                                   plan.dptr(m.off_tiles), _stream(stream)), "pa_prefill_varlen")


def pa_prefill_varlen_fused(dims: pa_dims, q, k, v, k_cache, v_cache, plan: PrefillPlan, scale: float, out,
                            stream=None):
    """pa_store_kvcache of the new tokens' k/v at the plan's slots + pa_prefill_varlen, in one launch."""
    m = plan.meta
    _check(lib().pa_prefill_varlen_fused(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache),
                                         plan.dptr(m.off_cu_seqlens_q), plan.dptr(m.off_cu_seqlens_k),
                                         plan.dptr(m.off_block_tables), plan.dptr(m.off_slot_mapping), float(scale),
                                         _ptr(out), ctypes.byref(m), plan.dptr(m.off_tiles), _stream(stream)),
           "pa_prefill_varlen_fused")


def decode_workspace(plan: DecodePlan, device="cuda") -> Optional[torch.Tensor]:
    n = int(plan.meta.workspace_bytes)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def pa_decode(dims: pa_dims, q, k_cache, v_cache, plan: DecodePlan, scale: float, out, workspace=None,
              stream=None):
    m = plan.meta
    ws_bytes = int(workspace.numel()) if isinstance(workspace, torch.Tensor) else 0
    _check(lib().pa_decode(ctypes.byref(dims), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                           plan.dptr(m.off_context_lens), plan.dptr(m.off_block_tables), float(scale), _ptr(out),
                           ctypes.byref(m), plan.dptr(m.off_items), plan.dptr(m.off_seq_items), _ptr(workspace),
                           ws_bytes, _stream(stream)), "pa_decode")


def pa_decode_fused(dims: pa_dims, q, k, v, k_cache, v_cache, plan: DecodePlan, scale: float, out, workspace=None,
                    stream=None):
    """Store each sequence's new K/V row and decode, in one launch (pa_store_kvcache + pa_decode)."""
    m = plan.meta
    ws_bytes = int(workspace.numel()) if isinstance(workspace, torch.Tensor) else 0
    _check(lib().pa_decode_fused(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache),
                                 plan.dptr(m.off_slot_mapping), plan.dptr(m.off_context_lens),
                                 plan.dptr(m.off_block_tables), float(scale), _ptr(out), ctypes.byref(m),
                                 plan.dptr(m.off_items), plan.dptr(m.off_seq_items), _ptr(workspace), ws_bytes,
                                 _stream(stream)), "pa_decode_fused")


def pa_decode_static(dims: pa_dims, q, k_cache, v_cache, plan: DecodePlan, scale: float, out, stream=None):
    """pa_decode without a workspace, for callers that cannot allocate device memory.

    The library's own 16 MiB scratch array stands in for the workspace; every
    call on a device shares it, so calls must not overlap on the GPU.  The
    first call on a device does a one-time address lookup: make it before any
    stream capture.
    """
    m = plan.meta
    _check(lib().pa_decode_static(ctypes.byref(dims), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                  plan.dptr(m.off_context_lens), plan.dptr(m.off_block_tables), float(scale),
                                  _ptr(out), ctypes.byref(m), plan.dptr(m.off_items), plan.dptr(m.off_seq_items),
                                  _stream(stream)), "pa_decode_static")


def shared_workspace(plan: SharedPlan, device="cuda", int8: bool = True) -> Optional[torch.Tensor]:
    """Workspace of a shared-prefix decode on either cache; with int8=False only pa_decode_shared's (without
    the fp16 copy of the shared parts)."""
    n = int(plan.meta.workspace_bytes)
    if int8:
        n = max(n, int(plan.meta.workspace_bytes_int8))
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def _shared_tables(plan: SharedPlan, block_tables) -> int:
    """Address of the block tables of a shared-prefix decode: the plan's, or the caller's."""
    assert plan.dev is not None, "upload the plan first"
    if block_tables is None:
        if plan.call_tables is None:
            raise ValueError("the plan was packed for device tables: pass block_tables")
        return plan.call_tables
    at = _int32(block_tables, "block_tables")
    rows, width = plan.call_shape or (plan.num_rows, plan.meta.max_blocks_per_seq)
    if block_tables.dim() != 2 or block_tables.shape[1] != width or block_tables.shape[0] < rows:
        raise ValueError(f"block_tables must be [{rows} rows or more, {width}]")
    return at


def pa_decode_shared(dims: pa_dims, q, k_cache, v_cache, plan: SharedPlan, scale: float, out, workspace=None,
                     block_tables=None, stream=None):
    """pa_decode of a batch whose groups share prefixes: each shared block is read once per group.

    ``block_tables``: the device table a plan without block lists was packed for.
    """
    bt = (plan.call_tables if block_tables is None and plan.dev is not None else None) or _shared_tables(plan, block_tables)
    dev = _device()
    ws, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    cached = dims.num_blocks * plan.call_page
    if not (plan.device == dev == q.get_device() == k_cache.get_device() == v_cache.get_device() == out.get_device()
            and q.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous() and out.is_contiguous()
            and q.dtype is k_cache.dtype is v_cache.dtype is out.dtype is _BF16
            and q.numel() >= plan.call_rows <= out.numel() and k_cache.numel() >= cached <= v_cache.numel()
            and (workspace is None or workspace.get_device() == dev and workspace.is_contiguous())
            and (block_tables is None or block_tables.get_device() == dev)):
        _refuse(plan.device, (q, k_cache, v_cache, out, workspace, block_tables),
                (("q", q, _BF16, plan.call_rows), ("k_cache", k_cache, _BF16, cached), ("v_cache", v_cache, _BF16, cached),
                 ("out", out, _BF16, plan.call_rows)))
    rc = (_lib or lib()).pa_decode_shared(ctypes.byref(dims), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), bt,
                                          scale, out.data_ptr(), plan.call_ref, *plan.call_arrays, ws, ws_bytes,
                                          _raw_stream(dev) if stream is None and _raw_stream else _stream(stream))
    if rc != PA_OK:
        _check(rc, "pa_decode_shared")


def pa_decode_shared_int8(dims: pa_dims, q, k_cache, v_cache, k_scale, v_scale, plan: SharedPlan, scale: float, out,
                          workspace=None, block_tables=None, stream=None):
    """pa_decode_shared over an INT8 cache (same plan and workspace)."""
    bt = (plan.call_tables if block_tables is None and plan.dev is not None else None) or _shared_tables(plan, block_tables)
    dev = _device()
    ws, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    pages = dims.num_blocks
    cached, scales = pages * plan.call_page, pages * plan.call_scales
    if not (plan.device == dev == q.get_device() == k_cache.get_device() == v_cache.get_device() == out.get_device()
            == k_scale.get_device() == v_scale.get_device()
            and q.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous() and out.is_contiguous()
            and k_scale.is_contiguous() and v_scale.is_contiguous()
            and q.dtype is out.dtype is _BF16 and k_cache.dtype is v_cache.dtype is _INT8
            and k_scale.dtype is v_scale.dtype is _FP16 and q.numel() >= plan.call_rows <= out.numel()
            and k_cache.numel() >= cached <= v_cache.numel() and k_scale.numel() >= scales <= v_scale.numel()
            and (workspace is None or workspace.get_device() == dev and workspace.is_contiguous())
            and (block_tables is None or block_tables.get_device() == dev)):
        _refuse(plan.device, (q, k_cache, v_cache, k_scale, v_scale, out, workspace, block_tables),
                (("q", q, _BF16, plan.call_rows), ("k_cache", k_cache, _INT8, cached), ("v_cache", v_cache, _INT8, cached),
                 ("k_scale", k_scale, _FP16, scales), ("v_scale", v_scale, _FP16, scales),
                 ("out", out, _BF16, plan.call_rows)))
    rc = (_lib or lib()).pa_decode_shared_int8(ctypes.byref(dims), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                               k_scale.data_ptr(), v_scale.data_ptr(), bt, scale, out.data_ptr(),
                                               plan.call_ref, *plan.call_arrays, plan.call_tiles, ws, ws_bytes,
                                               _raw_stream(dev) if stream is None and _raw_stream else _stream(stream))
    if rc != PA_OK:
        _check(rc, "pa_decode_shared_int8")


def pa_copy_blocks(dims: pa_dims, k_cache, v_cache, triples, num_triples: Optional[int] = None, stream=None):
    """Copy the first n rows of block src to block dst (K and V) for each (src, dst, n) triple."""
    n = int(triples.shape[0]) if num_triples is None else int(num_triples)
    _check(lib().pa_copy_blocks(ctypes.byref(dims), _ptr(k_cache), _ptr(v_cache), _ptr(triples), n,
                                _stream(stream)), "pa_copy_blocks")


class PagePool:
    """A page pool on the device: block tables, context lengths, reference counts and the pages of all layers.

    k_cache, v_cache: [layers, num_blocks, block_size, Hkv, D] (or one layer without that dimension), each
    layer contiguous; bf16, or int8 with k_scale, v_scale fp16 [layers, num_blocks, Hkv, block_size].
    block_tables int32 [rows, max_blocks], context_lens int32 [rows], ref_counts int32 [num_blocks].
    """

    def __init__(self, dims: pa_dims, k_cache, v_cache, block_tables, context_lens, ref_counts, k_scale=None,
                 v_scale=None):
        rows, width = block_tables.shape
        _int32(block_tables, "block_tables")
        _int32(context_lens, "context_lens", rows)
        _int32(ref_counts, "ref_counts", dims.num_blocks)
        if (k_scale is None) != (v_scale is None):
            raise ValueError("k_scale and v_scale go together")
        page = (dims.num_blocks, dims.block_size, dims.num_kv_heads, dims.head_dim)
        scale = (dims.num_blocks, dims.num_kv_heads, dims.block_size)
        k, v = self._layers(k_cache, page, k_scale is not None), self._layers(v_cache, page, k_scale is not None)
        ks, vs = ((None, None) if k_scale is None else (self._layers(x, scale, None) for x in (k_scale, v_scale)))
        parts = [x for x in (k, v, ks, vs) if x is not None]
        if any(x.shape[0] != k.shape[0] for x in parts) or k.stride(0) != v.stride(0) or \
                (ks is not None and ks.stride(0) != vs.stride(0)):
            raise ValueError("K and V (and their scales) must agree in layers and in the stride between them")
        if any(x.device != block_tables.device for x in parts + [context_lens, ref_counts]):
            raise ValueError("the pool's arrays must be on one device")
        self.block_tables, self.context_lens, self.ref_counts = block_tables, context_lens, ref_counts
        self.k_cache, self.v_cache, self.k_scale, self.v_scale = k_cache, v_cache, k_scale, v_scale
        self.struct = pa_pool(rows, width, k.shape[0], 0, _ptr(block_tables), _ptr(context_lens), _ptr(ref_counts),
                              _ptr(k), _ptr(v), _ptr(ks), _ptr(vs), k.stride(0) * k.element_size(),
                              0 if ks is None else ks.stride(0) * ks.element_size())
        self.ref = ctypes.byref(self.struct)
        n = ctypes.c_uint64(0)
        _check(lib().pa_pool_workspace(ctypes.byref(dims), self.ref, ctypes.byref(n)), "pa_pool_workspace")
        self.workspace = torch.empty(n.value, dtype=torch.uint8, device=block_tables.device)
        self.ws = (self.workspace.data_ptr(), n.value)
        self.device = block_tables.get_device()
        self.dims = pa_dims.from_buffer_copy(dims)  # the calls go by this copy
        self.dims_ref, self.dims_bytes = ctypes.byref(self.dims), bytes(dims)

    def check(self, dims: pa_dims) -> None:
        """Refuses a call with other dims than the pool's, or made with another device current."""
        if bytes(dims) != self.dims_bytes:
            raise ValueError("the pool was made with other dims")
        if self.device < 0 or _device() != self.device:
            raise ValueError(f"the pool is on {self.block_tables.device}, which is not the current CUDA device")

    @staticmethod
    def _layers(x, shape, int8):
        """x as [layers, *shape], each layer contiguous."""
        want = torch.float16 if int8 is None else torch.int8 if int8 else torch.bfloat16
        x = x.unsqueeze(0) if x.dim() == len(shape) else x
        if x.dtype != want or tuple(x.shape[1:]) != shape or not x[0].is_contiguous():
            raise ValueError(f"expected {want} [layers, {', '.join(map(str, shape))}] with contiguous layers, got "
                             f"{x.dtype} {tuple(x.shape)}")
        return x


def page_pool(dims: pa_dims, k_cache, v_cache, num_rows: int, max_blocks: int, k_scale=None, v_scale=None) -> PagePool:
    """An empty pool over the given caches."""
    new = lambda *shape, fill: torch.full(shape, fill, dtype=torch.int32, device=k_cache.device)
    return PagePool(dims, k_cache, v_cache, new(num_rows, max_blocks, fill=-1), new(num_rows, fill=0),
                    new(dims.num_blocks, fill=0), k_scale, v_scale)


def pa_pool_append(dims: pa_dims, pool: PagePool, rows, cu_new, slot_mapping, stream=None):
    """Give row rows[i] its next cu_new[i+1] - cu_new[i] tokens; their slots go to slot_mapping."""
    dev, n, tokens = pool.device, rows.numel(), slot_mapping.numel()
    args = (_int32(rows, "rows", None, dev), _int32(cu_new, "cu_new", n + 1, dev), n,
            _int32(slot_mapping, "slot_mapping", None, dev), tokens)
    pool.check(dims)
    rc = (_lib or lib()).pa_pool_append(pool.dims_ref, pool.ref, *args, *pool.ws, _stream_of(pool.device, stream))
    if rc != PA_OK:
        _check(rc, "pa_pool_append")


def pa_pool_fork(dims: pa_dims, pool: PagePool, parents, children, stream=None):
    """Row children[i] shares row parents[i]'s full pages and gets a copy of its partly filled one."""
    dev, n = pool.device, children.numel()
    args = (_int32(parents, "parents", n, dev), _int32(children, "children", None, dev), n)
    pool.check(dims)
    rc = (_lib or lib()).pa_pool_fork(pool.dims_ref, pool.ref, *args, *pool.ws, _stream_of(pool.device, stream))
    if rc != PA_OK:
        _check(rc, "pa_pool_fork")


def pa_pool_free(dims: pa_dims, pool: PagePool, rows, stream=None):
    """Empty the rows and give their pages back."""
    at = _int32(rows, "rows", None, pool.device)
    pool.check(dims)
    rc = (_lib or lib()).pa_pool_free(pool.dims_ref, pool.ref, at, rows.numel(), _stream_of(pool.device, stream))
    if rc != PA_OK:
        _check(rc, "pa_pool_free")


def pa_pool_compact(dims: pa_dims, pool: PagePool, remap, block_tables_out=None, ref_counts_out=None, stream=None):
    """Move the used pages to the lowest ids; remap[p] is page p's new id.  Tables and counts are rewritten in
    place, or into the given arrays."""
    dev = pool.device
    tables = pool.block_tables if block_tables_out is None else block_tables_out
    refs = pool.ref_counts if ref_counts_out is None else ref_counts_out
    pages = pool.ref_counts.numel()
    args = (_int32(remap, "remap", pages, dev), _int32(tables, "block_tables_out", pool.block_tables.numel(), dev),
            _int32(refs, "ref_counts_out", pages, dev))
    pool.check(dims)
    rc = (_lib or lib()).pa_pool_compact(pool.dims_ref, pool.ref, *args, *pool.ws, _stream_of(pool.device, stream))
    if rc != PA_OK:
        _check(rc, "pa_pool_compact")


def int8_cache(dims: pa_dims, device="cuda"):
    """Allocate an empty INT8 cache: (k_codes, v_codes, k_scale, v_scale).

    Codes int8 [num_blocks, block_size, Hkv, D]; scales fp16 [num_blocks, Hkv, block_size].
    """
    shape = (dims.num_blocks, dims.block_size, dims.num_kv_heads, dims.head_dim)
    sshape = (dims.num_blocks, dims.num_kv_heads, dims.block_size)
    return (torch.zeros(shape, dtype=torch.int8, device=device), torch.zeros(shape, dtype=torch.int8, device=device),
            torch.zeros(sshape, dtype=torch.float16, device=device),
            torch.zeros(sshape, dtype=torch.float16, device=device))


def pa_store_kvcache_int8(dims: pa_dims, k, v, k_cache, v_cache, k_scale, v_scale, slot_mapping,
                          num_tokens: Optional[int] = None, stream=None):
    """Quantise each new token's K/V head vectors (bf16) into int8 codes + fp16 scales at its slot."""
    n = int(k.shape[0]) if num_tokens is None else int(num_tokens)
    _check(lib().pa_store_kvcache_int8(ctypes.byref(dims), _ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache),
                                       _ptr(k_scale), _ptr(v_scale), _ptr(slot_mapping), n, _stream(stream)),
           "pa_store_kvcache_int8")


def prefill_workspace(plan: PrefillPlan, device="cuda") -> Optional[torch.Tensor]:
    """The INT8 prefill's workspace (its bf16 scratch cache) for this plan."""
    n = int(plan.meta.workspace_bytes)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def _call_workspace(plan: PrefillPlan, workspace, device, stream):
    """The caller's workspace, or one allocated for this call (kept from reuse until the
    call's stream has passed it)."""
    if workspace is None:
        workspace = prefill_workspace(plan, device)
        if workspace is not None and stream is not None:
            st = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
            workspace.record_stream(st)
    return workspace


def pa_prefill_varlen_int8(dims: pa_dims, q, k_cache, v_cache, k_scale, v_scale, plan: PrefillPlan, scale: float,
                           out, workspace=None, stream=None):
    """pa_prefill_varlen over an INT8 cache (same plan as pa_prefill_varlen; workspace of
    plan.meta.workspace_bytes, allocated here when not given)."""
    m = plan.meta
    workspace = _call_workspace(plan, workspace, q.device, stream)
    ws_bytes = int(workspace.numel()) if isinstance(workspace, torch.Tensor) else 0
    _check(lib().pa_prefill_varlen_int8(ctypes.byref(dims), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
                                        _ptr(v_scale), plan.dptr(m.off_cu_seqlens_q), plan.dptr(m.off_cu_seqlens_k),
                                        plan.dptr(m.off_block_tables), plan.dptr(m.off_scratch_tables),
                                        plan.dptr(m.off_scratch_items), float(scale), _ptr(out), ctypes.byref(m),
                                        plan.dptr(m.off_tiles), _ptr(workspace), ws_bytes, _stream(stream)),
           "pa_prefill_varlen_int8")


def pa_prefill_varlen_int8_fused(dims: pa_dims, q, k, v, k_cache, v_cache, k_scale, v_scale, plan: PrefillPlan,
                                 scale: float, out, workspace=None, stream=None):
    """pa_store_kvcache_int8 of the new tokens' k/v at the plan's slots + pa_prefill_varlen_int8, in one call."""
    m = plan.meta
    workspace = _call_workspace(plan, workspace, q.device, stream)
    ws_bytes = int(workspace.numel()) if isinstance(workspace, torch.Tensor) else 0
    _check(lib().pa_prefill_varlen_int8_fused(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(k_cache),
                                              _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
                                              plan.dptr(m.off_cu_seqlens_q), plan.dptr(m.off_cu_seqlens_k),
                                              plan.dptr(m.off_block_tables), plan.dptr(m.off_slot_mapping),
                                              plan.dptr(m.off_scratch_tables), plan.dptr(m.off_scratch_items),
                                              float(scale), _ptr(out), ctypes.byref(m), plan.dptr(m.off_tiles),
                                              _ptr(workspace), ws_bytes, _stream(stream)),
           "pa_prefill_varlen_int8_fused")


def pa_decode_int8_fused(dims: pa_dims, q, k, v, k_cache, v_cache, k_scale, v_scale, plan: DecodePlan,
                         scale: float, out, workspace=None, stream=None):
    """Quantising store of each sequence's new K/V row + INT8 decode, in one launch."""
    m = plan.meta
    ws_bytes = int(workspace.numel()) if isinstance(workspace, torch.Tensor) else 0
    _check(lib().pa_decode_int8_fused(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache),
                                      _ptr(k_scale), _ptr(v_scale), plan.dptr(m.off_slot_mapping),
                                      plan.dptr(m.off_context_lens), plan.dptr(m.off_block_tables), float(scale),
                                      _ptr(out), ctypes.byref(m), plan.dptr(m.off_items), plan.dptr(m.off_seq_items),
                                      _ptr(workspace), ws_bytes, _stream(stream)), "pa_decode_int8_fused")


def pa_decode_int8(dims: pa_dims, q, k_cache, v_cache, k_scale, v_scale, plan: DecodePlan, scale: float, out,
                   workspace=None, stream=None):
    """pa_decode over an INT8 cache (same plan and workspace as pa_decode)."""
    m = plan.meta
    ws_bytes = int(workspace.numel()) if isinstance(workspace, torch.Tensor) else 0
    _check(lib().pa_decode_int8(ctypes.byref(dims), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
                                _ptr(v_scale), plan.dptr(m.off_context_lens), plan.dptr(m.off_block_tables),
                                float(scale), _ptr(out), ctypes.byref(m), plan.dptr(m.off_items),
                                plan.dptr(m.off_seq_items), _ptr(workspace), ws_bytes, _stream(stream)),
           "pa_decode_int8")


def pa_copy_blocks_int8(dims: pa_dims, k_cache, v_cache, k_scale, v_scale, triples,
                        num_triples: Optional[int] = None, stream=None):
    """pa_copy_blocks on an INT8 cache: codes and each KV head's scale run."""
    n = int(triples.shape[0]) if num_triples is None else int(num_triples)
    _check(lib().pa_copy_blocks_int8(ctypes.byref(dims), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
                                     _ptr(v_scale), _ptr(triples), n, _stream(stream)), "pa_copy_blocks_int8")


def pa_selftest_bounded_wait(timeout_us: int, arrive_first: bool = False, stream=None):
    """Run the library's bounded mbarrier wait on a barrier nothing completes (or, with
    arrive_first, one it completes itself); a timeout shows as bit 4 of pa_read_device_error."""
    _check(lib().pa_selftest_bounded_wait(ctypes.c_uint32(int(timeout_us)), 1 if arrive_first else 0, _stream(stream)),
           "pa_selftest_bounded_wait")


def pa_stream_read(src: torch.Tensor, sink: torch.Tensor, stream=None):
    """Read every byte of the device tensor `src` once (streaming loads): the read-only
    bandwidth that bounds the decode kernels.  `sink` is a 4-byte device tensor."""
    _check(lib().pa_stream_read(_ptr(src), src.numel() * src.element_size(), _ptr(sink), _stream(stream)),
           "pa_stream_read")


def pa_read_device_error(stream=None) -> int:
    code = ctypes.c_uint32(0)
    _check(lib().pa_read_device_error(ctypes.byref(code), _stream(stream)), "pa_read_device_error")
    return int(code.value)
