"""ctypes binding of libmla_gb300.so (argument marshalling only).

Every function mirrors one C entry point of ``include/mla_gb300.h``: torch
tensors are checked for dtype / device / contiguity, their device pointers and
the current CUDA stream are passed through, and a non-OK status raises
``MLAError``.  All compute happens in the library's CUDA kernels; there is no
fallback path.  Call ``mla_decode_speculative_gb300.build.build()`` first (or
``__graft_entry__.build()``); loading a missing library raises.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
import threading
from typing import Optional

import torch

from . import build as _build

D_QK = 576
D_V = 512

MLA_OK = 0
MLA_ERR_INVALID_ARG = 1
MLA_ERR_UNSUPPORTED = 2
MLA_ERR_WORKSPACE = 3
MLA_ERR_CUDA = 4
MLA_ERR_DEVICE_CHECK = 5

MLA_KV_BF16 = 0
MLA_KV_FP8_E4M3 = 1
MLA_MERGE_SEGMENTS = 0
MLA_MERGE_STATES = 1
MLA_DECODE_SKIP_MERGE = 1
MLA_DECODE_UNIFORM_SEGMENTS = 2
MLA_DECODE_FUSED_MERGE = 4

DEVICE_ERRORS = {0: "MLA_DEV_OK", 1: "MLA_DEV_BAD_INDPTR", 2: "MLA_DEV_BAD_QLEN",
                 3: "MLA_DEV_BAD_BLOCK_ID", 4: "MLA_DEV_LEN_BOUND", 5: "MLA_DEV_BAD_SUBPAGE",
                 6: "MLA_DEV_WAIT_TIMEOUT", 7: "MLA_DEV_NO_FREE_BLOCK", 8: "MLA_DEV_BAD_FREE_RING",
                 9: "MLA_DEV_BAD_AXIS"}


class MLAError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


class DecodeArgs(ctypes.Structure):
    _fields_ = [("num_reqs", ctypes.c_int), ("num_rows", ctypes.c_int),
                ("num_heads", ctypes.c_int), ("max_qlen", ctypes.c_int),
                ("kv_dtype", ctypes.c_int), ("sm_scale", ctypes.c_float),
                ("kv_scale", ctypes.c_float), ("q", ctypes.c_void_p),
                ("kv_cache", ctypes.c_void_p), ("num_cache_rows", ctypes.c_int64),
                ("qo_indptr", ctypes.c_void_p), ("row_len", ctypes.c_void_p),
                ("subpage_table", ctypes.c_void_p), ("subpage_stride", ctypes.c_int),
                ("page_size", ctypes.c_int), ("num_segments", ctypes.c_int),
                ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("flags", ctypes.c_int),
                ("num_views", ctypes.c_int), ("wait_cycles", ctypes.c_int64)]


class MergeArgs(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int), ("num_rows", ctypes.c_int), ("num_heads", ctypes.c_int),
                ("num_parts", ctypes.c_int), ("segm_out", ctypes.c_void_p),
                ("segm_max", ctypes.c_void_p), ("segm_sum", ctypes.c_void_p),
                ("qo_indptr", ctypes.c_void_p), ("num_reqs", ctypes.c_int),
                ("max_qlen", ctypes.c_int), ("num_views", ctypes.c_int), ("part_out", ctypes.c_void_p), ("part_lse", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p)]


class TableArgs(ctypes.Structure):
    _fields_ = [("num_reqs", ctypes.c_int), ("num_rows", ctypes.c_int),
                ("prev_lens", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("qo_indptr", ctypes.c_void_p), ("world_size", ctypes.c_int),
                ("rank", ctypes.c_int), ("interleave", ctypes.c_int),
                ("block_size", ctypes.c_int), ("num_blocks", ctypes.c_int),
                ("block_table", ctypes.c_void_p), ("block_table_stride", ctypes.c_int),
                ("free_ring", ctypes.c_void_p), ("ring_in", ctypes.c_void_p),
                ("ring_out", ctypes.c_void_p), ("slot_map", ctypes.c_void_p)]


class Heads(ctypes.Structure):
    _fields_ = [("heads", ctypes.c_int), ("dim", ctypes.c_int), ("src", ctypes.c_void_p),
                ("src_row", ctypes.c_int64), ("src_head", ctypes.c_int64), ("dst", ctypes.c_void_p),
                ("dst_row", ctypes.c_int64), ("dst_head", ctypes.c_int64)]


class RotaryArgs(ctypes.Structure):
    _fields_ = [("num_rows", ctypes.c_int), ("num_axes", ctypes.c_int), ("rot_dim", ctypes.c_int),
                ("neighbours", ctypes.c_int), ("positions", ctypes.c_void_p), ("axis_stride", ctypes.c_int64),
                ("turns", ctypes.c_void_p), ("axes", ctypes.c_void_p), ("q", Heads), ("k", Heads), ("v", Heads),
                ("slot_map", ctypes.c_void_p), ("num_cache_rows", ctypes.c_int64)]


class GroupedArgs(ctypes.Structure):
    _fields_ = [("num_reqs", ctypes.c_int), ("num_rows", ctypes.c_int), ("num_heads", ctypes.c_int),
                ("num_kv_heads", ctypes.c_int), ("max_qlen", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("window", ctypes.c_int), ("sm_scale", ctypes.c_float), ("q", ctypes.c_void_p),
                ("q_row", ctypes.c_int64), ("k_cache", ctypes.c_void_p), ("k_row", ctypes.c_int64),
                ("v_cache", ctypes.c_void_p), ("v_row", ctypes.c_int64), ("num_cache_rows", ctypes.c_int64),
                ("qo_indptr", ctypes.c_void_p), ("row_len", ctypes.c_void_p),
                ("subpage_table", ctypes.c_void_p), ("subpage_stride", ctypes.c_int),
                ("page_size", ctypes.c_int), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("wait_cycles", ctypes.c_int64)]


_lib = None
_lock = threading.Lock()
EXPORTS = ("mla_page_size", "mla_plan_rows", "mla_shard_row_view", "mla_shard_row_views",
           "mla_decode_verify_workspace",
           "mla_decode_verify", "mla_decode_verify_noalloc", "mla_write_kv", "mla_merge_segments",
           "mla_update_block_tables", "mla_update_block_tables_lens", "mla_write_kv_scaled", "mla_decode_verify_scaled",
           "mla_rotary", "mla_rotary_write", "mla_decode_grouped_workspace", "mla_decode_grouped",
           "mla_decode_differential", "mla_get_device_error",
           "mla_last_error_string", "mla_status_string", "mla_abi_version")


def library_path() -> str:
    return _build.LIB_PATH


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"libmla_gb300.so not built ({path}); run "
                               "mla_decode_speculative_gb300.build.build() first")
        L = ctypes.CDLL(path)
        i32p, vp, c_int = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int
        L.mla_page_size.argtypes = [c_int]
        L.mla_page_size.restype = c_int
        L.mla_plan_rows.argtypes = [c_int, c_int, i32p, i32p, i32p, i32p, i32p, c_int, c_int, c_int,
                                    i32p, c_int, vp]
        L.mla_plan_rows.restype = c_int
        L.mla_shard_row_view.argtypes = [c_int, c_int, i32p, i32p, c_int, c_int, c_int, i32p, i32p,
                                         c_int, c_int, c_int, i32p, c_int, vp]
        L.mla_shard_row_view.restype = c_int
        L.mla_shard_row_views.argtypes = [c_int, c_int, i32p, i32p, c_int, c_int, i32p, i32p, c_int,
                                          c_int, c_int, i32p, c_int, vp]
        L.mla_shard_row_views.restype = c_int
        L.mla_decode_verify_workspace.argtypes = [ctypes.POINTER(DecodeArgs)]
        L.mla_decode_verify_workspace.restype = ctypes.c_size_t
        L.mla_decode_verify.argtypes = [ctypes.POINTER(DecodeArgs), vp, ctypes.c_size_t, vp]
        L.mla_decode_verify.restype = c_int
        L.mla_decode_verify_noalloc.argtypes = [ctypes.POINTER(DecodeArgs), vp]
        L.mla_decode_verify_noalloc.restype = c_int
        L.mla_write_kv.argtypes = [c_int, c_int, i32p, i32p, vp, c_int, c_int, c_int, i32p, c_int,
                                   c_int, c_int, vp, c_int, ctypes.c_float, ctypes.c_int64, vp]
        L.mla_write_kv.restype = c_int
        L.mla_update_block_tables.argtypes = [ctypes.POINTER(TableArgs), vp]
        L.mla_update_block_tables.restype = c_int
        L.mla_update_block_tables_lens.argtypes = [ctypes.POINTER(TableArgs), vp, vp]
        L.mla_update_block_tables_lens.restype = c_int
        L.mla_write_kv_scaled.argtypes = [c_int, vp, i32p, vp, vp, c_int, ctypes.c_int64, vp]
        L.mla_write_kv_scaled.restype = c_int
        L.mla_decode_verify_scaled.argtypes = [ctypes.POINTER(DecodeArgs), vp, c_int, vp, ctypes.c_size_t, vp]
        L.mla_decode_verify_scaled.restype = c_int
        L.mla_rotary.argtypes = L.mla_rotary_write.argtypes = [ctypes.POINTER(RotaryArgs), vp]
        L.mla_rotary.restype = L.mla_rotary_write.restype = c_int
        L.mla_decode_grouped_workspace.argtypes = [ctypes.POINTER(GroupedArgs), c_int]
        L.mla_decode_grouped_workspace.restype = ctypes.c_size_t
        L.mla_decode_grouped.argtypes = [ctypes.POINTER(GroupedArgs), vp, ctypes.c_size_t, vp]
        L.mla_decode_grouped.restype = c_int
        L.mla_decode_differential.argtypes = [ctypes.POINTER(GroupedArgs), vp, vp, ctypes.c_float, vp,
                                              ctypes.c_size_t, vp]
        L.mla_decode_differential.restype = c_int
        L.mla_merge_segments.argtypes = [ctypes.POINTER(MergeArgs), vp]
        L.mla_merge_segments.restype = c_int
        L.mla_get_device_error.argtypes = [ctypes.POINTER(ctypes.c_int32), vp]
        L.mla_get_device_error.restype = c_int
        L.mla_last_error_string.restype = ctypes.c_char_p
        L.mla_status_string.argtypes = [c_int]
        L.mla_status_string.restype = ctypes.c_char_p
        L.mla_abi_version.restype = c_int
        _lib = L
        return _lib


def _check(status: int, what: str):
    if status != MLA_OK:
        L = lib()
        raise MLAError(status, f"{what}: {L.mla_status_string(status).decode()}: "
                               f"{L.mla_last_error_string().decode()}")


def _stream(stream=None) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _ptr(t: Optional[torch.Tensor], dtype=None, name: str = "tensor") -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def page_size(block_size: int) -> int:
    return int(lib().mla_page_size(int(block_size)))


def plan_rows(seq_lens: torch.Tensor, qo_indptr: torch.Tensor, num_rows: int,
              block_table: Optional[torch.Tensor] = None, num_blocks: int = 0,
              block_size: int = 0, subpage_stride: int = 0, row_len=None, row_req=None,
              subpage_table=None, stream=None):
    """mla_plan_rows.  Returns (row_len [T], row_req [T], subpage_table [B, stride] or None)."""
    B = int(seq_lens.shape[0])
    dev = seq_lens.device
    if row_len is None:
        row_len = torch.empty(num_rows, dtype=torch.int32, device=dev)
    if row_req is None:
        row_req = torch.empty(num_rows, dtype=torch.int32, device=dev)
    bt_stride = 0
    if block_table is not None:
        bt_stride = int(block_table.shape[1])
        if subpage_table is None:
            subpage_table = torch.empty((B, subpage_stride), dtype=torch.int32, device=dev)
    _check(lib().mla_plan_rows(B, int(num_rows), _ptr(seq_lens, torch.int32, "seq_lens"),
                               _ptr(qo_indptr, torch.int32, "qo_indptr"),
                               _ptr(row_len, torch.int32, "row_len"),
                               _ptr(row_req, torch.int32, "row_req"),
                               _ptr(block_table, torch.int32, "block_table"), bt_stride,
                               int(num_blocks), int(block_size),
                               _ptr(subpage_table, torch.int32, "subpage_table"),
                               int(subpage_stride), _stream(stream)), "mla_plan_rows")
    return row_len, row_req, subpage_table


def shard_row_view(qo_indptr: torch.Tensor, row_len_global: torch.Tensor, world_size: int,
                   rank: int, interleave: int = 1, block_table: Optional[torch.Tensor] = None,
                   num_blocks: int = 0, block_size: int = 0, subpage_stride: int = 0,
                   row_len_local=None, subpage_table=None, stream=None):
    """mla_shard_row_view.  Returns (row_len_local [T], subpage_table or None)."""
    B = int(qo_indptr.shape[0]) - 1
    T = int(row_len_global.shape[0])
    dev = row_len_global.device
    if row_len_local is None:
        row_len_local = torch.empty(T, dtype=torch.int32, device=dev)
    bt_stride = 0
    if block_table is not None:
        bt_stride = int(block_table.shape[1])
        if subpage_table is None:
            subpage_table = torch.empty((B, subpage_stride), dtype=torch.int32, device=dev)
    _check(lib().mla_shard_row_view(B, T, _ptr(qo_indptr, torch.int32, "qo_indptr"),
                                    _ptr(row_len_global, torch.int32, "row_len_global"),
                                    int(world_size), int(rank), int(interleave),
                                    _ptr(row_len_local, torch.int32, "row_len_local"),
                                    _ptr(block_table, torch.int32, "block_table"), bt_stride,
                                    int(num_blocks), int(block_size),
                                    _ptr(subpage_table, torch.int32, "subpage_table"),
                                    int(subpage_stride), _stream(stream)), "mla_shard_row_view")
    return row_len_local, subpage_table


def shard_row_views(qo_indptr: torch.Tensor, row_len_global: torch.Tensor, world_size: int,
                    interleave: int = 1, block_tables: Optional[torch.Tensor] = None,
                    num_blocks: int = 0, block_size: int = 0, subpage_stride: int = 0,
                    row_len_local=None, subpage_tables=None, stream=None):
    """mla_shard_row_views: all W views in one launch.  block_tables [W, B, width];
    returns (row_len_local [W, T], subpage_tables [W, B, stride] or None)."""
    B = int(qo_indptr.shape[0]) - 1
    T = int(row_len_global.shape[0])
    W = int(world_size)
    dev = row_len_global.device
    if row_len_local is None:
        row_len_local = torch.empty((W, T), dtype=torch.int32, device=dev)
    bt_stride = 0
    if block_tables is not None:
        bt_stride = int(block_tables.shape[-1])
        if subpage_tables is None:
            subpage_tables = torch.empty((W, B, subpage_stride), dtype=torch.int32, device=dev)
    _check(lib().mla_shard_row_views(B, T, _ptr(qo_indptr, torch.int32, "qo_indptr"),
                                     _ptr(row_len_global, torch.int32, "row_len_global"), W,
                                     int(interleave), _ptr(row_len_local, torch.int32, "row_len_local"),
                                     _ptr(block_tables, torch.int32, "block_tables"), bt_stride,
                                     int(num_blocks), int(block_size),
                                     _ptr(subpage_tables, torch.int32, "subpage_tables"),
                                     int(subpage_stride), _stream(stream)), "mla_shard_row_views")
    return row_len_local, subpage_tables


def make_decode_args(q, kv_cache, qo_indptr, row_len, subpage_table, page_size_, num_segments,
                     max_qlen, sm_scale, kv_scale=1.0, out=None, lse=None, flags=0,
                     num_views=1, wait_cycles=0) -> DecodeArgs:
    T, H, dk = q.shape
    if dk != D_QK:
        raise ValueError("q must be [T, H, 576]")
    fp8 = kv_cache.dtype == torch.uint8
    if kv_cache.dtype not in (torch.uint8, torch.bfloat16) or kv_cache.shape[-1] != D_QK:
        raise ValueError("kv_cache must be [N, 576] bf16 or uint8 (e4m3 codes)")
    a = DecodeArgs()
    a.num_reqs = int(qo_indptr.shape[0]) - 1
    a.num_rows = int(T)
    a.num_heads = int(H)
    a.max_qlen = int(max_qlen)
    a.kv_dtype = MLA_KV_FP8_E4M3 if fp8 else MLA_KV_BF16
    a.sm_scale = float(sm_scale)
    a.kv_scale = float(kv_scale)
    a.q = _ptr(q, torch.bfloat16, "q")
    a.kv_cache = _ptr(kv_cache, None, "kv_cache")
    a.num_cache_rows = int(kv_cache.numel() // D_QK)
    a.qo_indptr = _ptr(qo_indptr, torch.int32, "qo_indptr")
    a.row_len = _ptr(row_len, torch.int32, "row_len")
    a.subpage_table = _ptr(subpage_table, torch.int32, "subpage_table")
    a.subpage_stride = int(subpage_table.shape[-1])
    a.page_size = int(page_size_)
    a.num_segments = int(num_segments)
    a.out = _ptr(out, torch.bfloat16, "out")
    a.lse = _ptr(lse, torch.float32, "lse")
    a.flags = int(flags)
    a.num_views = int(num_views)
    a.wait_cycles = int(wait_cycles)
    return a


def decode_verify_workspace_bytes(a: DecodeArgs) -> int:
    return int(lib().mla_decode_verify_workspace(ctypes.byref(a)))


def decode_verify(q, kv_cache, qo_indptr, row_len, subpage_table, page_size_, num_segments,
                  max_qlen, sm_scale, kv_scale=1.0, out=None, lse=None, workspace=None,
                  stream=None, skip_merge=False, num_views=1, uniform_segments=False,
                  wait_cycles=0, fused_merge=False):
    """mla_decode_verify.  Returns (out [T, H, 512] bf16, lse [T, H] f32, workspace).
    skip_merge: leave the segment partials in the workspace (MLA_DECODE_SKIP_MERGE).
    uniform_segments: the pages' equal split per request (MLA_DECODE_UNIFORM_SEGMENTS)
    instead of the balanced split.
    num_views V > 1: row_len [V, T], subpage_table [V, B, stride]; out [V, T, H, 512],
    lse [V, T, H] (V row views of the same queries, one launch).
    wait_cycles: bound on each in-kernel wait in SM cycles (0 = the library default).
    fused_merge: merge the balanced split's parts inside the decode kernel
    (MLA_DECODE_FUSED_MERGE) instead of a separate merge launch."""
    T, H, _ = q.shape
    V = max(1, int(num_views))
    lead = (V, T) if V > 1 else (T,)
    if out is None:
        out = torch.empty((*lead, H, D_V), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((*lead, H), dtype=torch.float32, device=q.device)
    a = make_decode_args(q, kv_cache, qo_indptr, row_len, subpage_table, page_size_,
                         num_segments, max_qlen, sm_scale, kv_scale, out, lse,
                         (MLA_DECODE_SKIP_MERGE if skip_merge else 0) |
                         (MLA_DECODE_UNIFORM_SEGMENTS if uniform_segments else 0) |
                         (MLA_DECODE_FUSED_MERGE if fused_merge else 0), num_views=V,
                         wait_cycles=wait_cycles)
    need = decode_verify_workspace_bytes(a)
    if need and (workspace is None or workspace.numel() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = _ptr(workspace, torch.uint8, "workspace") if need else None
    _check(lib().mla_decode_verify(ctypes.byref(a), ws_ptr, need, _stream(stream)),
           "mla_decode_verify")
    return out, lse, workspace


STATIC_SCRATCH_BYTES = 80 * 1024 * 1024


def decode_verify_noalloc(q, kv_cache, qo_indptr, row_len, subpage_table, page_size_,
                          num_segments, max_qlen, sm_scale, kv_scale=1.0, out=None, lse=None,
                          stream=None):
    """mla_decode_verify_noalloc: the library's own static device scratch instead of a
    caller workspace, for callers that cannot allocate device memory at the call (serving
    runtimes that reserve all device memory at start-up, C or plugin hosts without a device
    allocator).  Calls that overlap on the GPU share that scratch and must be serialised.
    Returns (out, lse)."""
    T, H, _ = q.shape
    if out is None:
        out = torch.empty((T, H, D_V), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    a = make_decode_args(q, kv_cache, qo_indptr, row_len, subpage_table, page_size_,
                         num_segments, max_qlen, sm_scale, kv_scale, out, lse)
    _check(lib().mla_decode_verify_noalloc(ctypes.byref(a), _stream(stream)),
           "mla_decode_verify_noalloc")
    return out, lse


def row_blocks(max_qlen: int, num_heads: int) -> int:
    """RB: 64-row blocks per request in the segment-partial layout."""
    return -(-max_qlen * num_heads // 64)


def workspace_views(workspace: torch.Tensor, num_reqs: int, max_qlen: int, num_rows: int,
                    num_heads: int, num_segments: int, num_views: int = 1):
    """The documented workspace layout (num_views = 1): (segm_out [B, RB, S, 8, 512, 8] bf16
    blocks -- row octet, dim, row in octet --, segm_max [T, H, S], segm_sum [T, H, S]); V
    views stack V such layouts."""
    num_reqs, num_rows = num_reqs * num_views, num_rows * num_views
    items = num_rows * num_heads * num_segments
    blocks = num_reqs * row_blocks(max_qlen, num_heads) * num_segments
    a256 = lambda x: (x + 255) & ~255
    o_bytes = a256(blocks * 512 * 64 * 2)
    m_bytes = a256(items * 4)
    segm_out = workspace[:blocks * 512 * 64 * 2].view(torch.bfloat16).view(
        num_reqs, row_blocks(max_qlen, num_heads), num_segments, 8, 512, 8)
    segm_max = workspace[o_bytes:o_bytes + items * 4].view(torch.float32).view(num_rows, num_heads, num_segments)
    segm_sum = workspace[o_bytes + m_bytes:o_bytes + m_bytes + items * 4].view(torch.float32).view(
        num_rows, num_heads, num_segments)
    return segm_out, segm_max, segm_sum


def merge_segments(segm_out, segm_max, segm_sum, qo_indptr, max_qlen, out=None, lse=None,
                   stream=None, num_views=1):
    """mla_merge_segments, segment mode: bf16 partial blocks [V*B, RB, S, 8, 512, 8] (the
    decode workspace layout) + [V*T, H, S] f32 base-2 stats; qo_indptr [B + 1] int32.
    num_views V > 1: out [V, T, H, 512], lse [V, T, H] (the V row views of one decode)."""
    VT, H, S = segm_max.shape
    V = max(1, int(num_views))
    T = VT // V
    lead = (V, T) if V > 1 else (T,)
    if out is None:
        out = torch.empty((*lead, H, D_V), dtype=torch.bfloat16, device=segm_out.device)
    if lse is None:
        lse = torch.empty((*lead, H), dtype=torch.float32, device=segm_out.device)
    m = MergeArgs()
    m.mode, m.num_rows, m.num_heads, m.num_parts = MLA_MERGE_SEGMENTS, T, H, S
    m.segm_out = _ptr(segm_out, torch.bfloat16, "segm_out")
    m.qo_indptr = _ptr(qo_indptr, torch.int32, "qo_indptr")
    m.num_reqs = int(qo_indptr.shape[0]) - 1
    m.max_qlen = int(max_qlen)
    m.num_views = V
    m.segm_max = _ptr(segm_max, torch.float32, "segm_max")
    m.segm_sum = _ptr(segm_sum, torch.float32, "segm_sum")
    m.out = _ptr(out, torch.bfloat16, "out")
    m.lse = _ptr(lse, torch.float32, "lse")
    _check(lib().mla_merge_segments(ctypes.byref(m), _stream(stream)), "mla_merge_segments")
    return out, lse


def merge_states(part_out, part_lse, out=None, lse=None, stream=None):
    """mla_merge_segments, state mode: [W,T,H,512] bf16 + [W,T,H] natural-log LSE."""
    W, T, H, dv = part_out.shape
    if out is None:
        out = torch.empty((T, H, D_V), dtype=torch.bfloat16, device=part_out.device)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=part_out.device)
    m = MergeArgs()
    m.mode, m.num_rows, m.num_heads, m.num_parts = MLA_MERGE_STATES, T, H, W
    m.part_out = _ptr(part_out, torch.bfloat16, "part_out")
    m.part_lse = _ptr(part_lse, torch.float32, "part_lse")
    m.out = _ptr(out, torch.bfloat16, "out")
    m.lse = _ptr(lse, torch.float32, "lse")
    _check(lib().mla_merge_segments(ctypes.byref(m), _stream(stream)), "mla_merge_segments")
    return out, lse


def write_kv(seq_lens, qo_indptr, kv_new, kv_cache, block_table, num_blocks, block_size,
             world_size=1, rank=0, kv_scale=1.0, interleave=1, stream=None):
    """mla_write_kv: owner-filtered paged write of the new tokens (kv_new [T, 576]
    bf16) into this rank's cache (bf16 [N, 576], or uint8 e4m3 codes)."""
    fp8 = kv_cache.dtype == torch.uint8
    _check(lib().mla_write_kv(int(seq_lens.shape[0]), int(kv_new.shape[0]),
                              _ptr(seq_lens, torch.int32, "seq_lens"),
                              _ptr(qo_indptr, torch.int32, "qo_indptr"),
                              _ptr(kv_new, torch.bfloat16, "kv_new"), int(world_size), int(rank),
                              int(interleave), _ptr(block_table, torch.int32, "block_table"),
                              int(block_table.shape[1]), int(num_blocks), int(block_size),
                              _ptr(kv_cache, None, "kv_cache"),
                              MLA_KV_FP8_E4M3 if fp8 else MLA_KV_BF16, float(kv_scale),
                              int(kv_cache.numel() // D_QK), _stream(stream)), "mla_write_kv")
    return kv_cache


def _current(stream):
    """(library, current device, raw stream) of a call.  The handle of the current stream is read
    without making a Stream object, which takes as long as the launch."""
    dev = torch.cuda.current_device()
    raw = torch._C._cuda_getCurrentRawStream(dev) if stream is None else int(stream.cuda_stream)
    return _lib or lib(), dev, raw


def _dev_ptr(t: torch.Tensor, dtype, dev: int, name: str) -> int:
    """Address of a contiguous tensor of this dtype on the current device (the library launches
    there), or a refusal."""
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        _ptr(t, dtype, name)
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{dev}")
    return t.data_ptr()


def update_block_tables(prev_lens, seq_lens, qo_indptr, block_table, free_ring, ring_in, block_size,
                        num_rows, ring_out=None, slot_map=None, world_size=1, rank=0, interleave=1,
                        stream=None, lens_out=None):
    """mla_update_block_tables: blocks for the requests that grow from prev_lens to seq_lens
    tokens, blocks back from those that shrink, and the new tokens' cache rows.  All int32:
    prev_lens, seq_lens [B], qo_indptr [B + 1], block_table [B, width] (updated), free_ring
    [num_blocks] (updated), ring_in [2] = (head, count).  lens_out [B], if given, gets the lengths
    that the requests hold blocks for after the call (mla_update_block_tables_lens).  Returns
    (slot_map [num_rows], ring_out [2])."""
    L, dev, raw = _current(stream)
    if ring_out is None:
        ring_out = torch.empty_like(ring_in)
    if slot_map is None:
        slot_map = torch.empty(num_rows, dtype=torch.int32, device=seq_lens.device)
    B, width = block_table.shape
    if prev_lens.numel() != B or seq_lens.numel() != B or qo_indptr.numel() != B + 1 or \
            ring_in.numel() != 2 or ring_out.numel() != 2 or slot_map.numel() < num_rows or \
            (lens_out is not None and lens_out.numel() != B):
        raise ValueError("prev_lens, seq_lens, lens_out [B], qo_indptr [B + 1], block_table [B, width], ring_in "
                         "and ring_out [2], slot_map [num_rows]")
    i32 = torch.int32
    a = TableArgs(B, num_rows, _dev_ptr(prev_lens, i32, dev, "prev_lens"), _dev_ptr(seq_lens, i32, dev, "seq_lens"),
                  _dev_ptr(qo_indptr, i32, dev, "qo_indptr"), world_size, rank, interleave, block_size,
                  free_ring.numel(), _dev_ptr(block_table, i32, dev, "block_table"), width,
                  _dev_ptr(free_ring, i32, dev, "free_ring"), _dev_ptr(ring_in, i32, dev, "ring_in"),
                  _dev_ptr(ring_out, i32, dev, "ring_out"), _dev_ptr(slot_map, i32, dev, "slot_map"))
    if lens_out is None:
        st = L.mla_update_block_tables(ctypes.byref(a), raw)
    else:
        st = L.mla_update_block_tables_lens(ctypes.byref(a), _dev_ptr(lens_out, i32, dev, "lens_out"), raw)
    if st:
        _check(st, "mla_update_block_tables")
    return slot_map, ring_out


def _check_scaled(kv_cache, kv_scales, scale_block):
    shape = kv_cache.shape
    if kv_cache.dtype is not torch.uint8 or len(shape) != 2 or shape[1] != D_QK:
        raise ValueError("kv_cache must be [N, 576] uint8 (e4m3 codes)")
    if scale_block < 1 or kv_scales.numel() * scale_block != shape[0]:
        raise ValueError("kv_scales must hold one float32 per scale_block rows of kv_cache")
    return shape[0]


def write_kv_scaled(kv_new, slot_map, kv_cache, kv_scales, scale_block, stream=None):
    """mla_write_kv_scaled: kv_new [T, 576] bf16 quantised into kv_cache [N, 576] uint8 (e4m3
    codes) at the rows slot_map [T] int32 names (-1: skipped), with a power-of-two float32 scale
    per scale_block rows in kv_scales [N / scale_block].  Returns (kv_cache, kv_scales)."""
    L, dev, raw = _current(stream)
    rows = _check_scaled(kv_cache, kv_scales, scale_block)
    shape = kv_new.shape
    if len(shape) != 2 or shape[1] != D_QK or slot_map.numel() < shape[0]:
        raise ValueError("kv_new must be [T, 576] and slot_map hold T entries")
    st = L.mla_write_kv_scaled(shape[0], _dev_ptr(kv_new, torch.bfloat16, dev, "kv_new"),
                               _dev_ptr(slot_map, torch.int32, dev, "slot_map"),
                               _dev_ptr(kv_cache, torch.uint8, dev, "kv_cache"),
                               _dev_ptr(kv_scales, torch.float32, dev, "kv_scales"), scale_block, rows, raw)
    if st:
        _check(st, "mla_write_kv_scaled")
    return kv_cache, kv_scales


def decode_verify_scaled(q, kv_cache, kv_scales, scale_block, qo_indptr, row_len, subpage_table, page_size_,
                         num_segments, max_qlen, sm_scale, out=None, lse=None, workspace=None,
                         stream=None, num_views=1, wait_cycles=0):
    """mla_decode_verify_scaled: decode_verify over e4m3 codes kv_cache [N, 576] uint8 with one
    float32 scale per scale_block rows in kv_scales [N / scale_block].  The other arguments and
    the result (out, lse, workspace) are decode_verify's."""
    L, dev, raw = _current(stream)
    T, H, dk = q.shape
    rows = _check_scaled(kv_cache, kv_scales, scale_block)
    V = max(1, int(num_views))
    B, width = qo_indptr.numel() - 1, subpage_table.shape[-1]
    if dk != D_QK or row_len.numel() != V * T or subpage_table.numel() != V * B * width:
        raise ValueError("q must be [T, H, 576], row_len [V, T] and subpage_table [V, B, width]")
    if out is None:
        out = torch.empty((V, T, H, D_V) if V > 1 else (T, H, D_V), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((V, T, H) if V > 1 else (T, H), dtype=torch.float32, device=q.device)
    if out.numel() != V * T * H * D_V or lse.numel() != V * T * H:
        raise ValueError("out must be [V, T, H, 512] and lse [V, T, H]")
    i32 = torch.int32
    a = DecodeArgs(B, T, H, max_qlen, MLA_KV_FP8_E4M3, sm_scale, 1.0, _dev_ptr(q, torch.bfloat16, dev, "q"),
                   _dev_ptr(kv_cache, torch.uint8, dev, "kv_cache"), rows,
                   _dev_ptr(qo_indptr, i32, dev, "qo_indptr"), _dev_ptr(row_len, i32, dev, "row_len"),
                   _dev_ptr(subpage_table, i32, dev, "subpage_table"), width, page_size_, num_segments,
                   _dev_ptr(out, torch.bfloat16, dev, "out"), _dev_ptr(lse, torch.float32, dev, "lse"), 0, V,
                   wait_cycles)
    ref = ctypes.byref(a)
    need = L.mla_decode_verify_workspace(ref)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    st = L.mla_decode_verify_scaled(ref, _dev_ptr(kv_scales, torch.float32, dev, "kv_scales"), scale_block,
                                    _dev_ptr(workspace, torch.uint8, dev, "workspace"), need, raw)
    if st:
        _check(st, "mla_decode_verify_scaled")
    return out, lse, workspace


def _packer(cls):
    """pack(...) of a ctypes structure's fields in order, nested ones in line: bytes of its layout.  Making
    the structure itself takes longer than the launch (23 fields 0.9 us, with nested ones 3)."""
    code = {ctypes.c_int: "i", ctypes.c_float: "f", ctypes.c_int64: "q", ctypes.c_void_p: "P"}
    flat = lambda c: "".join(code[t] if t in code else flat(t) for _, t in c._fields_)   # noqa: E731
    st = struct.Struct("@" + flat(cls) + "0q")
    assert st.size == ctypes.sizeof(cls)
    return st.pack


_pack_rotary, _pack_grouped = _packer(RotaryArgs), _packer(GroupedArgs)
_NO_HEADS = (0, 0, 0, 0, 0, 0, 0, 0)


def _packed(name, *argtypes):
    """The library's function `name` taking its argument structure as packed bytes."""
    return ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_char_p, *argtypes)((name, lib()))


_calls = {}


def _call(name, *argtypes):
    f = _calls.get(name)
    if f is None:
        f = _calls[name] = _packed(name, *argtypes)
    return f


_TURN = 2 ** 192 * 10 ** 60 // (2 * 3141592653589793238462643383279502884197169399375105820974944)  # 2^192 / (2 pi)


def rotary_turns(freq, device="cuda") -> torch.Tensor:
    """The table mla_rotary takes for pairs of `freq` radians per position (float64 [R / 2], below
    2^32): the turns per position in units of 2^-64, modulo 1, rounded once, as int64 [R / 2] on
    `device`."""
    f = torch.as_tensor(freq, dtype=torch.float64)
    if f.dim() != 1:
        raise ValueError("freq must be [R / 2]")
    units = []
    for x in f.tolist():
        if not abs(x) < 2.0 ** 32:
            raise ValueError(f"freq must be finite radians per position below 2^32, got {x}")
        m, e = math.frexp(x)   # x = m * 2^e, in whole numbers (m * 2^53) * 2^(e - 53)
        shift = 128 + 53 - e
        units.append(((int(m * 2 ** 53) * _TURN + (1 << shift - 1) >> shift) + 2 ** 63) % 2 ** 64 - 2 ** 63)
    return torch.tensor(units, dtype=torch.int64, device=device)


def _refuse_view(t, dev, name):
    """The error for a tensor that is not bf16, on the current device, with contiguous heads."""
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{dev}")
    raise ValueError(f"{name}: the values of a head must be contiguous")


def _heads(x, out, rows, dev, name, out_rows=None):
    """mla_heads of x [rows, heads, dim] to out [out_rows, heads, dim] (out None: in place)."""
    shape, step = x.shape, x.stride()
    bf = torch.bfloat16
    if len(shape) != 3 or shape[0] != rows:
        raise ValueError(f"{name} must be [{rows}, heads, dim]")
    if x.dtype is not bf or x.get_device() != dev or step[2] != 1 and shape[2] != 1:
        _refuse_view(x, dev, name)
    n, heads, dim = shape
    if out is None:
        ptr = x.data_ptr()
        return heads, dim, ptr, step[0], step[1], ptr, step[0], step[1]
    to, at = out.shape, out.stride()
    if len(to) != 3 or to[1] != heads or to[2] != dim or to[0] != (n if out_rows is None else out_rows):
        raise ValueError(f"the output of {name} must be [{n if out_rows is None else out_rows}, {heads}, {dim}]")
    if out.dtype is not bf or out.get_device() != dev or at[2] != 1 and dim != 1:
        _refuse_view(out, dev, f"the output of {name}")
    return heads, dim, x.data_ptr(), step[0], step[1], out.data_ptr(), at[0], at[1]


def _angles(positions, turns, axes, neighbours, dev):
    """The arguments before q, k and v: rows, axes, R, pairing and the tables."""
    shape, step = positions.shape, positions.stride()
    T = shape[-1]
    if positions.dtype is not torch.int32 or positions.get_device() != dev or len(shape) > 2 or T > 1 and step[-1] != 1:
        raise ValueError(f"positions must be [T] or [axes, T] int32 on cuda:{dev}, an axis's contiguous")
    pairs = turns.shape[0]
    if axes is not None and axes.shape[0] != pairs:
        raise ValueError("axes must name one axis per entry of turns")
    two = len(shape) == 2
    return (T, shape[0] if two else 1, 2 * pairs, 1 if neighbours else 0, positions.data_ptr(), step[0] if two else 0,
            _dev_ptr(turns, torch.int64, dev, "turns"), 0 if axes is None else _dev_ptr(axes, torch.int32, dev, "axes"))


def rotary(q, k, positions, turns, axes=None, neighbours=False, q_out=None, k_out=None, stream=None):
    """mla_rotary: rotary positions on q [T, H, dim] and k [T, Hk, dim] bf16 (either may be None),
    whose first R = 2 * turns.numel() values of a head are rotated.  positions [T] or [axes, T]
    int32; turns from rotary_turns; axes [R / 2] int32: which axis turns a pair (None: the first).
    neighbours: pairs are (2i, 2i + 1) instead of (i, i + R / 2).  In place without q_out / k_out;
    any strides, the values of a head contiguous.  Returns (q_out, k_out)."""
    _, dev, raw = _current(stream)
    head = _angles(positions, turns, axes, neighbours, dev)
    a = _pack_rotary(*head, *(_NO_HEADS if q is None else _heads(q, q_out, head[0], dev, "q")),
                     *(_NO_HEADS if k is None else _heads(k, k_out, head[0], dev, "k")), *_NO_HEADS, 0, 0)
    st = _call("mla_rotary", ctypes.c_void_p)(a, raw)
    if st:
        _check(st, "mla_rotary")
    return q if q_out is None else q_out, k if k_out is None else k_out


def rotary_write(q, k, v, positions, turns, slot_map, k_cache, v_cache, axes=None, neighbours=False, q_out=None,
                 stream=None):
    """mla_rotary_write: rotary on q [T, H, dim] (may be None) and k [T, Hk, dim], and row r of k
    (rotated) and of v [T, Hv, dim_v] written to row slot_map[r] (int32, -1: nowhere) of k_cache
    [N, Hk, dim] and v_cache [N, Hv, dim_v].  The other arguments are rotary's.  Returns q_out."""
    _, dev, raw = _current(stream)
    head = _angles(positions, turns, axes, neighbours, dev)
    T, N = head[0], k_cache.shape[0]
    if slot_map.shape[0] < T:
        raise ValueError("slot_map must hold T entries")
    a = _pack_rotary(*head, *(_NO_HEADS if q is None else _heads(q, q_out, T, dev, "q")),
                     *_heads(k, k_cache, T, dev, "k", N), *_heads(v, v_cache, T, dev, "v", N),
                     _dev_ptr(slot_map, torch.int32, dev, "slot_map"), N)
    st = _call("mla_rotary_write", ctypes.c_void_p)(a, raw)
    if st:
        _check(st, "mla_rotary_write")
    return q if q_out is None else q_out


def decode_grouped_workspace_bytes(num_heads, num_kv_heads, max_qlen, head_dim, differential=False) -> int:
    """mla_decode_grouped_workspace."""
    a = GroupedArgs(num_heads=num_heads, num_kv_heads=num_kv_heads, max_qlen=max_qlen, head_dim=head_dim)
    return int(lib().mla_decode_grouped_workspace(ctypes.byref(a), int(differential)))


def _empty(shape, dtype, device, stream):
    """An output or workspace of the call's own: memory of the stream that the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _rows_of(t, heads, width, dev, name):
    """(address, row stride) of a bf16 tensor whose rows hold `heads` x `width` values without gaps."""
    step = t.stride()
    if t.dtype is not torch.bfloat16 or t.get_device() != dev or step[-1] != 1:
        _refuse_view(t, dev, name)
    if heads > 1 and step[1] != width or len(step) == 4 and 2 * step[2] != width:
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    return t.data_ptr(), step[0]


def _grouped(q, k_cache, v_cache, qo_indptr, row_len, subpage_table, page_size_, max_qlen, sm_scale, window, out, lse,
             wait_cycles, dev, maps, stream=None):
    """(packed arguments, out, lse, (H, Hkv, D)) of a grouped call of 1 or 2 maps."""
    qs, ks, vs = q.shape, k_cache.shape, v_cache.shape
    T, H, D = qs[0], qs[1], qs[-1]
    N, Hkv = ks[0], ks[1]
    width = maps * D
    if len(qs) != 2 + maps or len(ks) != 2 + maps or len(vs) != 3 or ks[-1] != D or vs[0] != N or vs[1] != Hkv or \
            vs[2] != width or maps == 2 and (qs[2] != 2 or ks[2] != 2):
        raise ValueError("q must be [T, H, D], k_cache and v_cache [N, Hkv, D]" if maps == 1 else
                         "q must be [T, H, 2, D], k_cache [N, Hkv, 2, D] and v_cache [N, Hkv, 2 D]")
    B, pages = qo_indptr.shape[0] - 1, subpage_table.shape[-1]
    if row_len.numel() != T or subpage_table.numel() != B * pages:
        raise ValueError("row_len must be [T] and subpage_table [B, width]")
    if out is None:
        out = _empty((T, H, width), torch.bfloat16, q.device, stream)
    if lse is None:
        lse = _empty((T, H) if maps == 1 else (T, H, 2), torch.float32, q.device, stream)
    if out.numel() != T * H * width or lse.numel() != T * H * maps:
        raise ValueError("out must hold a value vector and lse a number per row and head (and map)")
    i32 = torch.int32
    a = _pack_grouped(B, T, H, Hkv, max_qlen, D, window, sm_scale, *_rows_of(q, H, width, dev, "q"),
                      *_rows_of(k_cache, Hkv, width, dev, "k_cache"), *_rows_of(v_cache, Hkv, width, dev, "v_cache"), N,
                      _dev_ptr(qo_indptr, i32, dev, "qo_indptr"), _dev_ptr(row_len, i32, dev, "row_len"),
                      _dev_ptr(subpage_table, i32, dev, "subpage_table"), pages, page_size_,
                      _dev_ptr(out, torch.bfloat16, dev, "out"), _dev_ptr(lse, torch.float32, dev, "lse"), wait_cycles)
    return a, out, lse, (H, Hkv, D)


def decode_grouped(q, k_cache, v_cache, qo_indptr, row_len, subpage_table, page_size_, max_qlen, sm_scale, window=0,
                   out=None, lse=None, workspace=None, stream=None, wait_cycles=0):
    """mla_decode_grouped: q [T, H, D] bf16 over k_cache, v_cache [N, Hkv, D] bf16 (D 64, 128 or
    256), each of any row stride; qo_indptr, row_len, subpage_table, page_size_ as decode_verify's.
    window: a row sees its last `window` tokens only (0: all).  workspace: uint8, at least
    decode_grouped_workspace_bytes (None: allocated).  Returns (out [T, H, D] bf16, lse [T, H]
    f32, workspace)."""
    _, dev, raw = _current(stream)
    a, out, lse, sizes = _grouped(q, k_cache, v_cache, qo_indptr, row_len, subpage_table, page_size_, max_qlen, sm_scale,
                                  window, out, lse, wait_cycles, dev, 1, stream)
    if workspace is None:
        need = decode_grouped_workspace_bytes(sizes[0], sizes[1], max_qlen, sizes[2])
        workspace = _empty(need, torch.uint8, q.device, stream)
    st = _call("mla_decode_grouped", ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p)(
        a, _dev_ptr(workspace, torch.uint8, dev, "workspace"), workspace.numel(), raw)
    if st:
        _check(st, "mla_decode_grouped")
    return out, lse, workspace


def decode_differential(q, k_cache, v_cache, lam, qo_indptr, row_len, subpage_table, page_size_, max_qlen, sm_scale,
                        gain=None, eps=1e-5, window=0, out=None, lse=None, workspace=None, stream=None, wait_cycles=0):
    """mla_decode_differential: q [T, H, 2, D] over k_cache [N, Hkv, 2, D] and v_cache [N, Hkv, 2 D]
    bf16 (D 64 or 128): map 0 minus lam[h] (float32 [H]) times map 1, then, with gain (float32
    [2 D]), the norm over the head's 2 D values.  Returns (out [T, H, 2 D] bf16, lse [T, H, 2]
    f32, workspace)."""
    _, dev, raw = _current(stream)
    a, out, lse, sizes = _grouped(q, k_cache, v_cache, qo_indptr, row_len, subpage_table, page_size_, max_qlen, sm_scale,
                                  window, out, lse, wait_cycles, dev, 2, stream)
    if lam.numel() != sizes[0] or gain is not None and gain.numel() != 2 * sizes[2]:
        raise ValueError("lam must be [H] and gain [2 D]")
    if workspace is None:
        need = decode_grouped_workspace_bytes(sizes[0], sizes[1], max_qlen, sizes[2], True)
        workspace = _empty(need, torch.uint8, q.device, stream)
    f32, vp = torch.float32, ctypes.c_void_p
    st = _call("mla_decode_differential", vp, vp, ctypes.c_float, vp, ctypes.c_size_t, vp)(
        a, _dev_ptr(lam, f32, dev, "lam"), None if gain is None else _dev_ptr(gain, f32, dev, "gain"), eps,
        _dev_ptr(workspace, torch.uint8, dev, "workspace"), workspace.numel(), raw)
    if st:
        _check(st, "mla_decode_differential")
    return out, lse, workspace


def get_device_error(stream=None) -> int:
    """mla_get_device_error: synchronises, returns and clears the device error code."""
    code = ctypes.c_int32(0)
    st = lib().mla_get_device_error(ctypes.byref(code), _stream(stream))
    if st not in (MLA_OK, MLA_ERR_DEVICE_CHECK):
        _check(st, "mla_get_device_error")
    return int(code.value)
