"""prefill_dsa_indexer_gb300: the DSA sparse-attention layer on one GB300 GPU.

Python binding of libdsa (include/dsa.h).  Every function here only
marshals torch tensors into pointers and sizes and calls the C ABI of the
same name; all arithmetic runs in the library's CUDA kernels.  There is no
CPU fallback: importing the package on a machine without the built library
raises, and calling it with CPU tensors raises.

The layer (vLLM blog "Day-0 support for Kimi K3.1 Pro", section "Sparse
attention in K3.1 Pro"): indexer logits over every cached token -> exact
top-k (2,048) -> page-to-slot translation -> sparse absorbed MLA over the
selected tokens' latents.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct

import torch

from . import inputs  # noqa: F401  (seeded synthetic inputs)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdsa.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_WORKSPACE, ERR_TIMEOUT, ERR_BOUNDS, ERR_RANGE = \
    0, -1, -2, -3, -4, -5, -6, -7
KEY_FP8, KEY_MXFP4, LATENT_FP8, LATENT_NVFP4 = 1, 2, 3, 4
PAGE_SIZE = 64
INDEX_HEADS, INDEX_DIM, LATENT_DIM, VALUE_DIM = 32, 128, 576, 512
DEFAULT_SM_SCALE = 1.0 / math.sqrt(192.0)


class DsaError(RuntimeError):
    pass


class _Cache(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("format", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_pages", ctypes.c_int64), ("tensor_scale", ctypes.c_float)]


class _Rows(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("bt_stride", ctypes.c_int64), ("num_requests", ctypes.c_int32),
                ("row_req", ctypes.c_void_p), ("row_ctx", ctypes.c_void_p), ("num_rows", ctypes.c_int32),
                ("max_ctx", ctypes.c_int32), ("rows_per_group", ctypes.c_int32)]


class _KvCache(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("format", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_pages", ctypes.c_int64), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class _RopeSpec(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("rot_dim", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class _RopeAxes(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("axis_stride", ctypes.c_int64),
                ("axis", ctypes.c_void_p), ("num_axes", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class _RopeTensor(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("num_heads", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("x_token_stride", ctypes.c_int64), ("x_head_stride", ctypes.c_int64),
                ("out_token_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64)]


class _KvSegments(ctypes.Structure):
    _fields_ = [("first_row", ctypes.c_void_p), ("shared_ctx", ctypes.c_void_p), ("num_segments", ctypes.c_int32),
                ("least_saved", ctypes.c_int64)]


class _KvStep(ctypes.Structure):
    _fields_ = [("num_requests", ctypes.c_int32), ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int64),
                ("context", ctypes.c_void_p), ("new_tokens", ctypes.c_void_p), ("first_own", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("bt_stride", ctypes.c_int64), ("free_pages", ctypes.c_void_p),
                ("free_count", ctypes.c_void_p), ("free_capacity", ctypes.c_int32), ("num_segments", ctypes.c_int32),
                ("segment_requests", ctypes.c_void_p), ("max_rows", ctypes.c_int32),
                ("rows_per_group", ctypes.c_int32), ("row_req", ctypes.c_void_p), ("row_ctx", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("row_start", ctypes.c_void_p),
                ("granted", ctypes.c_void_p), ("context_out", ctypes.c_void_p), ("free_count_out", ctypes.c_void_p),
                ("segment_rows", ctypes.c_void_p)]


class _KvRows(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("rot_offset", ctypes.c_int32), ("layout", ctypes.c_int32)]


_lib = None


def load_library(path: str | None = None):
    """Load libdsa.so; raises if it has not been built (no fallback)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise DsaError(f"libdsa.so not found at {p}: build it with prefill_dsa_indexer_gb300.build.build()")
    lib = ctypes.CDLL(p)
    P, I32, I64, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    lib.dsa_version.restype = ctypes.c_int
    lib.dsa_status_string.restype = ctypes.c_char_p
    lib.dsa_status_string.argtypes = [ctypes.c_int]
    lib.dsa_indexer_logits.restype = ctypes.c_int
    lib.dsa_indexer_logits.argtypes = [ctypes.POINTER(_Cache), ctypes.POINTER(_Rows), P, P, P, I64, P, P]
    lib.dsa_topk.restype = ctypes.c_int
    lib.dsa_topk.argtypes = [P, I64, P, I32, I32, I32, P, P, P, ctypes.c_size_t, P]
    lib.dsa_topk_workspace_size.restype = ctypes.c_size_t
    lib.dsa_topk_workspace_size.argtypes = [I32, I32, I32]
    lib.dsa_page_to_slot.restype = ctypes.c_int
    lib.dsa_page_to_slot.argtypes = [ctypes.POINTER(_Rows), I64, P, I32, P, P, P]
    for name in ("dsa_sparse_mla_decode", "dsa_sparse_mla_prefill"):
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int
        fn.argtypes = [ctypes.POINTER(_Cache), P, I32, P, I32, I32, F, P, P, P, P, ctypes.c_size_t, P]
    lib.dsa_sparse_mla_decode_noalloc.restype = ctypes.c_int
    lib.dsa_sparse_mla_decode_noalloc.argtypes = [ctypes.POINTER(_Cache), P, I32, P, I32, I32, F, P, P, P, P]
    lib.dsa_cache_insert.restype = ctypes.c_int
    lib.dsa_cache_insert.argtypes = [ctypes.POINTER(_Cache), ctypes.POINTER(_Cache), P, I32, P, P, P, P]
    lib.dsa_sparse_mla_workspace_size.restype = ctypes.c_size_t
    lib.dsa_sparse_mla_workspace_size.argtypes = [I32, I32, I32]
    lib.dsa_indexer_logits_hist.restype = ctypes.c_int
    lib.dsa_indexer_logits_hist.argtypes = [ctypes.POINTER(_Cache), ctypes.POINTER(_Rows), P, P, P, I64, P, P, P]
    lib.dsa_topk_hist.restype = ctypes.c_int
    lib.dsa_topk_hist.argtypes = [P, I64, P, I32, I32, I32, P, P, P, P]
    lib.dsa_indexer_topk.restype = ctypes.c_int
    lib.dsa_indexer_topk.argtypes = [ctypes.POINTER(_Cache), ctypes.POINTER(_Rows), P, P, I32, P, P, P,
                                     ctypes.c_size_t, P]
    lib.dsa_indexer_topk_workspace_size.restype = ctypes.c_size_t
    lib.dsa_indexer_topk_workspace_size.argtypes = [I32, I32]
    lib.dsa_topk_slots.restype = ctypes.c_int
    lib.dsa_topk_slots.argtypes = [P, I64, ctypes.POINTER(_Rows), I64, I32, P, P, P, P, ctypes.c_size_t, P]
    lib.dsa_selftest_wait_timeout.restype = ctypes.c_int
    lib.dsa_selftest_wait_timeout.argtypes = [P, P]
    lib.dsa_topk_slots_warm.restype = ctypes.c_int
    lib.dsa_topk_slots_warm.argtypes = [P, I64, ctypes.POINTER(_Rows), ctypes.POINTER(_Cache), I32, P, P, P, P,
                                        ctypes.c_size_t, P]
    lib.dsa_sparse_mla_decode_prepare.restype = ctypes.c_int
    lib.dsa_sparse_mla_decode_prepare.argtypes = [ctypes.POINTER(_Cache), P, I32, I32, I32, P, P, ctypes.c_size_t, P]
    lib.dsa_sparse_mla_decode_prepared.restype = ctypes.c_int
    lib.dsa_sparse_mla_decode_prepared.argtypes = [ctypes.POINTER(_Cache), P, I32, P, I32, I32, F, P, P, P, P,
                                                   ctypes.c_size_t, P]
    lib.dsa_msa_block_scores.restype = ctypes.c_int
    lib.dsa_msa_block_scores.argtypes = [P, I64, ctypes.POINTER(_Rows), P, P, I64, P, P]
    lib.dsa_msa_select.restype = ctypes.c_int
    lib.dsa_msa_select.argtypes = [P, I64, P, I32, I32, P, P, P]
    lib.dsa_msa_attention.restype = ctypes.c_int
    lib.dsa_msa_attention.argtypes = [P, I64, F, F, ctypes.POINTER(_Rows), P, F, I32, P, F, P, P, P,
                                      ctypes.c_size_t, P, P]
    lib.dsa_msa_attention_workspace_size.restype = ctypes.c_size_t
    lib.dsa_msa_attention_workspace_size.argtypes = [I32, I32]
    D = ctypes.c_double
    lib.dsa_rope_frequencies.restype = ctypes.c_int
    lib.dsa_rope_frequencies.argtypes = [I32, D, I32, D, I32, P, P]
    lib.dsa_rope_turns.restype = ctypes.c_int
    lib.dsa_rope_turns.argtypes = [P, I32, P]
    lib.dsa_rope.restype = ctypes.c_int
    lib.dsa_rope.argtypes = [ctypes.POINTER(_RopeSpec), ctypes.POINTER(_RopeTensor), I32, I32, I32, P]
    lib.dsa_kv_insert.restype = ctypes.c_int
    lib.dsa_kv_insert.argtypes = [ctypes.POINTER(_KvCache), P, I32, ctypes.POINTER(_KvRows),
                                  ctypes.POINTER(_RopeSpec), ctypes.POINTER(_RopeTensor), P, P]
    lib.dsa_kv_plan.restype = ctypes.c_int
    lib.dsa_kv_plan.argtypes = [ctypes.POINTER(_KvStep), P, P]
    lib.dsa_rope_sections.restype = ctypes.c_int
    lib.dsa_rope_sections.argtypes = [P, I32, I32, I32, P]
    lib.dsa_rope_with_axes.restype = ctypes.c_int
    lib.dsa_rope_with_axes.argtypes = [ctypes.POINTER(_RopeAxes), ctypes.POINTER(_RopeTensor), I32, I32, I32, P]
    lib.dsa_kv_insert_with_axes.restype = ctypes.c_int
    lib.dsa_kv_insert_with_axes.argtypes = [ctypes.POINTER(_KvCache), P, I32, ctypes.POINTER(_KvRows),
                                            ctypes.POINTER(_RopeAxes), ctypes.POINTER(_RopeTensor), P, P]
    lib.dsa_kv_attention.restype = ctypes.c_int
    lib.dsa_kv_attention.argtypes = [ctypes.POINTER(_KvCache), ctypes.POINTER(_Rows), P, I64, I32, F, P, P, P,
                                     ctypes.c_size_t, P, P]
    lib.dsa_kv_attention_shared.restype = ctypes.c_int
    lib.dsa_kv_attention_shared.argtypes = [ctypes.POINTER(_KvCache), ctypes.POINTER(_Rows),
                                            ctypes.POINTER(_KvSegments), P, I64, I32, F, P, P, P, ctypes.c_size_t, P, P]
    lib.dsa_kv_attention_shared_workspace_size.restype = ctypes.c_size_t
    lib.dsa_kv_attention_shared_workspace_size.argtypes = [ctypes.POINTER(_KvCache), I32, I32, I32, I32]
    lib.dsa_kv_attention_workspace_size.restype = ctypes.c_size_t
    lib.dsa_kv_attention_workspace_size.argtypes = [ctypes.POINTER(_KvCache), I32, I32, I32]
    if path is None:
        _lib = lib
    return lib


EXPORTED = ("dsa_version", "dsa_status_string", "dsa_indexer_logits", "dsa_topk", "dsa_page_to_slot",
            "dsa_sparse_mla_decode", "dsa_sparse_mla_prefill", "dsa_sparse_mla_workspace_size",
            "dsa_sparse_mla_decode_noalloc", "dsa_cache_insert", "dsa_indexer_logits_hist", "dsa_topk_hist",
            "dsa_indexer_topk", "dsa_indexer_topk_workspace_size", "dsa_topk_slots", "dsa_topk_workspace_size",
            "dsa_sparse_mla_decode_prepare", "dsa_sparse_mla_decode_prepared", "dsa_msa_block_scores",
            "dsa_msa_select", "dsa_msa_attention", "dsa_msa_attention_workspace_size", "dsa_topk_slots_warm",
            "dsa_selftest_wait_timeout", "dsa_rope_frequencies", "dsa_rope_turns", "dsa_rope", "dsa_kv_insert",
            "dsa_kv_attention", "dsa_kv_attention_workspace_size", "dsa_rope_sections", "dsa_rope_with_axes",
            "dsa_kv_insert_with_axes", "dsa_kv_plan", "dsa_kv_attention_shared",
            "dsa_kv_attention_shared_workspace_size")
HIST_BINS = 65536
NOALLOC_MAX_ROWS = 8


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise DsaError("libdsa takes device tensors only")
    if not t.is_contiguous():
        raise DsaError("libdsa takes contiguous tensors only")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(rc: int, what: str):
    if rc != OK:
        msg = load_library().dsa_status_string(rc).decode()
        raise DsaError(f"{what}: {msg} ({rc})")


def new_status(device=None) -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=device or "cuda")


def check_status(status: torch.Tensor, what: str = "device status"):
    """Synchronise-free read of a device status word (the caller has synchronised)."""
    v = int(status.item())
    if v != OK:
        raise DsaError(f"{what}: {load_library().dsa_status_string(v).decode()} ({v})")


def _cache(pool: torch.Tensor, fmt: int, tensor_scale: float = 1.0) -> _Cache:
    return _Cache(_ptr(pool), fmt, PAGE_SIZE, pool.shape[0], tensor_scale)


def _rows(block_table, row_req, row_ctx, max_ctx, rows_per_group=1) -> _Rows:
    return _Rows(_ptr(block_table), block_table.shape[1], block_table.shape[0], _ptr(row_req), _ptr(row_ctx),
                 row_ctx.shape[0], int(max_ctx), int(rows_per_group))


def indexer_logits(index_pool, key_fmt, block_table, row_req, row_ctx, max_ctx, q_idx, head_w, rows_per_group=1,
                   logits=None, status=None, stream=None):
    """dsa_indexer_logits: fp32 logits [R, max_ctx] (t >= row_ctx[r] untouched)."""
    R = row_ctx.shape[0]
    if logits is None:
        logits = torch.empty((R, max(int(max_ctx), 1)), dtype=torch.float32, device=q_idx.device)
    c, r = _cache(index_pool, key_fmt), _rows(block_table, row_req, row_ctx, max_ctx, rows_per_group)
    rc = load_library().dsa_indexer_logits(ctypes.byref(c), ctypes.byref(r), _ptr(q_idx), _ptr(head_w),
                                           _ptr(logits), logits.stride(0), _ptr(status), _stream(stream))
    _check(rc, "dsa_indexer_logits")
    return logits


def topk_workspace_size(num_rows: int, max_ctx: int, k: int = 2048) -> int:
    """dsa_topk_workspace_size: bytes of the histogram top-k's workspace (0: the shape needs none)."""
    return int(load_library().dsa_topk_workspace_size(num_rows, max_ctx, k))


def _ws(workspace):
    return (_ptr(workspace), workspace.numel() * workspace.element_size()) if workspace is not None else (None, 0)


def topk(logits, row_ctx, max_ctx, k=2048, out=None, status=None, stream=None, workspace=None):
    """dsa_topk: int32 [R, k] selected positions, ascending, -1 padded (`workspace`: optional, see
    topk_workspace_size)."""
    R = row_ctx.shape[0]
    if out is None:
        out = torch.empty((R, k), dtype=torch.int32, device=logits.device)
    wp, wb = _ws(workspace)
    rc = load_library().dsa_topk(_ptr(logits), logits.stride(0), _ptr(row_ctx), R, int(max_ctx), int(k), _ptr(out),
                                 _ptr(status), wp, wb, _stream(stream))
    _check(rc, "dsa_topk")
    return out


def new_hist(num_rows: int, device=None) -> torch.Tensor:
    """A zeroed per-row histogram for indexer_logits_hist / topk_hist (uint32 bits in int32)."""
    return torch.zeros((num_rows, HIST_BINS), dtype=torch.int32, device=device or "cuda")


def indexer_logits_hist(index_pool, key_fmt, block_table, row_req, row_ctx, max_ctx, q_idx, head_w, hist,
                        rows_per_group=1, logits=None, status=None, stream=None):
    """dsa_indexer_logits_hist: indexer_logits that also adds every logit to the zeroed histogram `hist`."""
    R = row_ctx.shape[0]
    if logits is None:
        logits = torch.empty((R, max(int(max_ctx), 1)), dtype=torch.float32, device=q_idx.device)
    c, r = _cache(index_pool, key_fmt), _rows(block_table, row_req, row_ctx, max_ctx, rows_per_group)
    rc = load_library().dsa_indexer_logits_hist(ctypes.byref(c), ctypes.byref(r), _ptr(q_idx), _ptr(head_w),
                                                _ptr(logits), logits.stride(0), _ptr(hist), _ptr(status),
                                                _stream(stream))
    _check(rc, "dsa_indexer_logits_hist")
    return logits


def topk_hist(logits, row_ctx, max_ctx, hist, k=2048, out=None, status=None, stream=None):
    """dsa_topk_hist: topk starting from the scorer's histogram of these logits (left zeroed)."""
    R = row_ctx.shape[0]
    if out is None:
        out = torch.empty((R, k), dtype=torch.int32, device=logits.device)
    rc = load_library().dsa_topk_hist(_ptr(logits), logits.stride(0), _ptr(row_ctx), R, int(max_ctx), int(k),
                                      _ptr(hist), _ptr(out), _ptr(status), _stream(stream))
    _check(rc, "dsa_topk_hist")
    return out


def indexer_topk_workspace_size(num_rows: int, max_ctx: int) -> int:
    return int(load_library().dsa_indexer_topk_workspace_size(int(num_rows), int(max_ctx)))


def indexer_topk(index_pool, key_fmt, block_table, row_req, row_ctx, max_ctx, q_idx, head_w, workspace, k=2048,
                 rows_per_group=1, out=None, status=None, stream=None):
    """dsa_indexer_topk: scorer + top-k in one call; `workspace` (uint8, zeroed before its first use)."""
    R = row_ctx.shape[0]
    if out is None:
        out = torch.empty((R, k), dtype=torch.int32, device=q_idx.device)
    c, r = _cache(index_pool, key_fmt), _rows(block_table, row_req, row_ctx, max_ctx, rows_per_group)
    rc = load_library().dsa_indexer_topk(ctypes.byref(c), ctypes.byref(r), _ptr(q_idx), _ptr(head_w), int(k),
                                         _ptr(out), _ptr(status), _ptr(workspace), workspace.numel(),
                                         _stream(stream))
    _check(rc, "dsa_indexer_topk")
    return out


def topk_slots(logits, block_table, row_req, row_ctx, max_ctx, pool_pages, k=2048, out=None, slots=None,
               status=None, stream=None, workspace=None):
    """dsa_topk_slots: (idx int32 [R, k], slots int32 [R, k]) — top-k with the page -> slot translation."""
    R = row_ctx.shape[0]
    if out is None:
        out = torch.empty((R, k), dtype=torch.int32, device=logits.device)
    if slots is None:
        slots = torch.empty((R, k), dtype=torch.int32, device=logits.device)
    r = _rows(block_table, row_req, row_ctx, max_ctx)
    wp, wb = _ws(workspace)
    rc = load_library().dsa_topk_slots(_ptr(logits), logits.stride(0), ctypes.byref(r), int(pool_pages), int(k),
                                       _ptr(out), _ptr(slots), _ptr(status), wp, wb, _stream(stream))
    _check(rc, "dsa_topk_slots")
    return out, slots


def topk_slots_warm(logits, block_table, row_req, row_ctx, max_ctx, lat_pool, lat_fmt, k=2048, out=None,
                    slots=None, status=None, stream=None, workspace=None):
    """dsa_topk_slots_warm: topk_slots whose output pass also prefetches the selected FP8 latents into L2."""
    R = row_ctx.shape[0]
    if out is None:
        out = torch.empty((R, k), dtype=torch.int32, device=logits.device)
    if slots is None:
        slots = torch.empty((R, k), dtype=torch.int32, device=logits.device)
    r = _rows(block_table, row_req, row_ctx, max_ctx)
    c = _cache(lat_pool, lat_fmt)
    wp, wb = _ws(workspace)
    rc = load_library().dsa_topk_slots_warm(_ptr(logits), logits.stride(0), ctypes.byref(r), ctypes.byref(c), int(k),
                                            _ptr(out), _ptr(slots), _ptr(status), wp, wb, _stream(stream))
    _check(rc, "dsa_topk_slots_warm")
    return out, slots


def page_to_slot(block_table, row_req, row_ctx, max_ctx, pool_pages, idx, out=None, status=None, stream=None):
    """dsa_page_to_slot: int32 [R, k] physical slots (-1 stays -1)."""
    if out is None:
        out = torch.empty_like(idx)
    r = _rows(block_table, row_req, row_ctx, max_ctx)
    rc = load_library().dsa_page_to_slot(ctypes.byref(r), int(pool_pages), _ptr(idx), idx.shape[1], _ptr(out),
                                         _ptr(status), _stream(stream))
    _check(rc, "dsa_page_to_slot")
    return out


def cache_insert(idx_pool, key_fmt, lat_pool, lat_fmt, tensor_scale, slots, index_keys, latents, status=None,
                 stream=None):
    """dsa_cache_insert: quantise new tokens (bf16 [n,128] keys, [n,576] latents) into the pools in place."""
    ci, cl = _cache(idx_pool, key_fmt), _cache(lat_pool, lat_fmt, tensor_scale)
    rc = load_library().dsa_cache_insert(ctypes.byref(ci), ctypes.byref(cl), _ptr(slots), slots.shape[0],
                                         _ptr(index_keys), _ptr(latents), _ptr(status), _stream(stream))
    _check(rc, "dsa_cache_insert")


def sparse_mla_workspace_size(num_rows, num_heads, k) -> int:
    return int(load_library().dsa_sparse_mla_workspace_size(num_rows, num_heads, k))


def _mla(name, lat_pool, lat_fmt, tensor_scale, q, slots, sm_scale, out, lse, workspace, status, stream):
    R, H, _ = q.shape
    k = slots.shape[1]
    if out is None:
        out = torch.empty((R, H, VALUE_DIM), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((R, H), dtype=torch.float32, device=q.device)
    ws_ptr, ws_bytes = None, 0
    if name in ("dsa_sparse_mla_decode", "dsa_sparse_mla_decode_prepared"):
        need = sparse_mla_workspace_size(R, H, k)
        if workspace is None and need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        if workspace is not None:
            ws_ptr, ws_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
    c = _cache(lat_pool, lat_fmt, tensor_scale)
    rc = getattr(load_library(), name)(ctypes.byref(c), _ptr(q), H, _ptr(slots), R, k, float(sm_scale), _ptr(out),
                                       _ptr(lse), _ptr(status), ws_ptr, ws_bytes, _stream(stream))
    _check(rc, name)
    return out, lse


def sparse_mla_decode(lat_pool, lat_fmt, tensor_scale, q, slots, sm_scale=DEFAULT_SM_SCALE, out=None, lse=None,
                      workspace=None, status=None, stream=None):
    """dsa_sparse_mla_decode: (out fp32 [R, H, 512], lse fp32 [R, H]); q is bf16 (or its int16 bits)."""
    return _mla("dsa_sparse_mla_decode", lat_pool, lat_fmt, tensor_scale, q, slots, sm_scale, out, lse, workspace,
                status, stream)


def sparse_mla_decode_noalloc(lat_pool, lat_fmt, tensor_scale, q, slots, out, lse, sm_scale=DEFAULT_SM_SCALE,
                              status=None, stream=None):
    """dsa_sparse_mla_decode_noalloc: as sparse_mla_decode, with the split-K scratch kept in the
    library's own fixed device array instead of a workspace (for callers that cannot allocate;
    at most NOALLOC_MAX_ROWS rows).  `out` and `lse` must be preallocated."""
    R, H, _ = q.shape
    c = _cache(lat_pool, lat_fmt, tensor_scale)
    rc = load_library().dsa_sparse_mla_decode_noalloc(ctypes.byref(c), _ptr(q), H, _ptr(slots), R, slots.shape[1],
                                                      float(sm_scale), _ptr(out), _ptr(lse), _ptr(status),
                                                      _stream(stream))
    _check(rc, "dsa_sparse_mla_decode_noalloc")
    return out, lse


def sparse_mla_decode_prepare(lat_pool, lat_fmt, tensor_scale, q, k, workspace, status=None, stream=None):
    """dsa_sparse_mla_decode_prepare: the rows' queries into the workspace in the kernel's layout."""
    R, H, _ = q.shape
    c = _cache(lat_pool, lat_fmt, tensor_scale)
    rc = load_library().dsa_sparse_mla_decode_prepare(ctypes.byref(c), _ptr(q), H, R, int(k), _ptr(status),
                                                      _ptr(workspace), workspace.numel() * workspace.element_size(),
                                                      _stream(stream))
    _check(rc, "dsa_sparse_mla_decode_prepare")


def sparse_mla_decode_prepared(lat_pool, lat_fmt, tensor_scale, q, slots, sm_scale=DEFAULT_SM_SCALE, out=None,
                               lse=None, workspace=None, status=None, stream=None):
    """dsa_sparse_mla_decode_prepared: sparse_mla_decode after sparse_mla_decode_prepare on `workspace`."""
    return _mla("dsa_sparse_mla_decode_prepared", lat_pool, lat_fmt, tensor_scale, q, slots, sm_scale, out, lse,
                workspace, status, stream)


def sparse_mla_prefill(lat_pool, lat_fmt, tensor_scale, q, slots, sm_scale=DEFAULT_SM_SCALE, out=None, lse=None,
                       status=None, stream=None):
    return _mla("dsa_sparse_mla_prefill", lat_pool, lat_fmt, tensor_scale, q, slots, sm_scale, out, lse, None,
                status, stream)


def selftest_wait_timeout(status, stream=None):
    """dsa_selftest_wait_timeout: a kernel whose bounded wait runs out; status gets DSA_ERR_TIMEOUT."""
    _check(load_library().dsa_selftest_wait_timeout(_ptr(status), _stream(stream)), "dsa_selftest_wait_timeout")


# ------------------------------------------------------------------ MSA block-sparse variant
MSA_PAGE, MSA_GROUPS, MSA_BLOCKS = 128, 4, 16


def msa_block_scores(idx_pool, block_table, row_req, row_ctx, max_ctx, q_idx, rows_per_group=1, scores=None,
                     status=None, stream=None):
    """dsa_msa_block_scores: fp32 [R, 4, ceil(max_ctx / 128)] block-max index scores."""
    R = row_ctx.shape[0]
    nb = max((int(max_ctx) + MSA_PAGE - 1) // MSA_PAGE, 1)
    if scores is None:
        scores = torch.empty((R, MSA_GROUPS, nb), dtype=torch.float32, device=q_idx.device)
    r = _rows(block_table, row_req, row_ctx, max_ctx, rows_per_group)
    rc = load_library().dsa_msa_block_scores(_ptr(idx_pool), idx_pool.shape[0], ctypes.byref(r), _ptr(q_idx),
                                             _ptr(scores), scores.shape[-1], _ptr(status), _stream(stream))
    _check(rc, "dsa_msa_block_scores")
    return scores


def msa_select(scores, row_ctx, max_ctx, blocks=None, status=None, stream=None):
    """dsa_msa_select: int32 [R, 4, 16] selected blocks, ascending, -1 padded."""
    R = row_ctx.shape[0]
    if blocks is None:
        blocks = torch.empty((R, MSA_GROUPS, MSA_BLOCKS), dtype=torch.int32, device=scores.device)
    rc = load_library().dsa_msa_select(_ptr(scores), scores.shape[-1], _ptr(row_ctx), R, int(max_ctx), _ptr(blocks),
                                       _ptr(status), _stream(stream))
    _check(rc, "dsa_msa_select")
    return blocks


def msa_attention_workspace_size(num_rows, heads_per_group) -> int:
    return int(load_library().dsa_msa_attention_workspace_size(int(num_rows), int(heads_per_group)))


def msa_attention(kv_pool, k_scale, v_scale, block_table, row_req, row_ctx, max_ctx, q, q_scale, blocks, sm_scale,
                  out=None, lse=None, workspace=None, status=None, stream=None):
    """dsa_msa_attention: (out fp32 [R, H, 128], lse fp32 [R, H]); q is e4m3 codes [R, H, 128]."""
    R, H, _ = q.shape
    hpg = H // MSA_GROUPS
    if out is None:
        out = torch.empty((R, H, 128), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((R, H), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty(max(msa_attention_workspace_size(R, hpg), 1), dtype=torch.uint8, device=q.device)
    r = _rows(block_table, row_req, row_ctx, max_ctx)
    rc = load_library().dsa_msa_attention(_ptr(kv_pool), kv_pool.shape[0], float(k_scale), float(v_scale),
                                          ctypes.byref(r), _ptr(q), float(q_scale), hpg, _ptr(blocks),
                                          float(sm_scale), _ptr(out), _ptr(lse), _ptr(workspace),
                                          workspace.numel() * workspace.element_size(), _ptr(status),
                                          _stream(stream))
    _check(rc, "dsa_msa_attention")
    return out, lse


# ------------------------------------------------------------------ dense K/V path
KV_BF16, KV_FP8 = 5, 6
DTYPE_BF16, DTYPE_FP32 = 1, 2
ROPE_INTERLEAVED, ROPE_HALF = 0, 1
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
ROPE_AXES_ORDERS = {"split": 0, "cycle": 1}
ROPE_MAX_TENSORS = 4
KV_PLAN_MAX_REQUESTS = 16384


def _host_ptr(t):
    """Address of a contiguous host tensor."""
    if t.is_cuda or not t.is_contiguous():
        raise DsaError("a contiguous host tensor is needed here")
    return ctypes.c_void_p(t.data_ptr())


def _expect(t, what, device, dtypes, shape=None):
    """Raise unless t is a tensor on device `device` of one of `dtypes` and, where given, of `shape`."""
    d = t.get_device()
    if d != device:
        raise DsaError("libdsa takes device tensors only" if d < 0 else
                       f"{what} is on device {d}, the call's other tensors on device {device}")
    if t.dtype not in dtypes:
        raise DsaError(f"{what} has dtype {t.dtype}: expected {' or '.join(str(d) for d in dtypes)}")
    if shape is not None and t.shape != shape:
        raise DsaError(f"{what} has shape {tuple(t.shape)}: expected {tuple(shape)}")


def _flat(t, what, device, dtypes, shape=None):
    """_expect of a contiguous tensor; its address."""
    if t.get_device() != device or t.dtype not in dtypes or (shape is not None and t.shape != shape):
        _expect(t, what, device, dtypes, shape)
    if not t.is_contiguous():
        raise DsaError(f"{what} is not contiguous")
    return t.data_ptr()


def _launch(what, device, stream, *args):
    """The library's `what`(*args, stream) on device `device`, whichever is current."""
    fn = _packed.get(what) or _packed_function(what)
    if device == torch._C._cuda_getDevice():  # (a tensor of the call is on a device: CUDA is initialised)
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream)
    if rc != OK:
        _check(rc, what)


_int32, _float32, _bfloat16 = torch.int32, torch.float32, torch.bfloat16
_I32, _F32, _BF16 = (_int32,), (_float32,), (_bfloat16,)

# The calls of a decode step are short, so their arguments are packed into bytes (in the C structs' layouts) for
# function objects of their own that take those, which costs a fraction of ctypes structures.
_PACK_ROPE_SPEC = struct.Struct("PPif").pack
_PACK_ROPE_AXES = struct.Struct("PPqPiif").pack
_PACK_ROPE_TENSORS = [None] + [struct.Struct("PPiiqqqq" * n).pack for n in range(1, 5)]
_PACK_KV_ROWS = struct.Struct("PPqqii").pack
_PACK_SEGMENTS = struct.Struct("PPiq").pack
_PACK_STEP = struct.Struct("iiqPPPPqPPiiPiiPPPPPPPPP").pack
_PACK_ROWS = struct.Struct("PqiPPiii0q").pack
_packed = {}


def _packed_function(name):
    """The library's `name` taking packed structs."""
    fn = _packed.get(name)
    if fn is None:
        P, I32, I64, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
        fn = load_library()[name]
        fn.restype = ctypes.c_int
        rope, insert = [P, P, I32, I32, I32, P], [P, P, I32, P, P, P, P, P]
        fn.argtypes = {"dsa_rope": rope, "dsa_rope_with_axes": rope, "dsa_kv_insert": insert,
                       "dsa_kv_insert_with_axes": insert, "dsa_kv_plan": [P, P, P],
                       "dsa_kv_attention": [P, P, P, I64, I32, F, P, P, P, ctypes.c_size_t, P, P],
                       "dsa_kv_attention_shared": [P, P, P, P, I64, I32, F, P, P, P, ctypes.c_size_t, P, P]}[name]
        _packed[name] = fn
    return fn


def rope_frequencies(rot_dim, theta, scaling="none", factor=1.0, trained_ctx=0):
    """dsa_rope_frequencies: (radians per position of each pair, float64 host [rot_dim / 2]; scale)."""
    if scaling not in ROPE_SCALINGS:
        raise DsaError(f"unknown rotary scaling {scaling!r}: one of {', '.join(ROPE_SCALINGS)}")
    freq, scale = torch.empty(max(int(rot_dim) // 2, 1), dtype=torch.float64), ctypes.c_float()
    rc = load_library().dsa_rope_frequencies(int(rot_dim), float(theta), ROPE_SCALINGS[scaling], float(factor),
                                             int(trained_ctx), _host_ptr(freq), ctypes.byref(scale))
    _check(rc, "dsa_rope_frequencies")
    return freq, scale.value


def rope_turns(inv_freq):
    """dsa_rope_turns: float64 host [n] radians per position -> int64 host [n] (2^-64 turns, uint64 bits)."""
    if inv_freq.dtype != torch.float64:
        raise DsaError("rope_turns takes float64 frequencies")
    turns = torch.empty(inv_freq.shape, dtype=torch.int64)
    _check(load_library().dsa_rope_turns(_host_ptr(inv_freq), inv_freq.numel(), _host_ptr(turns)), "dsa_rope_turns")
    return turns


def rope_sections(sections, order="split"):
    """dsa_rope_sections: the axis of each pair, uint8 host [pairs], from how many pairs each axis has: one axis's
    after the other's ("split"), or the axes in turn while they have pairs left ("cycle")."""
    if order not in ROPE_AXES_ORDERS:
        raise DsaError(f"unknown order of axes {order!r}: one of {', '.join(ROPE_AXES_ORDERS)}")
    counts = torch.tensor([int(n) for n in sections], dtype=torch.int32)
    pairs = int(counts.sum())
    axis = torch.empty(max(pairs, 1), dtype=torch.uint8)
    rc = load_library().dsa_rope_sections(_host_ptr(counts), counts.numel(), ROPE_AXES_ORDERS[order], pairs,
                                          _host_ptr(axis))
    _check(rc, "dsa_rope_sections")
    return axis


class RopeTable:
    """The angles of `rope` and `kv_insert` on the device: `turns` int64 [rot_dim / 2], and `scale`.  With `axis`
    (uint8 host [rot_dim / 2], rope_sections) a token has a position on each of num_axes axes, and pair i turns by
    the one on axis[i]."""

    def __init__(self, turns, scale=1.0, axis=None, num_axes=None):
        if turns.dtype != torch.int64 or not turns.is_cuda or not turns.is_contiguous() or turns.dim() != 1:
            raise DsaError("RopeTable takes a contiguous int64 device vector (rope_turns)")
        self.turns, self.scale, self.rot_dim = turns, float(scale), 2 * turns.shape[0]
        self.device, self.address = turns.get_device(), turns.data_ptr()
        self.num_axes, self.axis = 0, None  # 0: one position a token
        if axis is not None:
            if axis.dtype != torch.uint8 or axis.shape != turns.shape or axis.is_cuda or not axis.is_contiguous():
                raise DsaError(f"the pairs' axes are a contiguous uint8 host vector of {turns.shape[0]}")
            self.axis = axis.clone()
            self.axis_address = self.axis.data_ptr()
            self.num_axes = int(axis.max()) + 1 if num_axes is None else int(num_axes)
            if self.num_axes < 1:
                raise DsaError(f"positions of {self.num_axes} axes: 1 at least")


def rope_table(rot_dim, theta=10000.0, scaling="none", factor=1.0, trained_ctx=0, device="cuda", sections=None,
               order="split", restart=False):
    """The table of dsa_rope_frequencies' angles (for other angles: RopeTable(rope_turns(f).to(device), scale)).
    `sections`, as many pairs for each axis of positions, in `order` (rope_sections); with `restart` each axis's
    pairs have the frequencies of a rotary part of their own instead of their places' in the whole."""
    freq, scale = rope_frequencies(rot_dim, theta, scaling, factor, trained_ctx)
    if sections is None:
        return RopeTable(rope_turns(freq).to(device), scale)
    axis = rope_sections(sections, order)
    if 2 * axis.numel() != rot_dim:
        raise DsaError(f"the sections make up {axis.numel()} pairs: expected {rot_dim // 2}")
    if restart:
        for a, n in enumerate(sections):
            if n > 0:
                freq[axis == a] = rope_frequencies(2 * n, theta, scaling, factor, trained_ctx)[0]
    return RopeTable(rope_turns(freq).to(device), scale, axis, len(sections))


def _rope_spec(table, positions, device, num_tokens):
    if table.device != device:
        raise DsaError(f"the rotary table is on device {table.device}, the call's other tensors on device {device}")
    axes = table.num_axes
    shape = (axes, num_tokens) if axes else (num_tokens,)
    if positions.dtype is not _int32 or positions.shape != shape or positions.get_device() != device:
        _expect(positions, "positions", device, _I32, shape)
    if axes:
        stride, one = positions.stride()
        if (one != 1 and num_tokens > 1) or stride < 0:
            raise DsaError("the positions on an axis are contiguous")
        return _PACK_ROPE_AXES(table.address, positions.data_ptr(), stride, table.axis_address, axes, table.rot_dim,
                               table.scale)
    if not positions.is_contiguous():
        raise DsaError("positions is not contiguous")
    return _PACK_ROPE_SPEC(table.address, positions.data_ptr(), table.rot_dim, table.scale)


def _rope_tensor(x, out, layout, rot_dim, device, dtype, num_tokens):
    """The fields of a dsa_rope_tensor."""
    shape = x.shape
    if x.dtype is not dtype or len(shape) != 3 or shape[2] != rot_dim or shape[0] != num_tokens or \
            x.get_device() != device:
        if len(shape) != 3 or shape[2] != rot_dim or shape[0] != num_tokens:
            raise DsaError(
                f"rotated tensors are [{num_tokens}, heads, {rot_dim}] (a slice of larger heads): got {tuple(shape)}")
        _expect(x, "x", device, (dtype,))
    a, b, c = x.stride()
    p = x.data_ptr()
    if out is x:
        if c != 1:
            raise DsaError("the rotary dims of a head are contiguous")
        return p, p, shape[1], layout, a, b, a, b
    if out.dtype is not dtype or out.shape != shape or out.get_device() != device:
        _expect(out, "out", device, (dtype,), shape)
    d, e, f = out.stride()
    if c != 1 or f != 1:
        raise DsaError("the rotary dims of a head are contiguous")
    return p, out.data_ptr(), shape[1], layout, a, b, d, e


def rope(x, table, positions, layout=ROPE_INTERLEAVED, out=None, stream=None):
    """dsa_rope: rotate x [tokens, heads, rot_dim] (bf16 or fp32; usually a slice x[..., a:a + rot_dim]) by
    its tokens' positions [tokens] (int32; a table with axes: [axes, tokens], dsa_rope_with_axes), into `out`
    (default: in place).  x, layout and out may be lists of up to 4
    tensors of the same tokens, rotated by one launch.  Tokens at negative positions are left alone."""
    if type(x) is list or type(x) is tuple:
        many, count, first = True, len(x), x[0] if x else None
        layouts = layout if type(layout) is list or type(layout) is tuple else [layout] * count
        outs = x if out is None else out
        if not 1 <= count <= ROPE_MAX_TENSORS or len(outs) != count or len(layouts) != count:
            raise DsaError(f"rope takes 1 to {ROPE_MAX_TENSORS} tensors, and as many layouts and outputs")
    else:
        many, count, first = False, 1, x
        if isinstance(layout, (list, tuple)):
            raise DsaError("one tensor has one layout")
    n, device, dtype, rot = first.shape[0], first.get_device(), first.dtype, table.rot_dim
    if device < 0:
        raise DsaError("libdsa takes device tensors only")
    if dtype is not _bfloat16 and dtype is not _float32:
        raise DsaError(f"rope takes bf16 or fp32 tensors: got {dtype}")
    if many:
        fields = []
        for i in range(count):
            fields += _rope_tensor(x[i], outs[i], layouts[i], rot, device, dtype, n)
    else:
        outs = x if out is None else out
        fields = _rope_tensor(x, outs, layout, rot, device, dtype, n)
    _launch("dsa_rope_with_axes" if table.num_axes else "dsa_rope", device, stream,
            _rope_spec(table, positions, device, n), _PACK_ROPE_TENSORS[count](*fields), count,
            DTYPE_BF16 if dtype is _bfloat16 else DTYPE_FP32, n)
    return outs


rope_with_axes = rope  # (which of the two C calls is made goes by the table)


class KvCache:
    """A paged K/V pool [pages, kv_heads, 2 (K, V), page_size, head_dim]: bf16, or e4m3 codes (uint8 or
    float8_e4m3fn) with their scales.  An MSA pool is one: KvCache(kv_pool.view(-1, 4, 2, 128, 128), ks, vs)."""

    def __init__(self, pool, k_scale=1.0, v_scale=1.0):
        if pool.dim() != 5 or pool.shape[2] != 2:
            raise DsaError(f"a K/V pool is [pages, kv_heads, 2, page_size, head_dim]: got {tuple(pool.shape)}")
        if pool.dtype not in (torch.bfloat16, torch.uint8, torch.float8_e4m3fn):
            raise DsaError(f"a K/V pool is bf16 or e4m3 codes: got {pool.dtype}")
        self.pool, self.k_scale, self.v_scale = pool, float(k_scale), float(v_scale)
        self.format = KV_BF16 if pool.dtype == torch.bfloat16 else KV_FP8
        self.num_pages, self.kv_heads, _, self.page_size, self.head_dim = pool.shape
        self._c = _KvCache(_ptr(pool), self.format, self.page_size, self.num_pages, self.kv_heads, self.head_dim,
                           self.k_scale, self.v_scale)
        self.device, self._packed = pool.get_device(), bytes(self._c)


def kv_insert(kv, slots, k, v, rope=None, positions=None, layout=ROPE_HALF, rot_offset=0, q=None, q_out=None,
              status=None, stream=None):
    """dsa_kv_insert: write k, v [tokens, kv_heads, head_dim] bf16 (parts of packed rows) at their slots of
    the KvCache.  With `rope` (a RopeTable) and `positions` (as `rope` takes them), K's dims [rot_offset,
    rot_offset + rot_dim) are rotated first, and q [tokens, heads, rot_dim] too, into q_out (default: in place).
    Returns q_out."""
    if slots.dim() != 1:
        raise DsaError(f"slots is [tokens]: got {tuple(slots.shape)}")
    n, device, heads, dim = slots.shape[0], kv.device, kv.kv_heads, kv.head_dim
    shape, width = (n, heads, dim), heads * dim
    if k.dtype is not _bfloat16 or k.shape != shape or k.get_device() != device:
        _expect(k, "k", device, _BF16, shape)
    if v.dtype is not _bfloat16 or v.shape != shape or v.get_device() != device:
        _expect(v, "v", device, _BF16, shape)
    if slots.dtype is not _int32 or slots.get_device() != device:
        _expect(slots, "slots", device, _I32)
    if not slots.is_contiguous():
        raise DsaError("slots is not contiguous")
    k_stride, b, c = k.stride()
    v_stride, d, e = v.stride()
    if c != 1 or e != 1 or (heads > 1 and (b != dim or d != dim)):
        raise DsaError(f"the heads of a token of {'k' if c != 1 or (heads > 1 and b != dim) else 'v'} are packed")
    if n == 1:
        k_stride, v_stride = max(k_stride, width), max(v_stride, width)
    spec = qt = None
    if rope is not None:
        if positions is None:
            raise DsaError("rope needs positions")
        spec = _rope_spec(rope, positions, device, n)
        if q is not None:
            q_out = q if q_out is None else q_out
            qt = _PACK_ROPE_TENSORS[1](*_rope_tensor(q, q_out, layout, rope.rot_dim, device, _bfloat16, n))
    elif q is not None:
        raise DsaError("q is rotated only: it needs rope")
    _launch("dsa_kv_insert_with_axes" if rope is not None and rope.num_axes else "dsa_kv_insert", device, stream,
            kv._packed, slots.data_ptr(), n,
            _PACK_KV_ROWS(k.data_ptr(), v.data_ptr(), k_stride, v_stride, rot_offset, layout), spec, qt,
            None if status is None else _flat(status, "status", device, _I32))
    return q_out


kv_insert_with_axes = kv_insert  # (as rope_with_axes)


def kv_plan(context, new_tokens, block_table, free_pages, free_count, page_size, num_pages, row_req, row_ctx,
            positions=None, slots=None, first_own=None, segment_requests=None, segment_rows=None, row_start=None,
            granted=None, context_out=None, free_count_out=None, rows_per_group=1, status=None, stream=None):
    """dsa_kv_plan: the rows (row_req, row_ctx, positions, slots), new pages and lengths of a step in which request i
    gets new_tokens[i] tokens (-1: it has ended).  All tensors are int32; block_table, free_pages and the tensors
    from row_req on are written (not first_own and segment_requests)."""
    device = context.get_device()
    if device < 0:
        raise DsaError("libdsa takes device tensors only")
    if block_table.dim() != 2:
        raise DsaError("the block table is [requests, pages]")
    n, width = block_table.shape
    rows, segments = row_req.shape[0], 0
    if (segment_requests is None) != (segment_rows is None):
        raise DsaError("segment_requests and segment_rows come together")
    if segment_requests is not None:
        segments = max(segment_requests.numel() - 1, 0)

    def at(t, what, shape):
        return 0 if t is None else _flat(t, what, device, _I32, shape)
    of = (n,)
    step = _PACK_STEP(
        n, int(page_size), int(num_pages), _flat(context, "context", device, _I32, of),
        _flat(new_tokens, "new_tokens", device, _I32, of), at(first_own, "first_own", of),
        _flat(block_table, "block_table", device, _I32), width,
        _flat(free_pages, "free_pages", device, _I32, (free_pages.numel(),)),
        _flat(free_count, "free_count", device, _I32, (1,)), free_pages.numel(), segments,
        at(segment_requests, "segment_requests", (segments + 1,)), rows, int(rows_per_group),
        _flat(row_req, "row_req", device, _I32, (rows,)), _flat(row_ctx, "row_ctx", device, _I32, (rows,)),
        at(positions, "positions", (rows,)), at(slots, "slots", (rows,)), at(row_start, "row_start", (n + 1,)),
        at(granted, "granted", of), at(context_out, "context_out", of), at(free_count_out, "free_count_out", (1,)),
        at(segment_rows, "segment_rows", (segments + 1,)))
    _launch("dsa_kv_plan", device, stream, step, None if status is None else _flat(status, "status", device, _I32))


class KvPlan:
    """The rows of a batch's steps (kv_plan), in buffers allocated once, so that repeated calls and captured graphs
    allocate nothing: row_req, row_ctx, positions, slots [max_rows], row_start [num_requests + 1], granted and context
    [num_requests], free_count [1] and segment_rows [num_segments + 1] hold what the last `run` made."""

    _NAMES = ("row_req", "row_ctx", "positions", "slots", "row_start", "granted", "context", "free_count",
              "segment_rows")

    def __init__(self, num_requests, max_rows, page_size, num_pages, rows_per_group=1, num_segments=0, device="cuda"):
        n, rows, segments = int(num_requests), int(max_rows), int(num_segments)
        sizes = (rows, rows, rows, rows, n + 1, n, n, 1, segments + 1 if segments else 0)
        buffers = {name: torch.full((size,), -1 if name in ("positions", "slots") else 0, dtype=torch.int32,
                                    device=device) for name, size in zip(self._NAMES, sizes)}
        self.__dict__.update(buffers, status=new_status(device), _addresses=[t.data_ptr() for t in buffers.values()],
                             _sizes=(n, rows, segments, int(rows_per_group), int(page_size), int(num_pages)),
                             _device=buffers["row_req"].get_device())
        if self._device < 0:
            raise DsaError("libdsa takes device tensors only")

    def __setattr__(self, name, value):
        raise DsaError(f"a plan writes into its own buffers: {name} cannot be another")

    def run(self, context, new_tokens, block_table, free_pages, free_count, first_own=None, segment_requests=None,
            stream=None):
        """context and free_count may be the plan's own of the step before.  Returns self."""
        n, rows, segments, group, page_size, num_pages = self._sizes
        if (segment_requests is None) != (segments == 0):
            raise DsaError(f"the plan is of {segments} segments")
        d, of, table = self._device, (n,), block_table.shape
        if len(table) != 2 or table[0] != n:
            raise DsaError(f"the block table is [{n}, pages]: got {tuple(table)}")
        _launch("dsa_kv_plan", d, stream, _PACK_STEP(
            n, page_size, num_pages, _flat(context, "context", d, _I32, of), _flat(new_tokens, "new_tokens", d, _I32, of),
            0 if first_own is None else _flat(first_own, "first_own", d, _I32, of),
            _flat(block_table, "block_table", d, _I32), table[1], _flat(free_pages, "free_pages", d, _I32),
            _flat(free_count, "free_count", d, _I32, (1,)), free_pages.numel(), segments,
            0 if segments == 0 else _flat(segment_requests, "segment_requests", d, _I32, (segments + 1,)), rows, group,
            *self._addresses), self.status.data_ptr())
        return self


def kv_attention_workspace_size(kv, num_rows, num_heads, max_ctx) -> int:
    return int(load_library().dsa_kv_attention_workspace_size(kv._c, int(num_rows), int(num_heads), int(max_ctx)))


def kv_attention_shared_workspace_size(kv, num_rows, num_heads, max_ctx, num_segments) -> int:
    return int(load_library().dsa_kv_attention_shared_workspace_size(kv._c, int(num_rows), int(num_heads), int(max_ctx),
                                                                     int(num_segments)))


def _attention_buffers(kv, R, H, max_ctx, segments, device, out, lse, workspace):
    """The attention calls' outputs and workspace, allocated where they are None."""
    if out is None:
        out = torch.empty((R, H, kv.head_dim), dtype=torch.bfloat16, device=device)
    if lse is None:
        lse = torch.empty((R, H), dtype=torch.float32, device=device)
    if workspace is None:
        need = kv_attention_shared_workspace_size(kv, R, H, max_ctx, segments) if segments else \
            kv_attention_workspace_size(kv, R, H, max_ctx)
        workspace = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    return out, lse, workspace


def _attention(name, segments, packed, kv, block_table, row_req, row_ctx, max_ctx, q, sm_scale, rows_per_group, out,
               lse, workspace, status, stream):
    """The library's `name`; packed: what it takes of its segments."""
    R, H, D = q.shape
    device = kv.device
    if D != kv.head_dim or q.dtype is not _bfloat16 or q.get_device() != device:
        _expect(q, "q", device, _BF16, (R, H, kv.head_dim))
    a, b, c = q.stride()
    if c != 1 or (b != D and H > 1):
        raise DsaError("the heads of a row of q are packed")
    requests = block_table.shape
    if len(requests) != 2:
        raise DsaError("the block table is [requests, pages]")
    if out is None or lse is None or workspace is None:
        if stream is None:
            out, lse, workspace = _attention_buffers(kv, R, H, max_ctx, segments, q.device, out, lse, workspace)
        else:
            with torch.cuda.stream(stream):  # what is allocated here belongs to the stream that uses it
                out, lse, workspace = _attention_buffers(kv, R, H, max_ctx, segments, q.device, out, lse, workspace)
    rows = _PACK_ROWS(_flat(block_table, "block_table", device, _I32), requests[1], requests[0],
                      _flat(row_req, "row_req", device, _I32, (R,)), _flat(row_ctx, "row_ctx", device, _I32, (R,)), R,
                      int(max_ctx), int(rows_per_group))
    wp, wb = (None, 0) if workspace is None else (_flat(workspace, "workspace", device, (workspace.dtype,)),
                                                  workspace.nbytes)
    _launch(name, device, stream, kv._packed, rows, *packed, q.data_ptr(), a if R > 1 else H * D, H,
            D ** -0.5 if sm_scale is None else float(sm_scale), _flat(out, "out", device, _BF16, (R, H, D)),
            _flat(lse, "lse", device, _F32, (R, H)), wp, wb,
            None if status is None else _flat(status, "status", device, _I32))
    return out, lse


def kv_attention(kv, block_table, row_req, row_ctx, max_ctx, q, sm_scale=None, rows_per_group=1, out=None, lse=None,
                 workspace=None, status=None, stream=None):
    """dsa_kv_attention: (out bf16 [R, H, head_dim], lse fp32 [R, H]) of q bf16 [R, H, head_dim] (heads packed)
    over the KvCache's tokens below row_ctx; sm_scale defaults to 1 / sqrt(head_dim).  A captured graph does not
    keep the workspace alive: pass one that outlives it, and no other call that may run beside it uses."""
    return _attention("dsa_kv_attention", 0, (), kv, block_table, row_req, row_ctx, max_ctx, q, sm_scale,
                      rows_per_group, out, lse, workspace, status, stream)


def kv_attention_shared(kv, block_table, row_req, row_ctx, max_ctx, q, segment_rows, segment_ctx, sm_scale=None,
                        rows_per_group=1, out=None, lse=None, workspace=None, status=None, stream=None, least_saved=0):
    """dsa_kv_attention_shared: kv_attention of rows of which segment_rows[s] .. segment_rows[s + 1] - 1 (int32
    [segments + 1]) have their first segment_ctx[s] tokens (int32 [segments]) in common, read once for all of them
    where that saves `least_saved` bytes (0: the library's choice, 1: always)."""
    device, segments = kv.device, segment_ctx.shape[0]
    packed = _PACK_SEGMENTS(_flat(segment_rows, "segment_rows", device, _I32, (segments + 1,)),
                            _flat(segment_ctx, "segment_ctx", device, _I32, (segments,)), segments,
                            int(least_saved))
    return _attention("dsa_kv_attention_shared", segments, (packed,), kv, block_table, row_req, row_ctx, max_ctx, q,
                      sm_scale, rows_per_group, out, lse, workspace, status, stream)


class KvLayer:
    """One full-attention layer's step over a resident K/V pool: rotate q and k, insert k and v, attend.

    Buffers are allocated once per shape and reused, so repeated calls (and CUDA-graph capture of `run`)
    allocate nothing.  Rows are the step's new tokens; a padding row has position -1, slot -1, context 0.
    """

    def __init__(self, kv, block_table, max_ctx, num_rows, num_heads, rope=None, layout=ROPE_HALF, rot_offset=0,
                 rows_per_group=1, sm_scale=None, num_segments=0, least_saved=0):
        self.kv, self.block_table, self.max_ctx = kv, block_table, int(max_ctx)
        self.rope, self.layout, self.rot_offset = rope, layout, int(rot_offset)
        self.rows_per_group, self.sm_scale, self.least_saved = rows_per_group, sm_scale, int(least_saved)
        R, H, device = int(num_rows), int(num_heads), kv.pool.device
        self.out = torch.empty((R, H, kv.head_dim), dtype=torch.bfloat16, device=device)
        self.lse = torch.empty((R, H), dtype=torch.float32, device=device)
        need = max(kv_attention_workspace_size(kv, R, H, self.max_ctx),
                   kv_attention_shared_workspace_size(kv, R, H, self.max_ctx, num_segments))
        self.workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=device)
        self.status = new_status(device)

    def run(self, row_req, row_ctx, slots, positions, q, k, v, stream=None, segment_rows=None, segment_ctx=None):
        """q [R, H, head_dim] is rotated in place; returns (out, lse).  With segment_rows and segment_ctx (of at most
        num_segments segments) the rows' common prefixes are read once (kv_attention_shared), where that saves the layer's
        least_saved bytes."""
        if (segment_rows is None) != (segment_ctx is None):
            raise DsaError("segment_rows and segment_ctx come together")
        if self.rope is None:
            kv_insert(self.kv, slots, k, v, status=self.status, stream=stream)
        else:
            part = q[..., self.rot_offset:self.rot_offset + self.rope.rot_dim]
            kv_insert(self.kv, slots, k, v, rope=self.rope, positions=positions, layout=self.layout,
                      rot_offset=self.rot_offset, q=part, status=self.status, stream=stream)
        if segment_rows is not None:
            return kv_attention_shared(self.kv, self.block_table, row_req, row_ctx, self.max_ctx, q, segment_rows,
                                       segment_ctx, self.sm_scale, self.rows_per_group, out=self.out, lse=self.lse,
                                       workspace=self.workspace, status=self.status, stream=stream,
                                       least_saved=self.least_saved)
        return kv_attention(self.kv, self.block_table, row_req, row_ctx, self.max_ctx, q, self.sm_scale,
                            self.rows_per_group, out=self.out, lse=self.lse, workspace=self.workspace,
                            status=self.status, stream=stream)


class Layer:
    """One DSA layer invocation over resident caches: indexer -> top-k -> slots -> sparse MLA.

    Buffers are allocated once per shape and reused, so repeated calls (and
    CUDA-graph capture of `run`) allocate nothing.
    """

    def __init__(self, idx_pool, key_fmt, lat_pool, lat_fmt, tensor_scale, block_table, max_ctx, num_rows,
                 num_heads=96, k=2048, rows_per_group=1, prefill=False, sm_scale=DEFAULT_SM_SCALE, device="cuda",
                 single_pass=False):
        self.idx_pool, self.key_fmt = idx_pool, key_fmt
        self.lat_pool, self.lat_fmt, self.tensor_scale = lat_pool, lat_fmt, float(tensor_scale)
        self.block_table, self.max_ctx, self.k = block_table, int(max_ctx), int(k)
        self.rows_per_group, self.prefill, self.sm_scale = rows_per_group, prefill, sm_scale
        R, H = int(num_rows), int(num_heads)
        self.logits = torch.empty((R, max(self.max_ctx, 1)), dtype=torch.float32, device=device)
        self.idx = torch.empty((R, self.k), dtype=torch.int32, device=device)
        self.slots = torch.empty((R, self.k), dtype=torch.int32, device=device)
        # outputs and log-sum-exps in one buffer, so one copy moves a step's results
        self.outputs = torch.empty(R * H * (VALUE_DIM + 1), dtype=torch.float32, device=device)
        self.out = self.outputs[:R * H * VALUE_DIM].view(R, H, VALUE_DIM)
        self.lse = self.outputs[R * H * VALUE_DIM:].view(R, H)
        need = 0 if prefill else sparse_mla_workspace_size(R, H, self.k)
        self.workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=device)
        # the histogram top-k's counts and candidates (few long rows; none otherwise)
        tk = topk_workspace_size(R, self.max_ctx, self.k)
        self.topk_workspace = torch.empty(tk, dtype=torch.uint8, device=device) if tk > 0 else None
        self.status = new_status(device)
        # single pass: the scorer builds each row's histogram and the top-k starts from it (opt-in:
        # on one GB300 the scorer's histogram atomics cost more than the selection saves)
        self.single_pass = single_pass
        self.hist = new_hist(R, device) if single_pass else None

    def score(self, row_req, row_ctx, q_idx, head_w, stream=None):
        """Indexer logits (and, single pass, their histogram)."""
        if self.single_pass:
            indexer_logits_hist(self.idx_pool, self.key_fmt, self.block_table, row_req, row_ctx, self.max_ctx, q_idx,
                                head_w, self.hist, self.rows_per_group, logits=self.logits, status=self.status,
                                stream=stream)
        else:
            indexer_logits(self.idx_pool, self.key_fmt, self.block_table, row_req, row_ctx, self.max_ctx, q_idx,
                           head_w, self.rows_per_group, logits=self.logits, status=self.status, stream=stream)

    def select(self, row_req, row_ctx, q_mla, stream=None, prepared=False):
        """Top-k, page -> slot and sparse MLA over the scored logits (`prepared`: prepare() ran already)."""
        self.select_tokens(row_req, row_ctx, stream=stream)
        return self.attend(q_mla, stream=stream, prepared=prepared)

    def select_tokens(self, row_req, row_ctx, stream=None):
        """Top-k and page -> slot over the scored logits (into self.idx, self.slots)."""
        if self.single_pass:
            topk_hist(self.logits, row_ctx, self.max_ctx, self.hist, self.k, out=self.idx, status=self.status,
                      stream=stream)
            page_to_slot(self.block_table, row_req, row_ctx, self.max_ctx, self.lat_pool.shape[0], self.idx,
                         out=self.slots, status=self.status, stream=stream)
        elif not self.prefill:  # decode: top-k with page -> slot, warming L2 with the chosen latents
            topk_slots_warm(self.logits, self.block_table, row_req, row_ctx, self.max_ctx, self.lat_pool,
                            self.lat_fmt, self.k, out=self.idx, slots=self.slots, status=self.status, stream=stream,
                            workspace=self.topk_workspace)
        else:  # top-k with the page -> slot translation in its output pass
            topk_slots(self.logits, self.block_table, row_req, row_ctx, self.max_ctx, self.lat_pool.shape[0], self.k,
                       out=self.idx, slots=self.slots, status=self.status, stream=stream,
                       workspace=self.topk_workspace)

    def attend(self, q_mla, stream=None, prepared=False):
        """Sparse MLA over self.slots (`prepared`: prepare() ran already for these queries)."""
        if self.prefill:
            sparse_mla_prefill(self.lat_pool, self.lat_fmt, self.tensor_scale, q_mla, self.slots, self.sm_scale,
                               out=self.out, lse=self.lse, status=self.status, stream=stream)
        elif prepared:
            sparse_mla_decode_prepared(self.lat_pool, self.lat_fmt, self.tensor_scale, q_mla, self.slots,
                                       self.sm_scale, out=self.out, lse=self.lse, workspace=self.workspace,
                                       status=self.status, stream=stream)
        else:
            sparse_mla_decode(self.lat_pool, self.lat_fmt, self.tensor_scale, q_mla, self.slots, self.sm_scale,
                              out=self.out, lse=self.lse, workspace=self.workspace, status=self.status,
                              stream=stream)
        return self.out, self.lse

    def prepare(self, q_mla, stream=None):
        """Decode query conversion (independent of the scorer and the top-k; may run beside the top-k,
        which leaves most SMs free, and must be ordered before attend(prepared=True))."""
        if not self.prefill:
            sparse_mla_decode_prepare(self.lat_pool, self.lat_fmt, self.tensor_scale, q_mla, self.k, self.workspace,
                                      status=self.status, stream=stream)

    def run(self, row_req, row_ctx, q_idx, head_w, q_mla, stream=None):
        self.score(row_req, row_ctx, q_idx, head_w, stream=stream)
        return self.select(row_req, row_ctx, q_mla, stream=stream)
