"""ctypes binding of libpaged_attn.so (the C ABI in include/paged_attn.h).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI.  There is no fallback; if the library is missing or
cannot be built, every call raises.  PyTorch provides device memory and
streams.

The functions named ``pa_*`` mirror the C entry points one to one.
``paged_attention`` is the pages' model-facing call ("Week 3 Day 5: Paged
FlashAttention", Keep the Day 4 Interface): it allocates the output and a
workspace with torch and calls ``pa_paged_attention_sched``.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading
from typing import NamedTuple

from . import build as _build

PA_OK = 0
PA_ERR_INVALID_ARG = 1
PA_ERR_UNSUPPORTED = 2
PA_ERR_BAD_BLOCK_TABLE = 3
PA_ERR_WORKSPACE = 4
PA_ERR_CUDA = 5
PA_ERR_DEVICE_FLAG = 6

PA_BF16 = 0
PA_F32 = 1

PA_SCHED_AUTO = 0
PA_SCHED_DECODE = 1
PA_SCHED_PREFILL = 2

PA_FLAG_BAD_PAGE = 0x1
PA_FLAG_BAD_CONTEXT = 0x2
PA_FLAG_TIMEOUT = 0x4
PA_FLAG_BAD_TREE = 0x8
PA_FLAG_NO_PAGES = 0x10

TREE_MAX = 1024  # drafted slots of a sequence at most

_lock = threading.Lock()
_lib = None


class PagedAttentionError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        super().__init__(f"{what}: status {status} ({status_str(status)})" if what else
                         f"status {status} ({status_str(status)})")
        self.status = status


class pa_shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H_q", ctypes.c_int), ("H_kv", ctypes.c_int),
                ("L", ctypes.c_int), ("D", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("max_pages_per_seq", ctypes.c_int),
                ("dtype", ctypes.c_int)]


class pa_q4_pool(ctypes.Structure):
    _fields_ = [("key_codes", ctypes.c_void_p), ("key_scales", ctypes.c_void_p),
                ("value_codes", ctypes.c_void_p), ("value_scales", ctypes.c_void_p)]


def library_path() -> str:
    return _build.LIB


def load(auto_build: bool = True):
    """Loads libpaged_attn.so (building it first if it is stale)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if auto_build and not _build.up_to_date():
            _build.build()
        path = _build.LIB
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with __graft_entry__.build()")
        lib = ctypes.CDLL(path)
        vp, i32p, sz = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t
        sp = ctypes.POINTER(pa_shape)
        lib.pa_workspace_bytes.argtypes = [sp]
        lib.pa_workspace_bytes.restype = sz
        common = [sp, vp, vp, vp, i32p, i32p, ctypes.c_float, ctypes.c_int, vp, vp, sz, vp]
        lib.pa_paged_attention.argtypes = common
        lib.pa_paged_attention.restype = ctypes.c_int
        lib.pa_paged_attention_sched.argtypes = common + [ctypes.c_int]
        lib.pa_paged_attention_sched.restype = ctypes.c_int
        lib.pa_paged_attention_profiled.argtypes = common + [ctypes.c_int, vp, vp]
        lib.pa_paged_attention_profiled.restype = ctypes.c_int
        lib.pa_paged_attention_decode_noalloc.argtypes = [sp, vp, vp, vp, i32p, i32p,
                                                          ctypes.c_float, ctypes.c_int, vp, vp,
                                                          vp]
        lib.pa_paged_attention_decode_noalloc.restype = ctypes.c_int
        lib.pa_gather_debug.argtypes = [sp, vp, vp, i32p, i32p, ctypes.c_int, vp, vp, vp, vp]
        lib.pa_gather_debug.restype = ctypes.c_int
        lib.pa_check_device_flag.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32), ctypes.c_int,
                                             vp]
        lib.pa_check_device_flag.restype = ctypes.c_int
        lib.pa_validate_metadata.argtypes = [sp, i32p, i32p, ctypes.c_int, vp]
        lib.pa_validate_metadata.restype = ctypes.c_int
        lib.pa_choose_schedule.argtypes = [sp]
        lib.pa_choose_schedule.restype = ctypes.c_int
        lib.pa_launch_count.argtypes = [sp, ctypes.c_int]
        lib.pa_launch_count.restype = ctypes.c_int
        lib.pa_paged_attention_masked.argtypes = [sp, vp, vp, vp, i32p, i32p, ctypes.c_float,
                                                  ctypes.c_int, vp, ctypes.c_longlong, vp, vp,
                                                  sz, vp, ctypes.c_int]
        lib.pa_paged_attention_masked.restype = ctypes.c_int
        lib.pa_paged_attention_varlen.argtypes = [sp, vp, vp, vp, i32p, i32p, i32p, ctypes.c_int,
                                                  ctypes.c_float, ctypes.c_int, vp, vp, sz, vp,
                                                  ctypes.c_int]
        lib.pa_paged_attention_varlen.restype = ctypes.c_int
        lib.pa_validate_metadata_varlen.argtypes = [sp, i32p, i32p, i32p, ctypes.c_int,
                                                    ctypes.c_int, vp]
        lib.pa_validate_metadata_varlen.restype = ctypes.c_int
        lib.pa_selftest_wait_timeout.argtypes = [vp, sz, ctypes.c_uint, vp]
        lib.pa_selftest_wait_timeout.restype = ctypes.c_int
        lib.pa_append_kv.argtypes = [sp, vp, vp, vp, vp, i32p, i32p, vp, sz, vp]
        lib.pa_append_kv.restype = ctypes.c_int
        qp, f32, ci, ll = (ctypes.POINTER(pa_q4_pool), ctypes.c_float, ctypes.c_int,
                           ctypes.c_longlong)
        lib.pa_append_kv_q4.argtypes = [sp, vp, vp, qp, i32p, i32p, vp, sz, vp]
        lib.pa_append_kv_q4.restype = ci
        lib.pa_gather_kv_q4.argtypes = [sp, qp, i32p, i32p, ci, ci, vp, vp, vp, sz, vp]
        lib.pa_gather_kv_q4.restype = ci
        lib.pa_paged_attention_q4.argtypes = [sp, vp, qp, i32p, i32p, f32, ci, vp, vp, ll, vp, vp,
                                              sz, vp]
        lib.pa_paged_attention_q4.restype = ci
        lib.pa_q4_workspace_bytes.argtypes = [sp, ci]
        lib.pa_q4_workspace_bytes.restype = sz
        lib.pa_paged_attention_weights.argtypes = [sp, vp, vp, vp, i32p, i32p, f32, ci, vp, vp, ll,
                                                   vp, vp, sz, vp]
        lib.pa_paged_attention_weights.restype = ci
        lib.pa_weights_workspace_bytes.argtypes = [sp]
        lib.pa_weights_workspace_bytes.restype = sz
        evict = [i32p, i32p, vp, ll, ci, ci, i32p, ci, i32p, vp, ll, i32p, vp, sz, vp]
        lib.pa_evict_kv.argtypes = [sp, vp, vp] + evict
        lib.pa_evict_kv.restype = ci
        lib.pa_evict_kv_q4.argtypes = [sp, qp] + evict
        lib.pa_evict_kv_q4.restype = ci
        end = [vp, sz, vp]  # workspace, its bytes, stream
        lib.pa_tree_mask.argtypes = [ci, ci, i32p, vp, i32p] + end
        lib.pa_tree_mask.restype = ci
        lib.pa_tree_workspace_bytes.argtypes = [sp]
        lib.pa_tree_workspace_bytes.restype = sz
        lib.pa_paged_attention_tree.argtypes = [sp, vp, vp, vp, i32p, i32p, vp, f32, vp] + end
        lib.pa_paged_attention_tree.restype = ci
        lib.pa_paged_attention_tree_q4.argtypes = [sp, vp, qp, i32p, i32p, vp, f32, vp] + end
        lib.pa_paged_attention_tree_q4.restype = ci
        lib.pa_compact_kv.argtypes = [sp, vp, vp, i32p, i32p, i32p, ci, i32p, i32p] + end
        lib.pa_compact_kv.restype = ci
        lib.pa_compact_kv_q4.argtypes = [sp, qp, i32p, i32p, i32p, ci, i32p, i32p] + end
        lib.pa_compact_kv_q4.restype = ci
        lib.pa_pages_workspace_bytes.argtypes = [sp]
        lib.pa_pages_workspace_bytes.restype = sz
        lib.pa_fork_pages.argtypes = [sp, i32p, i32p, i32p, i32p, i32p, i32p, ci] + end
        lib.pa_fork_pages.restype = ci
        lib.pa_resize_pages.argtypes = [sp, i32p, i32p, i32p, i32p, i32p] + end
        lib.pa_resize_pages.restype = ci
        lib.pa_copy_pages.argtypes = [sp, vp, vp, i32p, ci] + end
        lib.pa_copy_pages.restype = ci
        lib.pa_copy_pages_q4.argtypes = [sp, qp, i32p, ci] + end
        lib.pa_copy_pages_q4.restype = ci
        lib.pa_status_str.argtypes = [ctypes.c_int]
        lib.pa_status_str.restype = ctypes.c_char_p
        _lib = lib
        return lib


def status_str(status: int) -> str:
    try:
        return load().pa_status_str(int(status)).decode()
    except Exception:  # pragma: no cover - library missing
        return "?"


def _ptr(x):
    """Device/host address of a torch tensor, or an int address, or None."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def make_shape(B, H_q, H_kv, L, D, num_pages, page_size, max_pages_per_seq, dtype=PA_BF16):
    return pa_shape(int(B), int(H_q), int(H_kv), int(L), int(D), int(num_pages),
                    int(page_size), int(max_pages_per_seq), int(dtype))


def shape_of(query, key_pages, block_table) -> pa_shape:
    """pa_shape of torch tensors laid out as in include/paged_attn.h."""
    import torch
    B, H_q, L, D = query.shape
    P, H_kv, ps, D2 = key_pages.shape
    if D2 != D:
        raise ValueError("query and pages disagree on head dim")
    if query.dtype != key_pages.dtype:
        raise ValueError("query and pages must share a dtype")
    dt = {torch.bfloat16: PA_BF16, torch.float32: PA_F32}.get(query.dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {query.dtype}")
    return make_shape(B, H_q, H_kv, L, D, P, ps, block_table.shape[1], dt)


# ---- one-to-one C entry points ---------------------------------------------
def pa_workspace_bytes(shape: pa_shape) -> int:
    return int(load().pa_workspace_bytes(ctypes.byref(shape)))


def pa_paged_attention(shape, query, key_pages, value_pages, block_table, context_lens, scale,
                       causal, out, workspace, workspace_bytes, stream=None) -> int:
    return load().pa_paged_attention(
        ctypes.byref(shape), _ptr(query), _ptr(key_pages), _ptr(value_pages), _ptr(block_table),
        _ptr(context_lens), float(scale), int(bool(causal)), _ptr(out), _ptr(workspace),
        int(workspace_bytes), _stream(stream))


def pa_paged_attention_sched(shape, query, key_pages, value_pages, block_table, context_lens,
                             scale, causal, out, workspace, workspace_bytes, stream=None,
                             schedule=PA_SCHED_AUTO) -> int:
    return load().pa_paged_attention_sched(
        ctypes.byref(shape), _ptr(query), _ptr(key_pages), _ptr(value_pages), _ptr(block_table),
        _ptr(context_lens), float(scale), int(bool(causal)), _ptr(out), _ptr(workspace),
        int(workspace_bytes), _stream(stream), int(schedule))


def pa_paged_attention_profiled(shape, query, key_pages, value_pages, block_table, context_lens,
                                scale, causal, out, workspace, workspace_bytes, stream=None,
                                schedule=PA_SCHED_AUTO, event_before=None,
                                event_after=None) -> int:
    """event_before / event_after: raw cudaEvent_t handles (int) or None."""
    return load().pa_paged_attention_profiled(
        ctypes.byref(shape), _ptr(query), _ptr(key_pages), _ptr(value_pages), _ptr(block_table),
        _ptr(context_lens), float(scale), int(bool(causal)), _ptr(out), _ptr(workspace),
        int(workspace_bytes), _stream(stream), int(schedule), event_before, event_after)


def pa_paged_attention_decode_noalloc(shape, query, key_pages, value_pages, block_table,
                                      context_lens, scale, causal, out, device_flag_out=None,
                                      stream=None) -> int:
    """Decode schedule with the library's fixed scratch array instead of a
    caller workspace (for callers that cannot allocate device memory).
    device_flag_out: optional device tensor of one 32-bit word that receives
    this call's PA_FLAG_* bits."""
    return load().pa_paged_attention_decode_noalloc(
        ctypes.byref(shape), _ptr(query), _ptr(key_pages), _ptr(value_pages), _ptr(block_table),
        _ptr(context_lens), float(scale), int(bool(causal)), _ptr(out), _ptr(device_flag_out),
        _stream(stream))


def pa_gather_debug(shape, key_pages, value_pages, block_table, context_lens, max_S, k_dense,
                    v_dense, workspace, stream=None) -> int:
    return load().pa_gather_debug(
        ctypes.byref(shape), _ptr(key_pages), _ptr(value_pages), _ptr(block_table),
        _ptr(context_lens), int(max_S), _ptr(k_dense), _ptr(v_dense), _ptr(workspace),
        _stream(stream))


def pa_paged_attention_masked(shape, query, key_pages, value_pages, block_table, context_lens,
                              scale, causal, mask, mask_S, out, workspace, workspace_bytes,
                              stream=None, schedule=PA_SCHED_AUTO) -> int:
    """mask: fp32 device tensor [B * H_q, L, mask_S] added to the scaled scores."""
    return load().pa_paged_attention_masked(
        ctypes.byref(shape), _ptr(query), _ptr(key_pages), _ptr(value_pages), _ptr(block_table),
        _ptr(context_lens), float(scale), int(bool(causal)), _ptr(mask), int(mask_S), _ptr(out),
        _ptr(workspace), int(workspace_bytes), _stream(stream), int(schedule))


def pa_paged_attention_varlen(shape, query, key_pages, value_pages, block_table, context_lens,
                              cu_q, total_q, scale, causal, out, workspace, workspace_bytes,
                              stream=None, schedule=PA_SCHED_AUTO) -> int:
    """Ragged batch: query/out [total_q, H_q, D] packed by token, cu_q int32
    device tensor [B + 1]; shape.L bounds every sequence's query count."""
    return load().pa_paged_attention_varlen(
        ctypes.byref(shape), _ptr(query), _ptr(key_pages), _ptr(value_pages), _ptr(block_table),
        _ptr(context_lens), _ptr(cu_q), int(total_q), float(scale), int(bool(causal)),
        _ptr(out), _ptr(workspace), int(workspace_bytes), _stream(stream), int(schedule))


def pa_validate_metadata_varlen(shape, block_table, context_lens, cu_q, total_q, causal,
                                stream=None) -> int:
    return load().pa_validate_metadata_varlen(
        ctypes.byref(shape), _ptr(block_table), _ptr(context_lens), _ptr(cu_q), int(total_q),
        int(bool(causal)), _stream(stream))


def pa_selftest_wait_timeout(workspace, workspace_bytes, timeout_us, stream=None) -> int:
    return load().pa_selftest_wait_timeout(_ptr(workspace), int(workspace_bytes),
                                           int(timeout_us), _stream(stream))


def pa_append_kv(shape, k_new, v_new, key_pages, value_pages, block_table, context_lens,
                 workspace, workspace_bytes, stream=None) -> int:
    return load().pa_append_kv(
        ctypes.byref(shape), _ptr(k_new), _ptr(v_new), _ptr(key_pages), _ptr(value_pages),
        _ptr(block_table), _ptr(context_lens), _ptr(workspace), int(workspace_bytes),
        _stream(stream))


def pa_check_device_flag(workspace, clear=False, stream=None):
    """Returns (status, flag word)."""
    f = ctypes.c_uint32(0)
    st = load().pa_check_device_flag(_ptr(workspace), ctypes.byref(f), int(bool(clear)),
                                     _stream(stream))
    return st, int(f.value)


def pa_validate_metadata(shape, block_table, context_lens, causal, stream=None) -> int:
    return load().pa_validate_metadata(ctypes.byref(shape), _ptr(block_table),
                                       _ptr(context_lens), int(bool(causal)), _stream(stream))


def pa_choose_schedule(shape) -> int:
    return int(load().pa_choose_schedule(ctypes.byref(shape)))


def pa_launch_count(shape, schedule=PA_SCHED_AUTO) -> int:
    return int(load().pa_launch_count(ctypes.byref(shape), int(schedule)))


# ---- the pages' model-facing call ------------------------------------------
def new_workspace(shape: pa_shape, device=None):
    """Zeroed workspace for `shape` on `device` (flag word starts at 0)."""
    import torch
    n = pa_workspace_bytes(shape)
    if n == 0:
        raise PagedAttentionError(PA_ERR_INVALID_ARG, "pa_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def paged_attention(query, key_pages, value_pages, block_table, context_lens, page_size,
                    scale=None, causal=True, *, mask=None, out=None, workspace=None,
                    schedule=PA_SCHED_AUTO, stream=None):
    """out[B, H_q, L, D] = softmax(scale * q.K^T + mask over visible keys) . V,
    with K/V read from the paged pool through block_table.  mask: optional
    fp32 CUDA tensor [B * H_q, L, S_mask] (S_mask >= the table's capacity, a
    multiple of 4) added to the scaled scores."""
    import torch
    shape = shape_of(query, key_pages, block_table)
    if shape.page_size != int(page_size):
        raise ValueError("page_size disagrees with key_pages.shape[2]")
    for name, t in (("query", query), ("key_pages", key_pages), ("value_pages", value_pages),
                    ("block_table", block_table), ("context_lens", context_lens)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if block_table.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_table and context_lens must be int32")
    if scale is None:
        scale = 1.0 / math.sqrt(query.shape[-1])
    if out is None:
        out = torch.empty_like(query)
    if workspace is None:
        workspace = new_workspace(shape, query.device)
    if mask is None:
        st = pa_paged_attention_sched(shape, query, key_pages, value_pages, block_table,
                                      context_lens, scale, causal, out, workspace,
                                      workspace.numel(), stream, schedule)
    else:
        if mask.dtype != torch.float32 or not mask.is_cuda or not mask.is_contiguous():
            raise ValueError("mask must be a contiguous fp32 CUDA tensor")
        if mask.dim() != 3 or mask.shape[0] != shape.B * shape.H_q or mask.shape[1] != shape.L:
            raise ValueError("mask must be [B * H_q, L, S_mask]")
        st = pa_paged_attention_masked(shape, query, key_pages, value_pages, block_table,
                                       context_lens, scale, causal, mask, mask.shape[2], out,
                                       workspace, workspace.numel(), stream, schedule)
    if st != PA_OK:
        raise PagedAttentionError(st, "pa_paged_attention")
    return out


def append_kv(k_new, v_new, key_pages, value_pages, block_table, context_lens, *,
              workspace=None, stream=None):
    """Stores k_new/v_new [B, H_kv, L, D] -- the last L positions of each
    context -- in their pages, through block_table (in place)."""
    import torch
    B_, H_kv, L, D = k_new.shape
    P, Hk, ps, Dk = key_pages.shape
    if Hk != H_kv or Dk != D or v_new.shape != k_new.shape:
        raise ValueError("k_new/v_new must be [B, H_kv, L, D] matching the pools")
    if k_new.dtype != key_pages.dtype or v_new.dtype != value_pages.dtype:
        raise ValueError("new rows must have the pools' dtype")
    dtype = PA_BF16 if key_pages.dtype == torch.bfloat16 else PA_F32
    shape = make_shape(B_, H_kv, H_kv, L, D, P, ps, block_table.shape[1], dtype)
    if workspace is None:
        workspace = torch.zeros(256, dtype=torch.uint8, device=key_pages.device)
    st = pa_append_kv(shape, k_new.contiguous(), v_new.contiguous(), key_pages, value_pages,
                      block_table, context_lens, workspace, workspace.numel(), stream)
    if st != PA_OK:
        raise PagedAttentionError(st, "pa_append_kv")
    return workspace


def shape_of_varlen(query, key_pages, block_table, max_L) -> pa_shape:
    """pa_shape of a ragged batch: query [total_q, H_q, D] packed by token,
    B = block_table.shape[0] sequences, L = max_L (bounds every L_b)."""
    import torch
    T, H_q, D = query.shape
    P, H_kv, ps, D2 = key_pages.shape
    if D2 != D:
        raise ValueError("query and pages disagree on head dim")
    if query.dtype != key_pages.dtype:
        raise ValueError("query and pages must share a dtype")
    dt = {torch.bfloat16: PA_BF16, torch.float32: PA_F32}.get(query.dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {query.dtype}")
    return make_shape(block_table.shape[0], H_q, H_kv, max(1, int(max_L)), D, P, ps,
                      block_table.shape[1], dt)


def paged_attention_varlen(query, key_pages, value_pages, block_table, context_lens, cu_q,
                           max_L, page_size, scale=None, causal=True, *, out=None,
                           workspace=None, schedule=PA_SCHED_AUTO, stream=None):
    """Ragged batch: out[total_q, H_q, D]; sequence b's queries are tokens
    cu_q[b] .. cu_q[b+1]-1 of `query` and the last positions of its context.
    max_L bounds every cu_q[b+1] - cu_q[b]."""
    import torch
    shape = shape_of_varlen(query, key_pages, block_table, max_L)
    if shape.page_size != int(page_size):
        raise ValueError("page_size disagrees with key_pages.shape[2]")
    for name, t in (("query", query), ("key_pages", key_pages), ("value_pages", value_pages),
                    ("block_table", block_table), ("context_lens", context_lens), ("cu_q", cu_q)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if block_table.dtype != torch.int32 or context_lens.dtype != torch.int32 or \
            cu_q.dtype != torch.int32:
        raise ValueError("block_table, context_lens and cu_q must be int32")
    if cu_q.numel() != shape.B + 1 or context_lens.numel() != shape.B:
        raise ValueError("cu_q must hold B + 1 offsets and context_lens B lengths")
    if scale is None:
        scale = 1.0 / math.sqrt(query.shape[-1])
    if out is None:
        out = torch.empty_like(query)
    if workspace is None:
        workspace = new_workspace(shape, query.device)
    st = pa_paged_attention_varlen(shape, query, key_pages, value_pages, block_table,
                                   context_lens, cu_q, query.shape[0], scale, causal, out,
                                   workspace, workspace.numel(), stream, schedule)
    if st != PA_OK:
        raise PagedAttentionError(st, "pa_paged_attention_varlen")
    return out


# ---- 4-bit pages, key weights and eviction -----------------------------------
def pa_append_kv_q4(shape, k_new, v_new, pool, block_table, context_lens, workspace,
                    workspace_bytes, stream=None) -> int:
    return load().pa_append_kv_q4(
        ctypes.byref(shape), _ptr(k_new), _ptr(v_new), _q4(pool), _ptr(block_table),
        _ptr(context_lens), _ptr(workspace), int(workspace_bytes), _stream(stream))


def pa_gather_kv_q4(shape, pool, block_table, context_lens, n, tail, k_dense, v_dense, workspace,
                    workspace_bytes, stream=None) -> int:
    return load().pa_gather_kv_q4(
        ctypes.byref(shape), _q4(pool), _ptr(block_table), _ptr(context_lens), int(n),
        int(bool(tail)), _ptr(k_dense), _ptr(v_dense), _ptr(workspace), int(workspace_bytes),
        _stream(stream))


def pa_q4_workspace_bytes(shape, key_weights=False) -> int:
    return int(load().pa_q4_workspace_bytes(ctypes.byref(shape), int(bool(key_weights))))


def pa_weights_workspace_bytes(shape) -> int:
    return int(load().pa_weights_workspace_bytes(ctypes.byref(shape)))


def pa_paged_attention_q4(shape, query, pool, block_table, context_lens, scale, causal,
                          key_weights, key_weights_out, weights_S, out, workspace,
                          workspace_bytes, stream=None) -> int:
    return load().pa_paged_attention_q4(
        ctypes.byref(shape), _ptr(query), _q4(pool), _ptr(block_table), _ptr(context_lens),
        float(scale), int(bool(causal)), _ptr(key_weights), _ptr(key_weights_out),
        int(weights_S), _ptr(out), _ptr(workspace), int(workspace_bytes), _stream(stream))


def pa_paged_attention_weights(shape, query, key_pages, value_pages, block_table, context_lens,
                               scale, causal, key_weights, key_weights_out, weights_S, out,
                               workspace, workspace_bytes, stream=None) -> int:
    return load().pa_paged_attention_weights(
        ctypes.byref(shape), _ptr(query), _ptr(key_pages), _ptr(value_pages), _ptr(block_table),
        _ptr(context_lens), float(scale), int(bool(causal)), _ptr(key_weights),
        _ptr(key_weights_out), int(weights_S), _ptr(out), _ptr(workspace), int(workspace_bytes),
        _stream(stream))


def pa_evict_kv(shape, key_pages, value_pages, block_table, context_lens, key_weights, weights_S,
                keep, recent, dst_block_table, dst_max_pages_per_seq, context_lens_out,
                key_weights_out, weights_out_S, kept, workspace, workspace_bytes,
                stream=None) -> int:
    return load().pa_evict_kv(
        ctypes.byref(shape), _ptr(key_pages), _ptr(value_pages), _ptr(block_table),
        _ptr(context_lens), _ptr(key_weights), int(weights_S), int(keep), int(recent),
        _ptr(dst_block_table), int(dst_max_pages_per_seq), _ptr(context_lens_out),
        _ptr(key_weights_out), int(weights_out_S), _ptr(kept), _ptr(workspace),
        int(workspace_bytes), _stream(stream))


def pa_evict_kv_q4(shape, pool, block_table, context_lens, key_weights, weights_S, keep, recent,
                   dst_block_table, dst_max_pages_per_seq, context_lens_out, key_weights_out,
                   weights_out_S, kept, workspace, workspace_bytes, stream=None) -> int:
    return load().pa_evict_kv_q4(
        ctypes.byref(shape), _q4(pool), _ptr(block_table), _ptr(context_lens),
        _ptr(key_weights), int(weights_S), int(keep), int(recent), _ptr(dst_block_table),
        int(dst_max_pages_per_seq), _ptr(context_lens_out), _ptr(key_weights_out),
        int(weights_out_S), _ptr(kept), _ptr(workspace), int(workspace_bytes), _stream(stream))


class Q4Pool:
    """A page pool held in 4 bits (layout in include/paged_attn.h): uint8
    codes [num_pages, H_kv, page_size, 64] and scales [..., 8] of keys and
    values, checked once here.  `dims` is (num_pages, H_kv, page_size)."""
    __slots__ = ("key_codes", "key_scales", "value_codes", "value_scales", "dims", "device",
                 "c_pool")

    def __init__(self, key_codes, key_scales, value_codes, value_scales):
        import torch
        if key_codes.dim() != 4:
            raise ValueError("key_codes must be uint8 [num_pages, H_kv, page_size, 64]")
        self.dims = tuple(key_codes.shape[:3])
        self.device = key_codes.device
        tensors = (("key_codes", key_codes, 64), ("key_scales", key_scales, 8),
                   ("value_codes", value_codes, 64), ("value_scales", value_scales, 8))
        for name, t, w in tensors:
            if t.dtype != torch.uint8 or tuple(t.shape) != (*self.dims, w):
                raise ValueError(f"{name} must be uint8 [num_pages, H_kv, page_size, {w}]")
            if not t.is_cuda or t.device != self.device or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous CUDA tensor on {self.device}")
            setattr(self, name, t)
        self.c_pool = pa_q4_pool(*[t.data_ptr() for t in self])

    def __iter__(self):
        return iter((self.key_codes, self.key_scales, self.value_codes, self.value_scales))


class Evicted(NamedTuple):
    """What an eviction leaves: the new lengths [B], the kept keys' weights
    [B, H_kv, keep] (or the caller's key_weights_out) and their old positions
    [B, H_kv, keep] (-1 past the end)."""
    context_lens: object
    key_weights: object
    kept: object


def _q4(pool):
    """A Q4Pool, four addresses or tensors, or None, for the C calls."""
    if isinstance(pool, Q4Pool):
        return ctypes.byref(pool.c_pool)
    return None if pool is None else ctypes.byref(pa_q4_pool(*[_ptr(t) for t in pool]))


def new_q4_pool(num_pages, H_kv, page_size, device=None) -> Q4Pool:
    """A 4-bit pool of zeros (head dim 128)."""
    import torch

    def new(n):
        return torch.zeros((num_pages, H_kv, page_size, n), dtype=torch.uint8,
                           device=device or "cuda")
    return Q4Pool(new(64), new(8), new(64), new(8))


def new_cache_workspace(device=None):
    """Zeroed workspace of append_kv_q4, gather_kv_q4 and evict_kv*."""
    import torch
    return torch.zeros(256, dtype=torch.uint8, device=device or "cuda")


# The calls below are made per layer and token: what they check is checked with
# few and cheap tensor queries, and torch is looked up once.
_torch = None


def _load_torch():
    global _torch
    import torch
    _torch = torch
    return torch


def _dtype_id(t):
    torch = _torch or _load_torch()
    if t is torch.bfloat16:
        return PA_BF16
    if t is torch.float32:
        return PA_F32
    raise ValueError(f"unsupported dtype {t}")


def _on_device(index, *named):
    """Every (name, tensor) is contiguous on CUDA device `index`."""
    for name, t in named:
        if t.get_device() != index or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous tensor on cuda:{index}")


def _table(block_table, context_lens, B):
    int32 = (_torch or _load_torch()).int32
    if block_table.dtype is not int32 or context_lens.dtype is not int32:
        raise ValueError("block tables and context lengths must be int32")
    if block_table.dim() != 2 or block_table.shape[0] != B or context_lens.shape != (B,):
        raise ValueError("block_table must be [B, max_pages_per_seq] and context_lens [B]")


def _pages_dims(key_pages, value_pages):
    """(num_pages, H_kv, page_size) of a checked bf16 or fp32 pool."""
    if key_pages.dim() != 4 or key_pages.shape != value_pages.shape or \
            key_pages.dtype != value_pages.dtype:
        raise ValueError("key and value pages must be alike, [num_pages, H_kv, page_size, D]")
    index = key_pages.get_device()
    if index < 0:
        raise ValueError("key_pages must be on a CUDA device")
    _on_device(index, ("key_pages", key_pages), ("value_pages", value_pages))
    return key_pages.shape[:3]


def _weights_shape(name, w, B_, H_kv, capacity):
    torch = _torch or _load_torch()
    if w.dtype is not torch.float32 or w.dim() != 3 or w.shape[:2] != (B_, H_kv) or \
            w.shape[2] < capacity:
        raise ValueError(f"{name} must be fp32 [B, H_kv, S] with S >= {capacity}")


def _launch(name, index, fn, *args):
    """fn(*args, stream) with device `index` current, on its current stream."""
    torch = _torch or _load_torch()
    raw = torch._C  # (the tensors are there, so CUDA is initialised)
    if raw._cuda_getDevice() == index:
        st = fn(*args, raw._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if st != PA_OK:
        raise PagedAttentionError(st, name)


def _streamed(fn):
    """Runs the call with its `stream` argument (a torch stream or a raw
    handle, of the tensors' device) current, so that what it allocates, zeroes
    and returns belongs to that stream too."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        import torch
        device = next((x.device for x in (*args, *kw.values()) if hasattr(x, "device")), None)
        if device is None or device.type != "cuda":
            return fn(*args, **kw)  # (which refuses it)
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device) if stream else \
                torch.cuda.default_stream(device)
        elif stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


@_streamed
def append_kv_q4(k_new, v_new, pool, block_table, context_lens, *, workspace=None):
    """Rounds k_new/v_new [B, H_kv, L, 128] (bf16 or fp32) -- the last L
    positions of each context -- to 4 bits into their pages (in place)."""
    P, H_kv, ps = pool.dims
    if k_new.dim() != 4 or k_new.shape[1] != H_kv or k_new.shape[3] != 128 or \
            v_new.shape != k_new.shape or v_new.dtype != k_new.dtype:
        raise ValueError("k_new/v_new must be alike, [B, H_kv, L, 128] matching the pool")
    B_, _, L, D = k_new.shape
    _table(block_table, context_lens, B_)
    k_new, v_new = k_new.contiguous(), v_new.contiguous()
    if workspace is None:
        workspace = new_cache_workspace(pool.device)
    index = pool.device.index
    _on_device(index, ("k_new", k_new), ("v_new", v_new), ("block_table", block_table),
               ("context_lens", context_lens), ("workspace", workspace))
    shape = pa_shape(B_, H_kv, H_kv, L, D, P, ps, block_table.shape[1], _dtype_id(k_new.dtype))
    _launch("pa_append_kv_q4", index, (_lib or load()).pa_append_kv_q4, ctypes.byref(shape),
            k_new.data_ptr(), v_new.data_ptr(), ctypes.byref(pool.c_pool),
            block_table.data_ptr(), context_lens.data_ptr(), workspace.data_ptr(),
            workspace.numel())
    return workspace


@_streamed
def gather_kv_q4(pool, block_table, context_lens, n, *, tail=False, dtype=None, workspace=None):
    """Dense dequantised (keys, values), each [B, H_kv, n, 128] of `dtype`
    (bf16 by default, or fp32; both exact): positions 0 .. n - 1, or with
    `tail` the last n of each context; zeros outside a context."""
    torch = _torch or _load_torch()
    dtype = dtype or torch.bfloat16
    P, H_kv, ps = pool.dims
    B_ = block_table.shape[0]
    _table(block_table, context_lens, B_)
    if workspace is None:
        workspace = new_cache_workspace(pool.device)
    index = pool.device.index
    _on_device(index, ("block_table", block_table), ("context_lens", context_lens),
               ("workspace", workspace))
    shape = pa_shape(B_, H_kv, H_kv, 1, 128, P, ps, block_table.shape[1], _dtype_id(dtype))
    k = torch.empty((B_, H_kv, n, 128), dtype=dtype, device=pool.device)
    v = torch.empty_like(k)
    _launch("pa_gather_kv_q4", index, (_lib or load()).pa_gather_kv_q4, ctypes.byref(shape),
            ctypes.byref(pool.c_pool), block_table.data_ptr(), context_lens.data_ptr(), n,
            bool(tail), k.data_ptr(), v.data_ptr(), workspace.data_ptr(), workspace.numel())
    return k, v


def _q4_shape(query, pool, block_table):
    P, H_kv, ps = pool.dims
    if query.dim() != 4 or query.shape[3] != 128:
        raise ValueError("query must be [B, H_q, L, 128]")
    B_, H_q, L, D = query.shape
    return pa_shape(B_, H_q, H_kv, L, D, P, ps, block_table.shape[1], _dtype_id(query.dtype))


def _workspace(n, device, name):
    """n bytes, the flag and the counters in front zeroed (all that needs it)."""
    import torch
    if n == 0:
        raise PagedAttentionError(PA_ERR_INVALID_ARG, name)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def new_q4_workspace(query, pool, block_table, key_weights=None):
    """Workspace of paged_attention_q4 for tensors of these shapes and for any
    with at most their B, L and table width, with key weights, without, or
    (None) for either."""
    import torch
    shape = _q4_shape(query, pool, block_table)
    kinds = (False, True) if key_weights is None else (key_weights,)
    with torch.cuda.device(query.device):
        n = max(pa_q4_workspace_bytes(shape, k) for k in kinds)
    return _workspace(n, query.device, "pa_q4_workspace_bytes")


def new_weights_workspace(query, key_pages, block_table):
    """Workspace of paged_attention_weights for tensors of these shapes and for
    any with at most their B, L and table width."""
    import torch
    with torch.cuda.device(query.device):
        n = pa_weights_workspace_bytes(shape_of(query, key_pages, block_table))
    return _workspace(n, query.device, "pa_weights_workspace_bytes")


def _attend(name, fn, pools, shape, query, block_table, context_lens, page_size, scale, causal,
            key_weights, key_weights_out, out, workspace):
    if shape.page_size != page_size:
        raise ValueError("page_size disagrees with the pool's")
    _table(block_table, context_lens, shape.B)
    index = query.get_device()
    if out is None:
        out = (_torch or _load_torch()).empty_like(query)
    elif out.shape != query.shape or out.dtype != query.dtype:
        raise ValueError("out must be like query")
    w_S = w_in = w_out = 0
    if key_weights_out is not None:
        _weights_shape("key_weights_out", key_weights_out, shape.B, shape.H_kv,
                       shape.max_pages_per_seq * shape.page_size)
        _on_device(index, ("key_weights_out", key_weights_out))
        w_S, w_out = key_weights_out.shape[2], key_weights_out.data_ptr()
        if key_weights is not None:
            if key_weights.shape != key_weights_out.shape or \
                    key_weights.dtype != key_weights_out.dtype:
                raise ValueError("key_weights must be like key_weights_out")
            _on_device(index, ("key_weights", key_weights))
            w_in = key_weights.data_ptr()
    elif key_weights is not None:
        raise ValueError("key_weights without key_weights_out")
    _on_device(index, ("query", query), ("block_table", block_table),
               ("context_lens", context_lens), ("out", out), ("workspace", workspace))
    if scale is None:
        scale = 1.0 / math.sqrt(shape.D)
    _launch(name, index, fn, ctypes.byref(shape), query.data_ptr(), *pools,
            block_table.data_ptr(), context_lens.data_ptr(), scale, bool(causal), w_in, w_out,
            w_S, out.data_ptr(), workspace.data_ptr(), workspace.numel())
    return out


@_streamed
def paged_attention_q4(query, pool, block_table, context_lens, page_size, scale=None, causal=True,
                       *, key_weights=None, key_weights_out=None, out=None, workspace=None):
    """paged_attention over a 4-bit pool (query bf16 or fp32).  With
    key_weights_out (fp32 [B, H_kv, S], S >= the table's capacity) the call
    also writes key_weights (zeros if None; may be key_weights_out itself)
    plus the probability each key received."""
    shape = _q4_shape(query, pool, block_table)
    if query.get_device() != pool.device.index:
        raise ValueError(f"query must be on {pool.device}")
    if workspace is None:
        workspace = new_q4_workspace(query, pool, block_table, key_weights_out is not None)
    return _attend("pa_paged_attention_q4", (_lib or load()).pa_paged_attention_q4,
                   (ctypes.byref(pool.c_pool),), shape, query, block_table, context_lens,
                   page_size, scale, causal, key_weights, key_weights_out, out, workspace)


@_streamed
def paged_attention_weights(query, key_pages, value_pages, block_table, context_lens, page_size,
                            scale=None, causal=True, *, key_weights=None, key_weights_out=None,
                            out=None, workspace=None):
    """paged_attention over bf16 pages that also writes key_weights_out (fp32
    [B, H_kv, S], S >= the table's capacity): key_weights (zeros if None; may
    be key_weights_out itself) plus the probability each key received."""
    P, H_kv, ps = _pages_dims(key_pages, value_pages)
    if query.dim() != 4 or query.dtype != key_pages.dtype or query.shape[3] != key_pages.shape[3]:
        raise ValueError("query must be [B, H_q, L, D] of the pages' dtype and head dim")
    B_, H_q, L, D = query.shape
    shape = pa_shape(B_, H_q, H_kv, L, D, P, ps, block_table.shape[1], _dtype_id(query.dtype))
    if shape.dtype != PA_BF16:
        raise PagedAttentionError(PA_ERR_UNSUPPORTED, "pa_paged_attention_weights")
    if query.get_device() != key_pages.get_device():
        raise ValueError(f"query must be on {key_pages.device}")
    if key_weights_out is None:
        raise ValueError("key_weights_out is what this call is for: use paged_attention")
    if workspace is None:
        workspace = new_weights_workspace(query, key_pages, block_table)
    return _attend("pa_paged_attention_weights", (_lib or load()).pa_paged_attention_weights,
                   (key_pages.data_ptr(), value_pages.data_ptr()), shape, query, block_table,
                   context_lens, page_size, scale, causal, key_weights, key_weights_out, out,
                   workspace)


def _evict(name, fn, pools, dims, dtype_id, device, block_table, context_lens, key_weights, keep,
           recent, dst_block_table, key_weights_out, workspace):
    torch = _torch or _load_torch()
    P, H_kv, ps = dims
    B_ = block_table.shape[0]
    _table(block_table, context_lens, B_)
    _table(dst_block_table, context_lens, B_)
    _weights_shape("key_weights", key_weights, B_, H_kv, block_table.shape[1] * ps)
    if workspace is None:
        workspace = new_cache_workspace(device)
    index = device.index
    _on_device(index, ("block_table", block_table), ("context_lens", context_lens),
               ("key_weights", key_weights), ("dst_block_table", dst_block_table),
               ("workspace", workspace))
    if not 1 <= keep <= dst_block_table.shape[1] * ps:
        raise ValueError("keep must be at least 1 and fit dst_block_table")
    if not 0 <= recent <= keep:
        raise ValueError("recent must be at least 0 and at most keep")
    shape = pa_shape(B_, H_kv, H_kv, 1, 128, P, ps, block_table.shape[1], dtype_id)
    lens = torch.empty(B_, dtype=torch.int32, device=device)
    weights = key_weights_out
    if weights is None:
        weights = torch.empty((B_, H_kv, keep), dtype=torch.float32, device=device)
    else:
        _weights_shape("key_weights_out", weights, B_, H_kv, keep)
        _on_device(index, ("key_weights_out", weights))
    kept = torch.empty((B_, H_kv, keep), dtype=torch.int32, device=device)
    _launch(name, index, fn, ctypes.byref(shape), *pools, block_table.data_ptr(),
            context_lens.data_ptr(), key_weights.data_ptr(), key_weights.shape[2], keep, recent,
            dst_block_table.data_ptr(), dst_block_table.shape[1], lens.data_ptr(),
            weights.data_ptr(), weights.shape[2], kept.data_ptr(), workspace.data_ptr(), workspace.numel())
    return Evicted(lens, weights, kept)


@_streamed
def evict_kv(key_pages, value_pages, block_table, context_lens, key_weights, keep, recent,
             dst_block_table, *, key_weights_out=None, workspace=None) -> Evicted:
    """Trims every (sequence, kv head) to its `recent` last keys and the
    heaviest others, `keep` in all, copied in order to the pages of
    dst_block_table [B, n] (other pages of the same pool).  Returns the new
    lengths, the kept keys' weights [B, H_kv, keep] and their old positions.
    key_weights_out (fp32 [B, H_kv, S], S >= keep, not key_weights) receives
    the weights, then zeros: with S the new table's capacity it goes straight
    into the next attention call."""
    dims = _pages_dims(key_pages, value_pages)
    if key_pages.shape[3] != 128:
        raise ValueError("head dim must be 128")
    return _evict("pa_evict_kv", (_lib or load()).pa_evict_kv,
                  (key_pages.data_ptr(), value_pages.data_ptr()), dims,
                  _dtype_id(key_pages.dtype), key_pages.device, block_table, context_lens,
                  key_weights, keep, recent, dst_block_table, key_weights_out, workspace)


@_streamed
def evict_kv_q4(pool, block_table, context_lens, key_weights, keep, recent, dst_block_table, *,
                key_weights_out=None, workspace=None) -> Evicted:
    """evict_kv of a 4-bit pool."""
    return _evict("pa_evict_kv_q4", (_lib or load()).pa_evict_kv_q4, (ctypes.byref(pool.c_pool),),
                  pool.dims, PA_BF16, pool.device, block_table, context_lens, key_weights, keep,
                  recent, dst_block_table, key_weights_out, workspace)


# ---- trees of drafted tokens --------------------------------------------------
def pa_tree_mask(B_, L, parents, mask, depths, workspace, workspace_bytes, stream=None) -> int:
    return load().pa_tree_mask(int(B_), int(L), _ptr(parents), _ptr(mask), _ptr(depths),
                               _ptr(workspace), int(workspace_bytes), _stream(stream))


def pa_tree_workspace_bytes(shape) -> int:
    return int(load().pa_tree_workspace_bytes(ctypes.byref(shape)))


def pa_paged_attention_tree(shape, query, key_pages, value_pages, block_table, context_lens,
                            tree_mask, scale, out, workspace, workspace_bytes, stream=None) -> int:
    return load().pa_paged_attention_tree(
        ctypes.byref(shape), _ptr(query), _ptr(key_pages), _ptr(value_pages), _ptr(block_table),
        _ptr(context_lens), _ptr(tree_mask), float(scale), _ptr(out), _ptr(workspace),
        int(workspace_bytes), _stream(stream))


def pa_paged_attention_tree_q4(shape, query, pool, block_table, context_lens, tree_mask, scale,
                               out, workspace, workspace_bytes, stream=None) -> int:
    return load().pa_paged_attention_tree_q4(
        ctypes.byref(shape), _ptr(query), _q4(pool), _ptr(block_table), _ptr(context_lens),
        _ptr(tree_mask), float(scale), _ptr(out), _ptr(workspace), int(workspace_bytes),
        _stream(stream))


def pa_compact_kv(shape, key_pages, value_pages, block_table, context_lens, path, path_n,
                  path_lens, context_lens_out, workspace, workspace_bytes, stream=None) -> int:
    return load().pa_compact_kv(
        ctypes.byref(shape), _ptr(key_pages), _ptr(value_pages), _ptr(block_table),
        _ptr(context_lens), _ptr(path), int(path_n), _ptr(path_lens), _ptr(context_lens_out),
        _ptr(workspace), int(workspace_bytes), _stream(stream))


def pa_compact_kv_q4(shape, pool, block_table, context_lens, path, path_n, path_lens,
                     context_lens_out, workspace, workspace_bytes, stream=None) -> int:
    return load().pa_compact_kv_q4(
        ctypes.byref(shape), _q4(pool), _ptr(block_table), _ptr(context_lens), _ptr(path),
        int(path_n), _ptr(path_lens), _ptr(context_lens_out), _ptr(workspace),
        int(workspace_bytes), _stream(stream))


def pa_pages_workspace_bytes(shape) -> int:
    return int(load().pa_pages_workspace_bytes(ctypes.byref(shape)))


def pa_fork_pages(shape, block_table, context_lens, page_refs, sources, targets, lens, n,
                  workspace, workspace_bytes, stream=None) -> int:
    return load().pa_fork_pages(
        ctypes.byref(shape), _ptr(block_table), _ptr(context_lens), _ptr(page_refs),
        _ptr(sources), _ptr(targets), _ptr(lens), int(n), _ptr(workspace), int(workspace_bytes),
        _stream(stream))


def pa_resize_pages(shape, block_table, context_lens, page_refs, new_lens, copies, workspace,
                    workspace_bytes, stream=None) -> int:
    return load().pa_resize_pages(
        ctypes.byref(shape), _ptr(block_table), _ptr(context_lens), _ptr(page_refs),
        _ptr(new_lens), _ptr(copies), _ptr(workspace), int(workspace_bytes), _stream(stream))


def pa_copy_pages(shape, key_pages, value_pages, copies, n, workspace, workspace_bytes,
                  stream=None) -> int:
    return load().pa_copy_pages(
        ctypes.byref(shape), _ptr(key_pages), _ptr(value_pages), _ptr(copies), int(n),
        _ptr(workspace), int(workspace_bytes), _stream(stream))


def pa_copy_pages_q4(shape, pool, copies, n, workspace, workspace_bytes, stream=None) -> int:
    return load().pa_copy_pages_q4(
        ctypes.byref(shape), _q4(pool), _ptr(copies), int(n), _ptr(workspace),
        int(workspace_bytes), _stream(stream))


def _c_int(name, x):
    if not 0 < x < 1 << 31:  # (ctypes keeps the low 32 bits of any number)
        raise ValueError(f"{name} must be positive and fit 32 bits")


def _int32(name, t, shape):
    if t.dtype is not (_torch or _load_torch()).int32 or t.shape != shape:
        raise ValueError(f"{name} must be int32 {list(shape)}")


@_streamed
def tree_mask(parents, *, workspace=None):
    """(mask, depths) of drafted trees: parents int32 [B, L], parents[b, i] < i
    the draft that draft i follows, -1 for the last position before the
    drafts, -2 for a slot without a draft.  mask int32 [B, L, (L + 31) // 32]
    holds, as bits, the drafts that draft i sees (its ancestors and itself);
    depths int32 [B, L] counts its ancestors (-1: no draft).  L <= 1024."""
    torch = _torch or _load_torch()
    if parents.dim() != 2 or parents.dtype is not torch.int32:
        raise ValueError("parents must be int32 [B, L]")
    index = parents.get_device()
    if index < 0:
        raise ValueError("parents must be on a CUDA device")
    if workspace is None:
        workspace = new_cache_workspace(parents.device)
    _on_device(index, ("parents", parents), ("workspace", workspace))
    B_, L = parents.shape
    mask = torch.empty((B_, L, (L + 31) // 32), dtype=torch.int32, device=parents.device)
    depths = torch.empty_like(parents)
    _launch("pa_tree_mask", index, (_lib or load()).pa_tree_mask, B_, L, parents.data_ptr(),
            mask.data_ptr(), depths.data_ptr(), workspace.data_ptr(), workspace.numel())
    return mask, depths


def new_tree_workspace(query, pool, block_table):
    """Workspace of paged_attention_tree (pool: the key pages) or
    paged_attention_tree_q4 (pool: the Q4Pool) for tensors of these shapes and
    for any with at most their B, L and table width."""
    import torch
    shape = _q4_shape(query, pool, block_table) if isinstance(pool, Q4Pool) else \
        shape_of(query, pool, block_table)
    with torch.cuda.device(query.device):
        n = pa_tree_workspace_bytes(shape)
    return _workspace(n, query.device, "pa_tree_workspace_bytes")


def _attend_tree(name, fn, pools, shape, query, block_table, context_lens, tree_mask, page_size,
                 scale, out, workspace):
    if shape.page_size != page_size:
        raise ValueError("page_size disagrees with the pool's")
    _table(block_table, context_lens, shape.B)
    _int32("tree_mask", tree_mask, (shape.B, shape.L, (shape.L + 31) // 32))
    index = query.get_device()
    if out is None:
        out = (_torch or _load_torch()).empty_like(query)
    elif out.shape != query.shape or out.dtype != query.dtype:
        raise ValueError("out must be like query")
    _on_device(index, ("query", query), ("block_table", block_table),
               ("context_lens", context_lens), ("tree_mask", tree_mask), ("out", out),
               ("workspace", workspace))
    if scale is None:
        scale = 1.0 / math.sqrt(shape.D)
    _launch(name, index, fn, ctypes.byref(shape), query.data_ptr(), *pools,
            block_table.data_ptr(), context_lens.data_ptr(), tree_mask.data_ptr(), scale,
            out.data_ptr(), workspace.data_ptr(), workspace.numel())
    return out


@_streamed
def paged_attention_tree(query, key_pages, value_pages, block_table, context_lens, tree_mask,
                         page_size, scale=None, *, out=None, workspace=None):
    """Attention of L drafted tokens per sequence (query [B, H_q, L, 128], the
    last L of context_lens, stored by append_kv): each sees every position
    before the drafts and the drafts of its row of tree_mask (int32 [B, L,
    (L + 31) // 32], from ``tree_mask`` or any other).  A slot whose row is 0
    holds no draft: its output is 0 and nobody sees it."""
    P, H_kv, ps = _pages_dims(key_pages, value_pages)
    if query.dim() != 4 or query.dtype != key_pages.dtype or query.shape[3] != key_pages.shape[3]:
        raise ValueError("query must be [B, H_q, L, D] of the pages' dtype and head dim")
    B_, H_q, L, D = query.shape
    shape = pa_shape(B_, H_q, H_kv, L, D, P, ps, block_table.shape[1], _dtype_id(query.dtype))
    if query.get_device() != key_pages.get_device():
        raise ValueError(f"query must be on {key_pages.device}")
    if workspace is None:
        workspace = new_tree_workspace(query, key_pages, block_table)
    return _attend_tree("pa_paged_attention_tree", (_lib or load()).pa_paged_attention_tree,
                        (key_pages.data_ptr(), value_pages.data_ptr()), shape, query, block_table,
                        context_lens, tree_mask, page_size, scale, out, workspace)


@_streamed
def paged_attention_tree_q4(query, pool, block_table, context_lens, tree_mask, page_size,
                            scale=None, *, out=None, workspace=None):
    """paged_attention_tree over a 4-bit pool (query bf16 or fp32)."""
    shape = _q4_shape(query, pool, block_table)
    if query.get_device() != pool.device.index:
        raise ValueError(f"query must be on {pool.device}")
    if workspace is None:
        workspace = new_tree_workspace(query, pool, block_table)
    return _attend_tree("pa_paged_attention_tree_q4", (_lib or load()).pa_paged_attention_tree_q4,
                        (ctypes.byref(pool.c_pool),), shape, query, block_table, context_lens,
                        tree_mask, page_size, scale, out, workspace)


def _compact(name, fn, pools, dims, dtype_id, device, block_table, context_lens, path, path_lens,
             L, workspace):
    torch = _torch or _load_torch()
    P, H_kv, ps = dims
    B_ = block_table.shape[0]
    _c_int("L", L)
    _table(block_table, context_lens, B_)
    if path.dim() != 2 or path.shape[1] < 1:
        raise ValueError("path must be int32 [B, n]")
    _int32("path", path, (B_, path.shape[1]))
    _int32("path_lens", path_lens, (B_,))
    if workspace is None:
        workspace = new_cache_workspace(device)
    index = device.index
    _on_device(index, ("block_table", block_table), ("context_lens", context_lens),
               ("path", path), ("path_lens", path_lens), ("workspace", workspace))
    shape = pa_shape(B_, H_kv, H_kv, L, 128, P, ps, block_table.shape[1], dtype_id)
    lens = torch.empty_like(context_lens)
    _launch(name, index, fn, ctypes.byref(shape), *pools, block_table.data_ptr(),
            context_lens.data_ptr(), path.data_ptr(), path.shape[1], path_lens.data_ptr(),
            lens.data_ptr(), workspace.data_ptr(), workspace.numel())
    return lens


@_streamed
def compact_kv(key_pages, value_pages, block_table, context_lens, path, path_lens, L, *,
               workspace=None):
    """Keeps, of the L drafts behind each context, path[b, :path_lens[b]]
    (ascending; int32 [B, n] and [B]): their rows move in place right behind
    the positions before the drafts.  Returns the new lengths [B]."""
    dims = _pages_dims(key_pages, value_pages)
    if key_pages.shape[3] != 128:
        raise ValueError("head dim must be 128")
    return _compact("pa_compact_kv", (_lib or load()).pa_compact_kv,
                    (key_pages.data_ptr(), value_pages.data_ptr()), dims,
                    _dtype_id(key_pages.dtype), key_pages.device, block_table, context_lens, path,
                    path_lens, L, workspace)


@_streamed
def compact_kv_q4(pool, block_table, context_lens, path, path_lens, L, *, workspace=None):
    """compact_kv of a 4-bit pool."""
    return _compact("pa_compact_kv_q4", (_lib or load()).pa_compact_kv_q4,
                    (ctypes.byref(pool.c_pool),), pool.dims, PA_BF16, pool.device, block_table,
                    context_lens, path, path_lens, L, workspace)


# ---- pages shared between sequences ---------------------------------------------
def _pages_shape(block_table, page_refs, page_size):
    return pa_shape(block_table.shape[0], 1, 1, 1, 128, page_refs.shape[0], page_size,
                    block_table.shape[1], PA_BF16)


def _page_state(block_table, context_lens, page_refs, page_size):
    """The CUDA device index of a checked table, lengths, page counts and page
    size."""
    _c_int("page_size", page_size)
    _table(block_table, context_lens, block_table.shape[0])
    _int32("page_refs", page_refs, (page_refs.shape[0],))
    index = block_table.get_device()
    if index < 0:
        raise ValueError("block_table must be on a CUDA device")
    _on_device(index, ("block_table", block_table), ("context_lens", context_lens),
               ("page_refs", page_refs))
    return index


def new_pages_workspace(block_table, page_refs):
    """Workspace of resize_pages (and fork_pages, copy_pages) for tables of at
    most these rows and pools of at most these pages."""
    n = pa_pages_workspace_bytes(_pages_shape(block_table, page_refs, 1))
    return _workspace(n, block_table.device, "pa_pages_workspace_bytes")


@_streamed
def fork_pages(block_table, context_lens, page_refs, sources, targets, page_size, lens=None, *,
               workspace=None):
    """Row targets[i] of block_table becomes a fork of row sources[i] (int32
    [n]): the pages of its first lens[i] positions (None: all) are named twice
    and counted in page_refs (int32 [num_pages], 0: free); nothing is copied.
    Targets must be empty (length 0); no fork of a call may read a row that
    one of them names as its target.  Table, lengths and counts change in
    place."""
    index = _page_state(block_table, context_lens, page_refs, page_size)
    _int32("sources", sources, (sources.shape[0],))
    _int32("targets", targets, (sources.shape[0],))
    at = 0
    if lens is not None:
        _int32("lens", lens, (sources.shape[0],))
        _on_device(index, ("lens", lens))
        at = lens.data_ptr()
    if workspace is None:
        workspace = new_cache_workspace(block_table.device)
    _on_device(index, ("sources", sources), ("targets", targets), ("workspace", workspace))
    shape = _pages_shape(block_table, page_refs, page_size)
    _launch("pa_fork_pages", index, (_lib or load()).pa_fork_pages, ctypes.byref(shape),
            block_table.data_ptr(), context_lens.data_ptr(), page_refs.data_ptr(),
            sources.data_ptr(), targets.data_ptr(), at, sources.shape[0], workspace.data_ptr(),
            workspace.numel())
    return workspace


@_streamed
def resize_pages(block_table, context_lens, page_refs, new_lens, page_size, *, copies=None,
                 workspace=None):
    """Gives every sequence the length new_lens[b] (int32 [B]; negative: left
    alone, 0: freed), in place: pages past a new end go back, longer sequences
    get the lowest free pages and, where others hold their partly filled last
    page, one of their own for it.  Returns copies int32 [B, 3]: (old page, new
    page, rows) for copy_pages, which every layer's pool needs before it is
    written to, or (-1, -1, 0)."""
    torch = _torch or _load_torch()
    index = _page_state(block_table, context_lens, page_refs, page_size)
    B_ = block_table.shape[0]
    _int32("new_lens", new_lens, (B_,))
    if copies is None:
        copies = torch.empty((B_, 3), dtype=torch.int32, device=block_table.device)
    else:
        _int32("copies", copies, (B_, 3))
    if workspace is None:
        workspace = new_pages_workspace(block_table, page_refs)
    _on_device(index, ("new_lens", new_lens), ("copies", copies), ("workspace", workspace))
    shape = _pages_shape(block_table, page_refs, page_size)
    _launch("pa_resize_pages", index, (_lib or load()).pa_resize_pages, ctypes.byref(shape),
            block_table.data_ptr(), context_lens.data_ptr(), page_refs.data_ptr(),
            new_lens.data_ptr(), copies.data_ptr(), workspace.data_ptr(), workspace.numel())
    return copies


def _copy_pages(name, fn, pools, dims, dtype_id, device, copies, workspace):
    P, H_kv, ps = dims
    if copies.dim() != 2:
        raise ValueError("copies must be int32 [n, 3]")
    _int32("copies", copies, (copies.shape[0], 3))
    if workspace is None:
        workspace = new_cache_workspace(device)
    _on_device(device.index, ("copies", copies), ("workspace", workspace))
    shape = pa_shape(1, H_kv, H_kv, 1, 128, P, ps, 1, dtype_id)
    _launch(name, device.index, fn, ctypes.byref(shape), *pools, copies.data_ptr(),
            copies.shape[0], workspace.data_ptr(), workspace.numel())
    return workspace


@_streamed
def copy_pages(key_pages, value_pages, copies, *, workspace=None):
    """Carries out the copies (int32 [n, 3]: old page, new page, rows) of
    resize_pages in one layer's pages, in place."""
    dims = _pages_dims(key_pages, value_pages)
    if key_pages.shape[3] != 128:
        raise ValueError("head dim must be 128")
    return _copy_pages("pa_copy_pages", (_lib or load()).pa_copy_pages,
                       (key_pages.data_ptr(), value_pages.data_ptr()), dims,
                       _dtype_id(key_pages.dtype), key_pages.device, copies, workspace)


@_streamed
def copy_pages_q4(pool, copies, *, workspace=None):
    """copy_pages of a 4-bit pool."""
    return _copy_pages("pa_copy_pages_q4", (_lib or load()).pa_copy_pages_q4,
                       (ctypes.byref(pool.c_pool),), pool.dims, PA_BF16, pool.device, copies,
                       workspace)
