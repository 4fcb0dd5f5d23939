"""Python binding of libvarlen_attn (the C ABI in include/varlen_attn.h).

Argument marshalling only: torch tensors become device pointers and int64
(row, head) strides, streams become cudaStream_t handles.  Every step of the
computation runs in the library's CUDA kernels; there is no fallback.  If the
library is missing or cannot be loaded, importing this module raises.

The raw entry points keep the C names (``varlen_attn_fwd`` ...) and return
the C status code.  ``attention_fwd`` / ``attention_bwd`` are conveniences
that allocate outputs / workspace with torch on the inputs' device and raise
``VarlenError`` on a non-zero status.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.machinery
import importlib.util
import math
import os
import warnings

import torch

from . import build as _build

VARLEN_OK = 0
VARLEN_ERR_NULL = -1
VARLEN_ERR_SHAPE = -2
VARLEN_ERR_HEAD_DIM = -3
VARLEN_ERR_ALIGN = -4
VARLEN_ERR_STRIDE = -5
VARLEN_ERR_WORKSPACE = -6
VARLEN_ERR_CUDA = -7
VARLEN_ERR_TIMEOUT = -8
VARLEN_ERR_DEVICE_BOUNDS = -9
VARLEN_ERR_ARCH = -10


class VarlenStride(ctypes.Structure):
    _fields_ = [("row", ctypes.c_int64), ("head", ctypes.c_int64)]


class VarlenDenseStride(ctypes.Structure):
    """Batch, row and head strides of one [batch, seqlen, H, D] tensor, in elements."""
    _fields_ = [("batch", ctypes.c_int64), ("row", ctypes.c_int64), ("head", ctypes.c_int64)]


class VarlenPageStride(ctypes.Structure):
    """Page, row and head strides of one page array [num_pages, page_size, heads, D], in elements."""
    _fields_ = [("page", ctypes.c_int64), ("row", ctypes.c_int64), ("head", ctypes.c_int64)]


class VarlenKvCache(ctypes.Structure):
    """varlen_kv_cache of the C header."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("seqlens", ctypes.c_void_p),
                ("sk", VarlenPageStride), ("sv", VarlenPageStride), ("table_stride", ctypes.c_int64),
                ("type", ctypes.c_int32), ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class VarlenPagePool(ctypes.Structure):
    """varlen_page_pool of the C header."""
    _fields_ = [("block_table", ctypes.c_void_p), ("seqlens", ctypes.c_void_p), ("seqlens_out", ctypes.c_void_p),
                ("free_pages", ctypes.c_void_p), ("free_count", ctypes.c_void_p), ("free_count_out", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages", ctypes.c_int32)]


class VarlenRotary(ctypes.Structure):
    """varlen_rotary of the C header."""
    _fields_ = [("turns", ctypes.c_void_p), ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("scale", ctypes.c_float)]


VARLEN_CACHE_BF16 = 0
VARLEN_CACHE_E4M3 = 1


class VarlenError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = "%s failed: %d (%s)" % (where, status, varlen_attn_status_string(status))
        if status == VARLEN_ERR_CUDA:
            msg += ": " + varlen_attn_last_cuda_error()
        super().__init__(msg)
        self.status = status


def _load() -> ctypes.CDLL:
    path = os.environ.get("VARLEN_ATTN_LIB", _build.LIB)
    if not os.path.exists(path):
        raise ImportError("libvarlen_attn not built at %s: run __graft_entry__.build() or "
                          "python -m packed_variable_length_varlen_gb300.build" % path)
    lib = ctypes.CDLL(path)
    S = VarlenStride
    vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    lib.varlen_attn_fwd.restype = ctypes.c_int
    lib.varlen_attn_fwd.argtypes = [vp, S, vp, S, vp, S, vp, vp, i32, i32, i32, i32, i32, i32, i32, f32,
                                    vp, S, vp, vp]
    lib.varlen_attn_bwd_workspace_size.restype = sz
    lib.varlen_attn_bwd_workspace_size.argtypes = [i32, i32, i32, i32]
    lib.varlen_attn_bwd.restype = ctypes.c_int
    lib.varlen_attn_bwd.argtypes = [vp, S, vp, S, vp, S, vp, S, vp, S, vp, vp, vp, i32, i32, i32, i32, i32, i32,
                                    i32, f32, vp, S, vp, S, vp, S, vp, sz, vp]
    lib.varlen_attn_fwd_causal.restype = ctypes.c_int
    lib.varlen_attn_fwd_causal.argtypes = lib.varlen_attn_fwd.argtypes
    lib.varlen_attn_bwd_causal.restype = ctypes.c_int
    lib.varlen_attn_bwd_causal.argtypes = lib.varlen_attn_bwd.argtypes
    lib.varlen_attn_fwd_window.restype = ctypes.c_int
    lib.varlen_attn_fwd_window.argtypes = [vp, S, vp, S, vp, S, vp, vp, i32, i32, i32, i32, i32, i32, i32, f32,
                                           i32, i32, vp, S, vp, vp]
    lib.varlen_attn_bwd_window.restype = ctypes.c_int
    lib.varlen_attn_bwd_window.argtypes = [vp, S, vp, S, vp, S, vp, S, vp, S, vp, vp, vp, i32, i32, i32, i32, i32,
                                           i32, i32, f32, i32, i32, vp, S, vp, S, vp, S, vp, sz, vp]
    lib.varlen_attn_bwd_deterministic.restype = ctypes.c_int
    lib.varlen_attn_bwd_deterministic.argtypes = lib.varlen_attn_bwd_window.argtypes
    lib.varlen_attn_fwd_fp8_workspace_size.restype = sz
    lib.varlen_attn_fwd_fp8_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    lib.varlen_attn_fwd_fp8_workspace_layout.restype = ctypes.c_int
    lib.varlen_attn_fwd_fp8_workspace_layout.argtypes = [i32, i32, i32, i32, i32, vp, vp]
    lib.varlen_attn_fwd_fp8.restype = ctypes.c_int
    lib.varlen_attn_fwd_fp8.argtypes = [vp, S, vp, S, vp, S, vp, vp, i32, i32, i32, i32, i32, i32, i32, f32, vp, S,
                                        vp, vp, sz, vp]
    lib.varlen_attn_fwd_fp8_window.restype = ctypes.c_int
    lib.varlen_attn_fwd_fp8_window.argtypes = [vp, S, vp, S, vp, S, vp, vp, i32, i32, i32, i32, i32, i32, i32, f32,
                                               i32, i32, vp, S, vp, vp, sz, vp]
    DS = VarlenDenseStride
    lib.varlen_attn_fwd_fp8_dense_workspace_size.restype = sz
    lib.varlen_attn_fwd_fp8_dense_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    lib.varlen_attn_fwd_fp8_dense.restype = ctypes.c_int
    lib.varlen_attn_fwd_fp8_dense.argtypes = [vp, DS, vp, DS, vp, DS, i32, i32, i32, i32, i32, f32, i32, vp, DS, vp,
                                              vp, sz, vp]
    lib.varlen_attn_fwd_dense.restype = ctypes.c_int
    lib.varlen_attn_fwd_dense.argtypes = [vp, DS, vp, DS, vp, DS, i32, i32, i32, i32, i32, f32, i32, vp, DS, vp, vp]
    lib.varlen_attn_bwd_dense_workspace_size.restype = sz
    lib.varlen_attn_bwd_dense_workspace_size.argtypes = [i32, i32, i32, i32]
    lib.varlen_attn_bwd_dense.restype = ctypes.c_int
    lib.varlen_attn_bwd_dense.argtypes = [vp, DS, vp, DS, vp, DS, vp, DS, vp, DS, vp, i32, i32, i32, i32, i32, f32,
                                          i32, vp, DS, vp, DS, vp, DS, vp, sz, vp]
    lib.varlen_attn_cache_write.restype = ctypes.c_int
    lib.varlen_attn_cache_write.argtypes = [vp, S, vp, S, vp, i32, i32, vp, vp]
    lib.varlen_attn_cache_read.restype = ctypes.c_int
    lib.varlen_attn_cache_read.argtypes = [vp, vp, i32, i32, vp, S, vp, S, vp]
    lib.varlen_attn_fwd_paged_workspace_size.restype = sz
    lib.varlen_attn_fwd_paged_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    lib.varlen_attn_fwd_paged.restype = ctypes.c_int
    lib.varlen_attn_fwd_paged.argtypes = [vp, S, vp, i32, i32, i32, i32, vp, f32, i32, i32, vp, S, vp, vp, sz, vp]
    lib.varlen_attn_fwd_paged_tree.restype = ctypes.c_int
    lib.varlen_attn_fwd_paged_tree.argtypes = [vp, S, vp, i32, i32, i32, i32, vp, f32, vp, i32, vp, i32, vp, S, vp, vp, sz,
                                               vp]
    lib.varlen_attn_cache_plan_workspace_size.restype = sz
    lib.varlen_attn_cache_plan_workspace_size.argtypes = [i32]
    lib.varlen_attn_cache_plan.restype = ctypes.c_int
    lib.varlen_attn_cache_plan.argtypes = [vp, vp, i32, vp, i32, vp, vp, vp, vp, vp, i32, vp, sz, vp]
    lib.varlen_attn_cache_trim.restype = ctypes.c_int
    lib.varlen_attn_cache_trim.argtypes = [vp, vp, vp, i32, vp]
    lib.varlen_attn_cache_move.restype = ctypes.c_int
    lib.varlen_attn_cache_move.argtypes = [vp, i32, vp, i32, i32, vp, i64, vp, i32, vp]
    lib.varlen_attn_rotary_turns.restype = ctypes.c_int
    lib.varlen_attn_rotary_turns.argtypes = [vp, i32, vp]
    lib.varlen_attn_rotary.restype = ctypes.c_int
    lib.varlen_attn_rotary.argtypes = [vp, S, vp, S, vp, vp, i32, i32, i32, i32, i32, vp, i32, vp, S, vp, S, vp]
    lib.varlen_attn_rotary_cache_write.restype = ctypes.c_int
    lib.varlen_attn_rotary_cache_write.argtypes = [vp, S, vp, S, vp, S, vp, vp, i32, i32, vp, vp, vp, S, vp]
    lib.varlen_attn_bwd_noalloc.restype = ctypes.c_int
    lib.varlen_attn_bwd_noalloc.argtypes = [vp, S, vp, S, vp, S, vp, S, vp, S, vp, vp, vp, i32, i32, i32, i32, i32,
                                            i32, i32, f32, vp, S, vp, S, vp, S, vp]
    lib.varlen_attn_bwd_noalloc_scratch_bytes.restype = sz
    lib.varlen_attn_bwd_noalloc_scratch_bytes.argtypes = []
    lib.varlen_attn_debug_noalloc_scratch.restype = ctypes.c_int
    lib.varlen_attn_debug_noalloc_scratch.argtypes = [vp, vp]
    lib.varlen_attn_bounds_checked.restype = ctypes.c_int
    lib.varlen_attn_bounds_checked.argtypes = []
    lib.varlen_attn_debug_set_span_slack.restype = ctypes.c_int
    lib.varlen_attn_debug_set_span_slack.argtypes = [i64]
    lib.varlen_attn_debug_skip_load.restype = ctypes.c_int
    lib.varlen_attn_debug_skip_load.argtypes = [ctypes.c_int, i64]
    lib.varlen_attn_get_device_status.restype = ctypes.c_int
    lib.varlen_attn_get_device_status.argtypes = [vp]
    lib.varlen_attn_status_string.restype = ctypes.c_char_p
    lib.varlen_attn_status_string.argtypes = [ctypes.c_int]
    lib.varlen_attn_last_cuda_error.restype = ctypes.c_char_p
    lib.varlen_attn_last_cuda_error.argtypes = []
    lib.varlen_attn_tile_count.restype = i64
    lib.varlen_attn_tile_count.argtypes = [vp, i32, i32, i32, i32]
    lib.varlen_attn_debug_schedule.restype = ctypes.c_int
    lib.varlen_attn_debug_schedule.argtypes = [vp, i32, i32, i32, i32, i32, vp, i64, vp]
    lib.varlen_attn_selftest_wait_timeout.restype = ctypes.c_int
    lib.varlen_attn_selftest_wait_timeout.argtypes = [ctypes.c_uint64, vp]
    lib.varlen_attn_debug_mma_cycles.restype = ctypes.c_int
    lib.varlen_attn_debug_mma_cycles.argtypes = [i32, i32, i32, vp, vp]
    lib.varlen_attn_debug_set_phase_events.restype = ctypes.c_int
    lib.varlen_attn_debug_set_phase_events.argtypes = [vp, ctypes.c_int]
    lib.varlen_attn_num_sms.restype = ctypes.c_int
    lib.varlen_attn_num_sms.argtypes = []
    return lib


def _load_binding(lib):
    """The native binding (csrc/varlen_binding.cpp) over the library's functions, or None: then every call goes by
    ctypes, with the same results.  One that was built for another header than the library is not loaded."""
    if not _build.binding_built(lib._name):
        return None
    try:
        loader = importlib.machinery.ExtensionFileLoader("_varlen_binding", _build.BINDING)
        native = importlib.util.module_from_spec(importlib.util.spec_from_loader("_varlen_binding", loader))
        loader.exec_module(native)
    except ImportError as e:
        warnings.warn("small calls go by ctypes: %s cannot be loaded (%s)" % (_build.BINDING, e))
        return None
    native.bind(*(ctypes.cast(getattr(lib, "varlen_attn_" + name), ctypes.c_void_p).value
                  for name in ("rotary", "rotary_cache_write", "cache_plan", "cache_trim", "cache_move", "fwd_paged_tree",
                               "fwd_paged_workspace_size")))
    return native


LIB = _load()
LIB_PATH = LIB._name
NATIVE = _load_binding(LIB)

EXPORTED = ("varlen_attn_fwd", "varlen_attn_bwd_workspace_size", "varlen_attn_bwd",
            "varlen_attn_get_device_status", "varlen_attn_status_string", "varlen_attn_tile_count",
            "varlen_attn_debug_schedule", "varlen_attn_selftest_wait_timeout", "varlen_attn_num_sms",
            "varlen_attn_debug_set_phase_events", "varlen_attn_bwd_noalloc", "varlen_attn_last_cuda_error",
            "varlen_attn_fwd_causal", "varlen_attn_bwd_causal", "varlen_attn_fwd_dense",
            "varlen_attn_bwd_dense_workspace_size", "varlen_attn_bwd_dense", "varlen_attn_fwd_window",
            "varlen_attn_bwd_window", "varlen_attn_bwd_deterministic", "varlen_attn_fwd_fp8_workspace_size",
            "varlen_attn_fwd_fp8_workspace_layout", "varlen_attn_fwd_fp8", "varlen_attn_bwd_noalloc_scratch_bytes",
            "varlen_attn_debug_noalloc_scratch", "varlen_attn_bounds_checked", "varlen_attn_debug_set_span_slack",
            "varlen_attn_debug_skip_load", "varlen_attn_debug_mma_cycles", "varlen_attn_fwd_fp8_window",
            "varlen_attn_fwd_fp8_dense_workspace_size", "varlen_attn_fwd_fp8_dense", "varlen_attn_cache_write",
            "varlen_attn_cache_read", "varlen_attn_fwd_paged_workspace_size", "varlen_attn_fwd_paged",
            "varlen_attn_fwd_paged_tree", "varlen_attn_cache_plan_workspace_size", "varlen_attn_cache_plan",
            "varlen_attn_cache_trim", "varlen_attn_cache_move", "varlen_attn_rotary_turns", "varlen_attn_rotary",
            "varlen_attn_rotary_cache_write")

# Size of the fixed device array varlen_attn_bwd_noalloc uses as scratch, as
# compiled into the library.
NOALLOC_SCRATCH_BYTES = int(LIB.varlen_attn_bwd_noalloc_scratch_bytes())


# ---------------------------------------------------------------- marshalling

def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stride(t) -> VarlenStride:
    if t is None:
        return VarlenStride(0, 0)
    if t.dim() != 3 or t.stride(2) != 1:
        raise ValueError("NHD tensors must be [rows, heads, head_dim] with unit innermost stride")
    return VarlenStride(t.stride(0), t.stride(1))


def _dstride(t) -> VarlenDenseStride:
    if t is None:
        return VarlenDenseStride(0, 0, 0)
    if t.dim() != 4 or t.stride(3) != 1:
        raise ValueError("dense tensors must be [batch, seqlen, heads, head_dim] with unit innermost stride")
    return VarlenDenseStride(t.stride(0), t.stride(1), t.stride(2))


def _ref(struct):
    return None if struct is None else ctypes.byref(struct)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    return ctypes.c_void_p(int(stream))


# ---------------------------------------------------------------- raw ABI

def _band(causal, window):
    """(left, right) of the window entry points for `causal` / `window`
    (causal sets right = 0), or None when neither masks anything."""
    left, right = int(window[0]), int(window[1])
    if causal:
        right = 0
    if left < 0 and right < 0:
        return None
    return max(left, -1), max(right, -1)


def varlen_attn_fwd(q, k, v, cu_seqlens_q, cu_seqlens_k, batch, total_q, total_k, num_heads, head_dim,
                    max_seqlen_q, max_seqlen_k, scale, out, lse, stream=None, causal=False, window=(-1, -1)) -> int:
    band = _band(causal, window)
    head = (_ptr(q), _stride(q), _ptr(k), _stride(k), _ptr(v), _stride(v), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
            batch, total_q, total_k, num_heads, head_dim, max_seqlen_q, max_seqlen_k, scale)
    tail = (_ptr(out), _stride(out), _ptr(lse), _stream(stream))
    if band is None:
        return LIB.varlen_attn_fwd(*head, *tail)
    if band == (-1, 0):
        return LIB.varlen_attn_fwd_causal(*head, *tail)
    return LIB.varlen_attn_fwd_window(*head, *band, *tail)


def varlen_attn_fwd_window(q, k, v, cu_seqlens_q, cu_seqlens_k, batch, total_q, total_k, num_heads, head_dim,
                           max_seqlen_q, max_seqlen_k, scale, window_left, window_right, out, lse,
                           stream=None) -> int:
    return LIB.varlen_attn_fwd_window(_ptr(q), _stride(q), _ptr(k), _stride(k), _ptr(v), _stride(v),
                                      _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), batch, total_q, total_k, num_heads,
                                      head_dim, max_seqlen_q, max_seqlen_k, scale, window_left, window_right,
                                      _ptr(out), _stride(out), _ptr(lse), _stream(stream))


def varlen_attn_fwd_causal(q, k, v, cu_seqlens_q, cu_seqlens_k, batch, total_q, total_k, num_heads, head_dim,
                           max_seqlen_q, max_seqlen_k, scale, out, lse, stream=None) -> int:
    return varlen_attn_fwd(q, k, v, cu_seqlens_q, cu_seqlens_k, batch, total_q, total_k, num_heads, head_dim,
                           max_seqlen_q, max_seqlen_k, scale, out, lse, stream, causal=True)


def varlen_attn_bwd_workspace_size(batch, total_q, num_heads, head_dim) -> int:
    return int(LIB.varlen_attn_bwd_workspace_size(batch, total_q, num_heads, head_dim))


def varlen_attn_bwd(q, k, v, out, dout, lse, cu_seqlens_q, cu_seqlens_k, batch, total_q, total_k, num_heads,
                    head_dim, max_seqlen_q, max_seqlen_k, scale, dq, dk, dv, workspace, workspace_bytes,
                    stream=None, causal=False, window=(-1, -1), deterministic=False) -> int:
    band = _band(causal, window)
    head = (_ptr(q), _stride(q), _ptr(k), _stride(k), _ptr(v), _stride(v), _ptr(out), _stride(out), _ptr(dout),
            _stride(dout), _ptr(lse), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), batch, total_q, total_k, num_heads,
            head_dim, max_seqlen_q, max_seqlen_k, scale)
    tail = (_ptr(dq), _stride(dq), _ptr(dk), _stride(dk), _ptr(dv), _stride(dv), _ptr(workspace), workspace_bytes,
            _stream(stream))
    if deterministic:
        return LIB.varlen_attn_bwd_deterministic(*head, *(band or (-1, -1)), *tail)
    if band is None:
        return LIB.varlen_attn_bwd(*head, *tail)
    if band == (-1, 0):
        return LIB.varlen_attn_bwd_causal(*head, *tail)
    return LIB.varlen_attn_bwd_window(*head, *band, *tail)


def varlen_attn_bwd_window(q, k, v, out, dout, lse, cu_seqlens_q, cu_seqlens_k, batch, total_q, total_k,
                           num_heads, head_dim, max_seqlen_q, max_seqlen_k, scale, window_left, window_right, dq, dk,
                           dv, workspace, workspace_bytes, stream=None) -> int:
    return LIB.varlen_attn_bwd_window(_ptr(q), _stride(q), _ptr(k), _stride(k), _ptr(v), _stride(v), _ptr(out),
                                      _stride(out), _ptr(dout), _stride(dout), _ptr(lse), _ptr(cu_seqlens_q),
                                      _ptr(cu_seqlens_k), batch, total_q, total_k, num_heads, head_dim,
                                      max_seqlen_q, max_seqlen_k, scale, window_left, window_right, _ptr(dq),
                                      _stride(dq), _ptr(dk), _stride(dk), _ptr(dv), _stride(dv), _ptr(workspace),
                                      workspace_bytes, _stream(stream))


def varlen_attn_bwd_causal(q, k, v, out, dout, lse, cu_seqlens_q, cu_seqlens_k, batch, total_q, total_k,
                           num_heads, head_dim, max_seqlen_q, max_seqlen_k, scale, dq, dk, dv, workspace,
                           workspace_bytes, stream=None) -> int:
    return varlen_attn_bwd(q, k, v, out, dout, lse, cu_seqlens_q, cu_seqlens_k, batch, total_q, total_k,
                           num_heads, head_dim, max_seqlen_q, max_seqlen_k, scale, dq, dk, dv, workspace,
                           workspace_bytes, stream, causal=True)


def varlen_attn_fwd_fp8_workspace_size(batch, total_q, total_k, num_heads, head_dim) -> int:
    return int(LIB.varlen_attn_fwd_fp8_workspace_size(batch, total_q, total_k, num_heads, head_dim))


def varlen_attn_fwd_fp8_workspace_layout(batch, total_q, total_k, num_heads, head_dim):
    """(status, [amax, q codes, k codes, V^T codes] byte offsets, V^T row length)."""
    off = (ctypes.c_size_t * 4)()
    cols = ctypes.c_int64()
    st = LIB.varlen_attn_fwd_fp8_workspace_layout(batch, total_q, total_k, num_heads, head_dim,
                                                  ctypes.addressof(off), ctypes.addressof(cols))
    return st, list(off), int(cols.value)


def varlen_attn_fwd_fp8(q, k, v, cu_seqlens_q, cu_seqlens_k, batch, total_q, total_k, num_heads, head_dim,
                        max_seqlen_q, max_seqlen_k, scale, out, lse, workspace, workspace_bytes, stream=None,
                        causal=False, window=(-1, -1)) -> int:
    band = _band(causal, window)
    head = (_ptr(q), _stride(q), _ptr(k), _stride(k), _ptr(v), _stride(v), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
            batch, total_q, total_k, num_heads, head_dim, max_seqlen_q, max_seqlen_k, scale)
    tail = (_ptr(out), _stride(out), _ptr(lse), _ptr(workspace), workspace_bytes, _stream(stream))
    if band is None:
        return LIB.varlen_attn_fwd_fp8(*head, *tail)
    return LIB.varlen_attn_fwd_fp8_window(*head, *band, *tail)


def varlen_attn_fwd_fp8_window(q, k, v, cu_seqlens_q, cu_seqlens_k, batch, total_q, total_k, num_heads, head_dim,
                               max_seqlen_q, max_seqlen_k, scale, window_left, window_right, out, lse, workspace,
                               workspace_bytes, stream=None) -> int:
    return LIB.varlen_attn_fwd_fp8_window(_ptr(q), _stride(q), _ptr(k), _stride(k), _ptr(v), _stride(v),
                                          _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), batch, total_q, total_k, num_heads,
                                          head_dim, max_seqlen_q, max_seqlen_k, scale, window_left, window_right,
                                          _ptr(out), _stride(out), _ptr(lse), _ptr(workspace), workspace_bytes,
                                          _stream(stream))


def varlen_attn_fwd_fp8_dense_workspace_size(batch, seqlen_q, seqlen_k, num_heads, head_dim) -> int:
    return int(LIB.varlen_attn_fwd_fp8_dense_workspace_size(batch, seqlen_q, seqlen_k, num_heads, head_dim))


def varlen_attn_fwd_fp8_dense(q, k, v, batch, seqlen_q, seqlen_k, num_heads, head_dim, scale, causal, out, lse,
                              workspace, workspace_bytes, stream=None) -> int:
    return LIB.varlen_attn_fwd_fp8_dense(_ptr(q), _dstride(q), _ptr(k), _dstride(k), _ptr(v), _dstride(v), batch,
                                         seqlen_q, seqlen_k, num_heads, head_dim, scale, int(bool(causal)), _ptr(out),
                                         _dstride(out), _ptr(lse), _ptr(workspace), workspace_bytes,
                                         _stream(stream))


def varlen_attn_fwd_dense(q, k, v, batch, seqlen_q, seqlen_k, num_heads, head_dim, scale, causal, out, lse,
                          stream=None) -> int:
    return LIB.varlen_attn_fwd_dense(_ptr(q), _dstride(q), _ptr(k), _dstride(k), _ptr(v), _dstride(v), batch,
                                     seqlen_q, seqlen_k, num_heads, head_dim, scale, int(bool(causal)), _ptr(out),
                                     _dstride(out), _ptr(lse), _stream(stream))


def varlen_attn_bwd_dense_workspace_size(batch, seqlen_q, num_heads, head_dim) -> int:
    return int(LIB.varlen_attn_bwd_dense_workspace_size(batch, seqlen_q, num_heads, head_dim))


def varlen_attn_bwd_dense(q, k, v, out, dout, lse, batch, seqlen_q, seqlen_k, num_heads, head_dim, scale, causal,
                          dq, dk, dv, workspace, workspace_bytes, stream=None) -> int:
    return LIB.varlen_attn_bwd_dense(_ptr(q), _dstride(q), _ptr(k), _dstride(k), _ptr(v), _dstride(v), _ptr(out),
                                     _dstride(out), _ptr(dout), _dstride(dout), _ptr(lse), batch, seqlen_q, seqlen_k,
                                     num_heads, head_dim, scale, int(bool(causal)), _ptr(dq), _dstride(dq), _ptr(dk),
                                     _dstride(dk), _ptr(dv), _dstride(dv), _ptr(workspace), workspace_bytes,
                                     _stream(stream))


def varlen_attn_bwd_noalloc(q, k, v, out, dout, lse, cu_seqlens_q, cu_seqlens_k, batch, total_q, total_k,
                            num_heads, head_dim, max_seqlen_q, max_seqlen_k, scale, dq, dk, dv, stream=None) -> int:
    """The backward for callers that cannot allocate device memory: scratch
    comes from a fixed library-owned device array (see the C header)."""
    return LIB.varlen_attn_bwd_noalloc(_ptr(q), _stride(q), _ptr(k), _stride(k), _ptr(v), _stride(v), _ptr(out),
                                       _stride(out), _ptr(dout), _stride(dout), _ptr(lse), _ptr(cu_seqlens_q),
                                       _ptr(cu_seqlens_k), batch, total_q, total_k, num_heads, head_dim,
                                       max_seqlen_q, max_seqlen_k, scale, _ptr(dq), _stride(dq), _ptr(dk),
                                       _stride(dk), _ptr(dv), _stride(dv), _stream(stream))


def varlen_attn_cache_write(k, v, cu_seqlens, batch, total, cache, stream=None) -> int:
    """cache: a VarlenKvCache (PagedCache.struct), or None."""
    return LIB.varlen_attn_cache_write(_ptr(k), _stride(k), _ptr(v), _stride(v), _ptr(cu_seqlens), batch, total,
                                       _ref(cache), _stream(stream))


def varlen_attn_cache_read(cache, cu_seqlens, batch, total, k, v, stream=None) -> int:
    return LIB.varlen_attn_cache_read(_ref(cache), _ptr(cu_seqlens), batch, total, _ptr(k), _stride(k), _ptr(v),
                                      _stride(v), _stream(stream))


def varlen_attn_fwd_paged_workspace_size(batch, total_q, num_heads, num_kv_heads, head_dim) -> int:
    return int(LIB.varlen_attn_fwd_paged_workspace_size(batch, total_q, num_heads, num_kv_heads, head_dim))


def varlen_attn_fwd_paged(q, cu_seqlens_q, batch, total_q, num_heads, max_seqlen_q, cache, scale, window_left,
                          window_right, out, lse, workspace, workspace_bytes, stream=None) -> int:
    return LIB.varlen_attn_fwd_paged(_ptr(q), _stride(q), _ptr(cu_seqlens_q), batch, total_q, num_heads,
                                     max_seqlen_q, _ref(cache), scale, window_left, window_right, _ptr(out),
                                     _stride(out), _ptr(lse), _ptr(workspace), workspace_bytes, _stream(stream))


def varlen_attn_fwd_paged_tree(q, cu_seqlens_q, batch, total_q, num_heads, max_seqlen_q, cache, scale, masks, mask_words,
                               positions, window_left, out, lse, workspace, workspace_bytes, stream=None) -> int:
    return LIB.varlen_attn_fwd_paged_tree(_ptr(q), _stride(q), _ptr(cu_seqlens_q), batch, total_q, num_heads,
                                          max_seqlen_q, _ref(cache), scale, _ptr(masks), mask_words, _ptr(positions),
                                          window_left, _ptr(out), _stride(out), _ptr(lse), _ptr(workspace),
                                          workspace_bytes, _stream(stream))


def varlen_attn_cache_plan_workspace_size(batch) -> int:
    return int(LIB.varlen_attn_cache_plan_workspace_size(batch))


def varlen_attn_cache_plan(pool, new_lens, batch, parents, total, cu_seqlens, slots, positions, unplaced, masks,
                           mask_words, workspace, workspace_bytes, stream=None) -> int:
    """pool: a VarlenPagePool (PagePool.struct), or None."""
    return LIB.varlen_attn_cache_plan(_ref(pool), _ptr(new_lens), batch, _ptr(parents), total, _ptr(cu_seqlens),
                                      _ptr(slots), _ptr(positions), _ptr(unplaced), _ptr(masks), mask_words,
                                      _ptr(workspace), workspace_bytes, _stream(stream))


def varlen_attn_cache_trim(pool, lens, cu_seqlens, batch, stream=None) -> int:
    return LIB.varlen_attn_cache_trim(_ref(pool), _ptr(lens), _ptr(cu_seqlens), batch, _stream(stream))


def varlen_attn_cache_move(caches, cu_seqlens, batch, total, kept, kept_stride, kept_lens, max_kept, stream=None) -> int:
    """caches: VarlenKvCache structs."""
    arr = (VarlenKvCache * len(caches))(*caches)
    return LIB.varlen_attn_cache_move(arr, len(caches), _ptr(cu_seqlens), batch, total, _ptr(kept), kept_stride,
                                      _ptr(kept_lens), max_kept, _stream(stream))


def varlen_attn_rotary_turns(frequencies):
    """(status, turns): frequencies in radians a position as whole 2^-64 turns."""
    n = len(frequencies)
    turns = (ctypes.c_uint64 * max(n, 1))()
    st = LIB.varlen_attn_rotary_turns((ctypes.c_double * max(n, 1))(*frequencies), n, turns)
    return st, list(turns)[:n]


def varlen_attn_rotary(q, k, positions, cu_seqlens, batch, total, num_heads, num_kv_heads, head_dim, rotary, inverse,
                       q_out, k_out, stream=None) -> int:
    """rotary: a VarlenRotary (Rotary.struct), or None."""
    return LIB.varlen_attn_rotary(_ptr(q), _stride(q), _ptr(k), _stride(k), _ptr(positions), _ptr(cu_seqlens), batch,
                                  total, num_heads, num_kv_heads, head_dim, _ref(rotary), int(bool(inverse)), _ptr(q_out),
                                  _stride(q_out), _ptr(k_out), _stride(k_out), _stream(stream))


def varlen_attn_rotary_cache_write(q, k, v, positions, slots, total, num_heads, cache, rotary, q_out, stream=None) -> int:
    return LIB.varlen_attn_rotary_cache_write(_ptr(q), _stride(q), _ptr(k), _stride(k), _ptr(v), _stride(v),
                                              _ptr(positions), _ptr(slots), total, num_heads, _ref(cache), _ref(rotary),
                                              _ptr(q_out), _stride(q_out), _stream(stream))


def varlen_attn_debug_noalloc_scratch():
    """(status, scratch device address, context id) that the next
    varlen_attn_bwd_noalloc call on this thread would use; launches nothing."""
    addr = ctypes.c_void_p(0)
    ctx = ctypes.c_ulonglong(0)
    st = LIB.varlen_attn_debug_noalloc_scratch(ctypes.byref(addr), ctypes.byref(ctx))
    return st, int(addr.value or 0), int(ctx.value)


def varlen_attn_bounds_checked() -> bool:
    """True for a library built with device-side bounds checks."""
    return bool(LIB.varlen_attn_bounds_checked())


def varlen_attn_debug_set_span_slack(nbytes: int) -> int:
    return LIB.varlen_attn_debug_set_span_slack(int(nbytes))


def varlen_attn_debug_skip_load(which: int, n: int) -> int:
    return LIB.varlen_attn_debug_skip_load(int(which), int(n))


def varlen_attn_get_device_status(stream=None) -> int:
    return LIB.varlen_attn_get_device_status(_stream(stream))


def varlen_attn_status_string(status: int) -> str:
    return LIB.varlen_attn_status_string(status).decode()


def varlen_attn_last_cuda_error() -> str:
    return LIB.varlen_attn_last_cuda_error().decode()


def varlen_attn_tile_count(cu_seqlens_host, batch, total, num_heads, tile) -> int:
    cu = torch.as_tensor(cu_seqlens_host, dtype=torch.int32).contiguous()
    return int(LIB.varlen_attn_tile_count(ctypes.c_void_p(cu.data_ptr()), batch, total, num_heads, tile))


def varlen_attn_debug_schedule(cu_seqlens, batch, total, num_heads, tile, grid, out_records, max_records,
                               stream=None) -> int:
    return LIB.varlen_attn_debug_schedule(_ptr(cu_seqlens), batch, total, num_heads, tile, grid,
                                          _ptr(out_records), max_records, _stream(stream))


def varlen_attn_selftest_wait_timeout(budget_ns: int, stream=None) -> int:
    return LIB.varlen_attn_selftest_wait_timeout(budget_ns, _stream(stream))


def varlen_attn_debug_mma_cycles(n_mma, n_cols, mode, cycles, stream=None) -> int:
    """cycles: a CUDA int64 tensor (one element) that receives the count."""
    return LIB.varlen_attn_debug_mma_cycles(n_mma, n_cols, mode, _ptr(cycles), _stream(stream))


_PHASE_KEEP = None


def varlen_attn_debug_set_phase_events(events) -> int:
    """events: four torch.cuda.Event(enable_timing=True) objects, or None."""
    global _PHASE_KEEP
    if not events:
        _PHASE_KEEP = None
        return LIB.varlen_attn_debug_set_phase_events(None, 0)
    for e in events:
        e.record()  # materialise the handle on the current device
    arr = (ctypes.c_void_p * 4)(*[e.cuda_event for e in events])
    _PHASE_KEEP = (events, arr)
    return LIB.varlen_attn_debug_set_phase_events(arr, 4)


def varlen_attn_num_sms() -> int:
    return LIB.varlen_attn_num_sms()


# ---------------------------------------------------------------- conveniences

def _check(status, where):
    if status != VARLEN_OK:
        raise VarlenError(status, where)


def attention_fwd(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q=0, max_seqlen_k=0, scale=None,
                  out=None, lse=None, stream=None, causal=False, window=(-1, -1)):
    """O and LSE for packed q/k/v ([rows, H, D] bf16 on one CUDA device);
    `causal` / `window` = (left, right) select the masked entry points
    (causal sets right = 0; a negative side is unbounded)."""
    total_q, H, D = q.shape
    total_k = k.shape[0]
    batch = cu_seqlens_q.numel() - 1
    scale = float(D ** -0.5) if scale is None else float(scale)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if lse is None:
        lse = torch.empty(H, total_q, dtype=torch.float32, device=q.device)
    _check(varlen_attn_fwd(q, k, v, cu_seqlens_q, cu_seqlens_k, batch, total_q, total_k, H, D, max_seqlen_q,
                           max_seqlen_k, scale, out, lse, stream, causal, window), "varlen_attn_fwd")
    return out, lse


def attention_fwd_fp8(q, k, v, cu_seqlens_q, cu_seqlens_k, scale=None, out=None, lse=None, workspace=None,
                      stream=None, causal=False, window=(-1, -1)):
    """E4M3 forward of packed bf16 q/k/v ([rows, H, 128]): quantised per
    (segment, head) into `workspace` (allocated when None), O in bf16 and
    LSE, optionally under a causal or sliding-window band.  Returns (out,
    lse, workspace)."""
    total_q, H, D = q.shape
    total_k = k.shape[0]
    batch = cu_seqlens_q.numel() - 1
    scale = float(D ** -0.5) if scale is None else float(scale)
    nbytes = varlen_attn_fwd_fp8_workspace_size(batch, total_q, total_k, H, D)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if lse is None:
        lse = torch.empty(H, total_q, dtype=torch.float32, device=q.device)
    _check(varlen_attn_fwd_fp8(q, k, v, cu_seqlens_q, cu_seqlens_k, batch, total_q, total_k, H, D, 0, 0, scale, out,
                               lse, workspace, workspace.numel(), stream, causal, window), "varlen_attn_fwd_fp8")
    return out, lse, workspace


def attention_bwd(q, k, v, out, dout, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q=0, max_seqlen_k=0,
                  scale=None, dq=None, dk=None, dv=None, workspace=None, stream=None, causal=False,
                  window=(-1, -1), deterministic=False):
    """dQ, dK, dV for the forward above (every operand keeps its strides)."""
    total_q, H, D = q.shape
    total_k = k.shape[0]
    batch = cu_seqlens_q.numel() - 1
    scale = float(D ** -0.5) if scale is None else float(scale)
    dq = torch.empty_like(q, memory_format=torch.contiguous_format) if dq is None else dq
    dk = torch.empty_like(k, memory_format=torch.contiguous_format) if dk is None else dk
    dv = torch.empty_like(v, memory_format=torch.contiguous_format) if dv is None else dv
    nbytes = varlen_attn_bwd_workspace_size(batch, total_q, H, D)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    _check(varlen_attn_bwd(q, k, v, out, dout, lse, cu_seqlens_q, cu_seqlens_k, batch, total_q, total_k, H, D,
                           max_seqlen_q, max_seqlen_k, scale, dq, dk, dv, workspace, workspace.numel(), stream,
                           causal, window, deterministic), "varlen_attn_bwd")
    return dq, dk, dv


def attention_fwd_dense(q, k, v, scale=None, causal=False, out=None, lse=None, stream=None):
    """O and LSE for dense batched q [B, Sq, H, D], k / v [B, Sk, H, D] (bf16,
    one CUDA device); lse is [H, B * Sq]."""
    B, Sq, H, D = q.shape
    Sk = k.shape[1]
    scale = float(D ** -0.5) if scale is None else float(scale)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if lse is None:
        lse = torch.empty(H, B * Sq, dtype=torch.float32, device=q.device)
    _check(varlen_attn_fwd_dense(q, k, v, B, Sq, Sk, H, D, scale, causal, out, lse, stream), "varlen_attn_fwd_dense")
    return out, lse


def attention_fwd_fp8_dense(q, k, v, scale=None, causal=False, out=None, lse=None, workspace=None, stream=None):
    """E4M3 forward of dense batched bf16 q [B, Sq, H, 128], k / v
    [B, Sk, H, 128]: quantised per (batch entry, head) into `workspace`
    (allocated when None); returns (out, lse [H, B * Sq], workspace)."""
    B, Sq, H, D = q.shape
    Sk = k.shape[1]
    scale = float(D ** -0.5) if scale is None else float(scale)
    nbytes = varlen_attn_fwd_fp8_dense_workspace_size(B, Sq, Sk, H, D)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if lse is None:
        lse = torch.empty(H, B * Sq, dtype=torch.float32, device=q.device)
    _check(varlen_attn_fwd_fp8_dense(q, k, v, B, Sq, Sk, H, D, scale, causal, out, lse, workspace,
                                     workspace.numel(), stream), "varlen_attn_fwd_fp8_dense")
    return out, lse, workspace


def attention_bwd_dense(q, k, v, out, dout, lse, scale=None, causal=False, dq=None, dk=None, dv=None,
                        workspace=None, stream=None):
    """dQ, dK, dV for attention_fwd_dense."""
    B, Sq, H, D = q.shape
    Sk = k.shape[1]
    scale = float(D ** -0.5) if scale is None else float(scale)
    dq = torch.empty_like(q, memory_format=torch.contiguous_format) if dq is None else dq
    dk = torch.empty_like(k, memory_format=torch.contiguous_format) if dk is None else dk
    dv = torch.empty_like(v, memory_format=torch.contiguous_format) if dv is None else dv
    nbytes = varlen_attn_bwd_dense_workspace_size(B, Sq, H, D)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    _check(varlen_attn_bwd_dense(q, k, v, out, dout, lse, B, Sq, Sk, H, D, scale, causal, dq, dk, dv, workspace,
                                 workspace.numel(), stream), "varlen_attn_bwd_dense")
    return dq, dk, dv


# ---------------------------------------------------------------- paged cache

class PagedCache:
    """A paged key/value cache: the tensors a program keeps, checked once.

    k_pages / v_pages  [num_pages, page_size, num_kv_heads, D], bf16 or
                       float8_e4m3fn, unit innermost stride
    block_table        [batch, max_pages] int32: page of each page_size positions
    seqlens            [batch] int32: positions each sequence holds
    k_scale / v_scale  E4M3 only: bf16 [num_pages, num_kv_heads, page_size],
                       contiguous

    The tensors are kept, not copied: what a program writes into them (a new
    page in the table, longer seqlens) is seen by later calls.  ``struct`` is
    the C description of them: their addresses, so they stay where they are
    (no resize_ or set_), and another tensor in the place of one is refused.
    """

    def __init__(self, k_pages, v_pages, block_table, seqlens, k_scale=None, v_scale=None):
        if k_pages.dim() != 4 or k_pages.shape != v_pages.shape or k_pages.dtype != v_pages.dtype:
            raise ValueError("k_pages and v_pages must be [num_pages, page_size, heads, head_dim] of one type")
        if k_pages.stride(3) != 1 or v_pages.stride(3) != 1:
            raise ValueError("pages must have a unit innermost stride")
        if k_pages.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise ValueError("pages must be bfloat16 or float8_e4m3fn")
        e4m3 = k_pages.dtype == torch.float8_e4m3fn
        pages, page_size, heads, dim = k_pages.shape
        if block_table.dim() != 2 or block_table.dtype != torch.int32 or (block_table.shape[1] > 1
                                                                          and block_table.stride(1) != 1):
            raise ValueError("block_table must be int32 [batch, max_pages] with unit innermost stride")
        if seqlens.dtype != torch.int32 or seqlens.dim() != 1 or not seqlens.is_contiguous() \
                or seqlens.shape[0] != block_table.shape[0]:
            raise ValueError("seqlens must be contiguous int32 [batch]")
        for s in (k_scale, v_scale):
            if (s is not None) != e4m3:
                raise ValueError("E4M3 pages need k_scale and v_scale, bf16 pages take none")
            if e4m3 and (s.dtype != torch.bfloat16 or tuple(s.shape) != (pages, heads, page_size)
                         or not s.is_contiguous()):
                raise ValueError("scales must be contiguous bfloat16 [num_pages, heads, page_size]")
        self.tensors = [t for t in (k_pages, v_pages, block_table, seqlens, k_scale, v_scale) if t is not None]
        if any(t.device != k_pages.device for t in self.tensors):
            raise ValueError("the cache's tensors must be on one device")
        self.k_pages, self.v_pages, self.block_table, self.seqlens = k_pages, v_pages, block_table, seqlens
        self.k_scale, self.v_scale = k_scale, v_scale
        self.device, self.batch, self.num_kv_heads, self.head_dim = k_pages.device, seqlens.shape[0], heads, dim
        c = VarlenKvCache()
        c.k, c.v, c.block_table, c.seqlens = (t.data_ptr() for t in (k_pages, v_pages, block_table, seqlens))
        if e4m3:
            c.k_scale, c.v_scale = k_scale.data_ptr(), v_scale.data_ptr()
        c.sk, c.sv = VarlenPageStride(*k_pages.stride()[:3]), VarlenPageStride(*v_pages.stride()[:3])
        c.table_stride = block_table.stride(0)
        c.type = VARLEN_CACHE_E4M3 if e4m3 else VARLEN_CACHE_BF16
        c.num_pages, c.page_size, c.num_kv_heads, c.head_dim = pages, page_size, heads, dim
        c.max_pages = block_table.shape[1]
        self.struct, self.ref, self.at = c, ctypes.byref(c), _at(c, self.device)

    def __setattr__(self, name, value):
        # set once: calls use the struct, which another value here would not reach (the same tensor again is what
        # `cache.seqlens += n` assigns)
        if name in self.__dict__ and self.__dict__[name] is not value:
            raise AttributeError("PagedCache.%s is fixed: write into the tensor, or make another PagedCache" % name)
        object.__setattr__(self, name, value)


@functools.lru_cache(maxsize=1024)
def _strides(row, head):
    """A VarlenStride for the C entry points, which take it by value (making one costs as much as a launch's checks)."""
    return VarlenStride(row, head)


def _packed(cache, t, heads, rows=None):
    """(pointer, strides) of packed rows t, checked for what the C entry
    points cannot see: type, shape, place."""
    n, h, d = t.shape
    st = t.stride()
    if t.dtype != torch.bfloat16 or h != heads or d != cache.head_dim or st[2] != 1 or (rows is not None and n != rows):
        raise ValueError("packed rows must be bfloat16 [rows, heads, head_dim] with unit innermost stride (here %s "
                         "heads of %d%s)" % (heads, cache.head_dim, "" if rows is None else ", %d rows" % rows))
    if t.device != cache.device:
        raise ValueError("every tensor must be on the cache's device")
    return t.data_ptr(), _strides(st[0], st[1])


def _fresh_packed(cache, rows, heads):
    """(tensor, pointer, strides) of new contiguous packed rows."""
    d = cache.head_dim
    t = torch.empty((rows, heads, d), dtype=torch.bfloat16, device=cache.device)
    return t, t.data_ptr(), _strides(heads * d, d)


def _cu(cache, cu):
    if cu.dtype != torch.int32 or cu.dim() != 1 or cu.shape[0] != cache.batch + 1 or not cu.is_contiguous():
        raise ValueError("cu_seqlens must be contiguous int32 [batch + 1]")
    if cu.device != cache.device:
        raise ValueError("every tensor must be on the cache's device")
    return cu.data_ptr()


def _paged_call(entry, cache, stream, fresh, args):
    """Runs a C entry point with the cache's (or another handle's) device current.  Tensors that the
    call allocated (`fresh`) belong to the current stream: another `stream`
    waits for it (their memory may still be in use there), and they are kept
    from reuse until `stream` is done with them."""
    dev = cache.device.index
    if dev is None:
        raise ValueError("the cache must be on a CUDA device")
    handle = here = torch._C._cuda_getCurrentRawStream(dev)
    if stream is not None:
        handle = stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)
    if handle != here and fresh:
        own = torch.cuda.ExternalStream(handle, device=cache.device)
        own.wait_stream(torch.cuda.current_stream(cache.device))
        for t in fresh:
            t.record_stream(own)
    if dev == torch._C._cuda_getDevice():  # (CUDA is set up: the handle's tensors are there)
        st = entry(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = entry(*args, handle)
    if st != VARLEN_OK:
        raise VarlenError(st, entry.__name__)


def _at(struct, device):
    """A handle as the native binding takes it: its C description's address and its device's index (-1: none)."""
    return ctypes.addressof(struct), -1 if device.index is None else device.index


def _native(got, entry):
    """What the native binding answered, a status other than VARLEN_OK raised as _paged_call does."""
    if type(got) is int and got != VARLEN_OK:
        raise VarlenError(got, entry)
    return got


def cache_write(cache, k, v, cu_seqlens, stream=None):
    """Writes packed new rows k, v ([rows, num_kv_heads, D] bf16) into the
    cache: the rows of segment b become the last ones of its seqlens[b]
    positions (seqlens already counts them)."""
    kp, ks = _packed(cache, k, cache.num_kv_heads)
    rows = k.shape[0]
    vp, vs = _packed(cache, v, cache.num_kv_heads, rows)
    _paged_call(LIB.varlen_attn_cache_write, cache, stream, (),
                (kp, ks, vp, vs, _cu(cache, cu_seqlens), cache.batch, rows, cache.ref))


def cache_read(cache, cu_seqlens, total, k=None, v=None, stream=None):
    """The last rows of every sequence, packed by cu_seqlens into bf16 k, v
    ([total, num_kv_heads, D], allocated when None); returns (k, v)."""
    fresh = []
    if k is None:
        k, kp, ks = _fresh_packed(cache, total, cache.num_kv_heads)
        fresh.append(k)
    else:
        kp, ks = _packed(cache, k, cache.num_kv_heads, total)
    if v is None:
        v, vp, vs = _fresh_packed(cache, total, cache.num_kv_heads)
        fresh.append(v)
    else:
        vp, vs = _packed(cache, v, cache.num_kv_heads, total)
    _paged_call(LIB.varlen_attn_cache_read, cache, stream, fresh,
                (cache.ref, _cu(cache, cu_seqlens), cache.batch, total, kp, ks, vp, vs))
    return k, v


@functools.lru_cache(maxsize=256)
def _paged_workspace_bytes(batch, total_q, num_heads, num_kv_heads, head_dim):
    return varlen_attn_fwd_paged_workspace_size(batch, total_q, num_heads, num_kv_heads, head_dim)


def attention_fwd_paged(q, cache, cu_seqlens_q, max_seqlen_q=0, scale=None, out=None, lse=None, workspace=None,
                        stream=None, causal=False, window=(-1, -1)):
    """O and LSE of packed queries ([rows, H, D] bf16, H a multiple of the
    cache's heads) over the cache, the last query of a segment at its
    sequence's last position; `causal` / `window` as in attention_fwd.
    max_seqlen_q, where known, lets short calls run on fewer kernels."""
    total_q, H, D = q.shape
    qp, qs = _packed(cache, q, H)
    cu = _cu(cache, cu_seqlens_q)
    fresh = []
    if out is None:
        out, op, os_ = _fresh_packed(cache, total_q, H)
        fresh.append(out)
    else:
        op, os_ = _packed(cache, out, H, total_q)
    if lse is None:
        lse = torch.empty((H, total_q), dtype=torch.float32, device=cache.device)
        fresh.append(lse)
    elif lse.dtype != torch.float32 or tuple(lse.shape) != (H, total_q) or not lse.is_contiguous() \
            or lse.device != cache.device:
        raise ValueError("lse must be contiguous float32 [H, rows] on the cache's device")
    if workspace is None:
        nbytes = _paged_workspace_bytes(cache.batch, total_q, H, cache.num_kv_heads, D)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=cache.device)
        fresh.append(workspace)
    else:
        if workspace.device != cache.device or not workspace.is_contiguous():
            raise ValueError("the workspace must be contiguous and on the cache's device")
        nbytes = workspace.numel() * workspace.element_size()
    left, right = _band(causal, window) or (-1, -1)
    _paged_call(LIB.varlen_attn_fwd_paged, cache, stream, fresh,
                (qp, qs, cu, cache.batch, total_q, H, max_seqlen_q, cache.ref, D ** -0.5 if scale is None else scale,
                 left, right, op, os_, lse.data_ptr(), workspace.data_ptr(), nbytes))
    return out, lse


def attention_fwd_paged_tree(q, cache, cu_seqlens_q, masks, max_seqlen_q=0, scale=None, window_left=-1, positions=None,
                             out=None, lse=None, workspace=None, stream=None):
    """O and LSE of packed queries over the cache, which already holds their own
    rows: each sees the context and those new rows of its segment whose bit its
    row of masks ([rows, words] int32, as StepPlan has them) has set.  With
    window_left >= 0 the context is seen that far back from positions ([rows]
    int32); everything else as in attention_fwd_paged.  The window takes nothing
    from the masks: where a path has more than window_left + 1 rows, a row sees those
    of its path that attention_fwd_paged's window would hide from it, unless the
    caller clears their bits (cache_plan sets one for every row above)."""
    if NATIVE is not None and stream is None and out is None and lse is None and workspace is None:
        got = NATIVE.attention_fwd_paged_tree(cache.at, cache.batch, q, cu_seqlens_q, masks, max_seqlen_q, scale, window_left,
                                              positions)
        if got is not NotImplemented:
            return _native(got, "varlen_attn_fwd_paged_tree")
    total_q, H, D = q.shape
    qp, qs = _packed(cache, q, H)
    cu = _cu(cache, cu_seqlens_q)
    if masks.dtype not in (torch.int32, torch.uint32) or masks.dim() != 2 or masks.shape[0] != total_q \
            or not masks.is_contiguous() or masks.device != cache.device:
        raise ValueError("masks must be contiguous int32 [rows, words] on the cache's device")
    pos = None if positions is None else _list(cache, positions, total_q, "positions", "rows")
    fresh = []
    if out is None:
        out, op, os_ = _fresh_packed(cache, total_q, H)
        fresh.append(out)
    else:
        op, os_ = _packed(cache, out, H, total_q)
    if lse is None:
        lse = torch.empty((H, total_q), dtype=torch.float32, device=cache.device)
        fresh.append(lse)
    elif lse.dtype != torch.float32 or tuple(lse.shape) != (H, total_q) or not lse.is_contiguous() \
            or lse.device != cache.device:
        raise ValueError("lse must be contiguous float32 [H, rows] on the cache's device")
    if workspace is None:
        nbytes = _paged_workspace_bytes(cache.batch, total_q, H, cache.num_kv_heads, D)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=cache.device)
        fresh.append(workspace)
    else:
        if workspace.device != cache.device or not workspace.is_contiguous():
            raise ValueError("the workspace must be contiguous and on the cache's device")
        nbytes = workspace.numel() * workspace.element_size()
    _paged_call(LIB.varlen_attn_fwd_paged_tree, cache, stream, fresh,
                (qp, qs, cu, cache.batch, total_q, H, max_seqlen_q, cache.ref, D ** -0.5 if scale is None else scale,
                 masks.data_ptr(), masks.shape[1], pos, min(max(window_left, -1), 0x7fffffff), op, os_, lse.data_ptr(),
                 workspace.data_ptr(), nbytes))
    return out, lse


# ---------------------------------------------------------------- a step's lists

def _list(owner, t, n, name, what, dtype=torch.int32):
    """Address of a contiguous list of n entries on the owner's device."""
    if t.dtype != dtype or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError("%s must be contiguous %s [%s]" % (name, str(dtype)[6:], what))
    if t.device != owner.device:
        raise ValueError("every tensor must be on one device (%s is not)" % name)
    return t.data_ptr()


class _Fixed:
    """A handle whose attributes are set once: calls go by addresses that another
    tensor in the place of one would not change."""

    def __setattr__(self, name, value):
        if name in self.__dict__ and self.__dict__[name] is not value:
            raise AttributeError("%s.%s is fixed: write into the tensor, or make another %s"
                                 % (type(self).__name__, name, type(self).__name__))
        object.__setattr__(self, name, value)


class PagePool(_Fixed):
    """The pages of a cache as steps hand them out and take them back.

    block_table     [batch, max_pages] int32, the table of the caches (all layers')
    seqlens         [batch] int32: positions each sequence holds
    free_pages      [num_pages] int32: a stack whose first free_count pages are free
    free_count      [1] int32
    seqlens_out, free_count_out   where the state after a call goes; None: in place

    As PagedCache, it keeps the tensors themselves."""

    def __init__(self, block_table, seqlens, free_pages, free_count, page_size, seqlens_out=None, free_count_out=None):
        if block_table.dim() != 2 or block_table.dtype != torch.int32 or (block_table.shape[1] > 1
                                                                          and block_table.stride(1) != 1):
            raise ValueError("block_table must be int32 [batch, max_pages] with unit innermost stride")
        self.device, self.batch = block_table.device, block_table.shape[0]
        self.block_table, self.seqlens, self.free_pages, self.free_count = block_table, seqlens, free_pages, free_count
        self.seqlens_out = seqlens if seqlens_out is None else seqlens_out
        self.free_count_out = free_count if free_count_out is None else free_count_out
        c = VarlenPagePool()
        c.block_table, c.table_stride = block_table.data_ptr(), block_table.stride(0)
        c.seqlens = _list(self, seqlens, self.batch, "seqlens", "batch")
        c.seqlens_out = _list(self, self.seqlens_out, self.batch, "seqlens_out", "batch")
        c.free_pages = _list(self, free_pages, free_pages.numel(), "free_pages", "num_pages")
        c.free_count = _list(self, free_count, 1, "free_count", "1")
        c.free_count_out = _list(self, self.free_count_out, 1, "free_count_out", "1")
        c.num_pages, c.page_size, c.max_pages = free_pages.numel(), page_size, block_table.shape[1]
        self.struct, self.ref, self.at = c, ctypes.byref(c), _at(c, self.device)


class StepPlan(_Fixed):
    """What cache_plan writes for steps of up to `total` new rows of `batch`
    sequences: cu_seqlens [batch + 1], positions [total], unplaced [batch] (int32),
    slots [total] (int64) and, with mask_words > 0, masks [total, mask_words]
    (int32).  Made once, filled by every step."""

    def __init__(self, batch, total, device, mask_words=0):
        if not (0 <= batch < 1 << 31 and 0 <= total < 1 << 31 and 0 <= mask_words < 1 << 31):
            raise ValueError("batch, total and mask_words are numbers of 31 bits")

        def new(*shape, dtype=torch.int32):
            return torch.zeros(shape, dtype=dtype, device=device)
        self.batch, self.total, self.mask_words = batch, total, mask_words
        self.cu_seqlens, self.positions, self.unplaced = new(batch + 1), new(total), new(batch)
        self.slots = new(total, dtype=torch.int64)
        self.masks = new(total, mask_words) if mask_words > 0 else None
        nbytes = varlen_attn_cache_plan_workspace_size(batch)
        self.workspace = new(max(nbytes, 16), dtype=torch.uint8)
        self.device = self.slots.device
        self.args = (self.cu_seqlens.data_ptr(), self.slots.data_ptr(), self.positions.data_ptr(), self.unplaced.data_ptr(),
                     None if self.masks is None else self.masks.data_ptr(), mask_words, self.workspace.data_ptr(), nbytes)


def cache_plan(pool, plan, new_lens, parents=None, stream=None):
    """Fills `plan` for a step with new_lens[b] new rows of sequence b ([batch]
    int32), takes the pages that they need from `pool` and advances its lengths.
    parents ([total] int32, packed like the rows): the row of its own segment that
    each one continues, negative for the context; then plan.masks and the rows'
    depths in plan.positions follow the trees.  Returns plan."""
    if plan.batch != pool.batch or plan.device != pool.device:
        raise ValueError("the plan is not one for this pool's batch and device")
    if parents is not None and plan.masks is None:
        raise ValueError("trees need a plan with mask_words > 0")
    if NATIVE is not None and stream is None:
        got = NATIVE.cache_plan(pool.at, pool.batch, new_lens, parents, plan.total, plan.args)
        if got is not NotImplemented:
            _native(got, "varlen_attn_cache_plan")
            return plan
    up = None
    if parents is not None:
        up = _list(pool, parents, plan.total, "parents", "total")
    _paged_call(LIB.varlen_attn_cache_plan, pool, stream, (),
                (pool.ref, _list(pool, new_lens, pool.batch, "new_lens", "batch"), pool.batch, up, plan.total) + plan.args)
    return plan


def cache_trim(pool, lens, cu_seqlens=None, stream=None):
    """Shortens sequence b to lens[b] positions or, with the cu_seqlens of a step,
    to lens[b] of that step's rows, and puts the pages that this leaves empty back."""
    if NATIVE is not None and stream is None:
        got = NATIVE.cache_trim(pool.at, pool.batch, lens, cu_seqlens)
        if got is not NotImplemented:
            _native(got, "varlen_attn_cache_trim")
            return
    _paged_call(LIB.varlen_attn_cache_trim, pool, stream, (),
                (pool.ref, _list(pool, lens, pool.batch, "lens", "batch"),
                 None if cu_seqlens is None else _list(pool, cu_seqlens, pool.batch + 1, "cu_seqlens", "batch + 1"),
                 pool.batch))


def cache_move(caches, cu_seqlens, kept, kept_lens, stream=None):
    """In every cache of `caches` (layers over one table; or one cache) new row
    kept[b, i] of sequence b becomes its new row i, i < kept_lens[b]; kept
    [batch, most] int32, ascending in a row.  The caches' seqlens count all new
    rows of cu_seqlens; cache_trim drops the others."""
    if isinstance(caches, PagedCache):
        caches = (caches,)
    if len(caches) == 0:
        return
    first = caches[0]
    if NATIVE is not None and stream is None:
        got = NATIVE.cache_move([c.at for c in caches], first.batch, cu_seqlens, kept, kept_lens)
        if got is not NotImplemented:
            _native(got, "varlen_attn_cache_move")
            return
    for c in caches:
        if c.device != first.device:
            raise ValueError("the caches must be on one device")
    ref = first.ref if len(caches) == 1 else (VarlenKvCache * len(caches))(*[c.struct for c in caches])
    if kept.dtype != torch.int32 or kept.dim() != 2 or kept.shape[0] != first.batch or kept.device != first.device \
            or (kept.shape[1] > 1 and kept.stride(1) != 1):
        raise ValueError("kept must be int32 [batch, most] with unit innermost stride on the caches' device")
    _paged_call(LIB.varlen_attn_cache_move, first, stream, (),
                (ref, len(caches), _cu(first, cu_seqlens), first.batch, 0x7fffffff, kept.data_ptr(), kept.stride(0),
                 _list(first, kept_lens, first.batch, "kept_lens", "batch"), kept.shape[1]))


# ---------------------------------------------------------------- rotary positions

def rotary_frequencies(rotary_dim, base=10000.0, stretch=1.0, how="ramp", trained=8192, low=1.0, high=32.0):
    """(frequencies, scale): rotary_dim / 2 float64 radians a position, f_i =
    base^(-2 i / rotary_dim), for contexts `stretch` times the `trained` ones, and
    the factor on the turned elements that goes with it.  how:
      "linear"  all frequencies / stretch;
      "base"    a larger base, base * stretch^(rotary_dim / (rotary_dim - 2)), so
                that the slowest pair is stretched whole and the fastest not at all;
      "ramp"    pairs that turn at least `high` times within `trained` positions are
                kept, those that turn at most `low` times are stretched, linear in
                the number of turns between; scale 0.1 ln(stretch) + 1.
    Models differ in such ramps (linear in the pair's index instead of in its turns,
    scale 1 instead): theirs are frequencies and a scale of the caller's own, which
    Rotary takes as they are."""
    if rotary_dim < 2 or rotary_dim % 2 or base <= 0 or stretch <= 0 or how not in ("linear", "base", "ramp"):
        raise ValueError("rotary_dim must be even, base and stretch positive, how linear, base or ramp")
    i = torch.arange(0, rotary_dim, 2, dtype=torch.float64)
    if stretch == 1:
        return base ** (-i / rotary_dim), 1.0
    if how == "base":
        wide = base * stretch ** (rotary_dim / (rotary_dim - 2)) if rotary_dim > 2 else base
        return wide ** (-i / rotary_dim), 1.0
    f = base ** (-i / rotary_dim)
    if how == "linear":
        return f / stretch, 1.0
    keep = torch.clamp((f * trained / (2 * math.pi) - low) / (high - low), 0, 1)
    return f * keep + f / stretch * (1 - keep), 0.1 * math.log(stretch) + 1


class Rotary(_Fixed):
    """Rotary positions: the frequencies (radians a position, one for each pair, any
    sequence or tensor) as the kernels take them, how the pairs lie (interleaved:
    2i and 2i + 1; else i and i + rotary_dim / 2) and the factor on what they give."""

    def __init__(self, frequencies, interleaved=False, scale=1.0, device=None):
        if isinstance(frequencies, torch.Tensor):
            if device is None and frequencies.is_cuda:
                device = frequencies.device
            frequencies = frequencies.tolist()
        st, turns = varlen_attn_rotary_turns([float(f) for f in frequencies])
        _check(st, "varlen_attn_rotary_turns")
        whole = [t - (1 << 64) if t >= 1 << 63 else t for t in turns]  # the same bits
        self.turns = torch.tensor(whole, dtype=torch.int64, device="cuda" if device is None else device)
        self.device, self.rotary_dim = self.turns.device, 2 * len(turns)
        self.interleaved, self.scale = bool(interleaved), float(scale)
        c = VarlenRotary()
        c.turns, c.rotary_dim, c.interleaved, c.scale = self.turns.data_ptr(), 2 * len(turns), int(self.interleaved), self.scale
        self.struct, self.ref, self.at = c, ctypes.byref(c), _at(c, self.device)


def _rows(owner, t, name, dim, total, heads=None):
    """(heads, address, strides) of packed rows."""
    n, h, d = t.shape
    st = t.stride()
    if n != total or d != dim or st[2] != 1 or t.dtype != torch.bfloat16 or (heads is not None and h != heads):
        raise ValueError("%s must be bfloat16 [%d, %s, %d] with unit innermost stride"
                         % (name, total, "heads" if heads is None else heads, dim))
    if t.device != owner.device:
        raise ValueError("every tensor must be on one device (%s is not)" % name)
    return h, t.data_ptr(), _strides(st[0], st[1])


def _turned(owner, t, out, name, dim, total, fresh):
    """Arguments of an input and of the output that it is turned into (allocated when None)."""
    h, p, s = _rows(owner, t, name, dim, total)
    if out is None:
        out = torch.empty((total, h, dim), dtype=torch.bfloat16, device=owner.device)
        fresh.append(out)
        return out, h, p, s, out.data_ptr(), _strides(h * dim, dim)
    _, op, os_ = _rows(owner, out, name + "_out", dim, total, h)
    return out, h, p, s, op, os_


_NO_STRIDE = VarlenStride(0, 0)


def _rotary(q, k, rope, positions, cu_seqlens, q_out, k_out, stream, inverse):
    if NATIVE is not None and stream is None:
        got = NATIVE.rotary(rope.at, inverse, q, k, positions, cu_seqlens, q_out, k_out)
        if got is not NotImplemented:
            return _native(got, "varlen_attn_rotary")
    total, _, dim = q.shape
    fresh = []
    q_out, H, qp, qs, qop, qos = _turned(rope, q, q_out, "q", dim, total, fresh)
    if k is None:
        k_out, Hk, kp, ks, kop, kos = None, 0, None, _NO_STRIDE, None, _NO_STRIDE
    else:
        k_out, Hk, kp, ks, kop, kos = _turned(rope, k, k_out, "k", dim, total, fresh)
    if positions is not None:
        pos, cu, batch = _list(rope, positions, total, "positions", "rows"), None, 0
    elif cu_seqlens is not None:
        pos, batch = None, cu_seqlens.numel() - 1
        cu = _list(rope, cu_seqlens, batch + 1, "cu_seqlens", "batch + 1")
    else:
        raise ValueError("rows need positions or cu_seqlens")
    _paged_call(LIB.varlen_attn_rotary, rope, stream, fresh,
                (qp, qs, kp, ks, pos, cu, batch, total, H, Hk, dim, rope.ref, inverse, qop, qos, kop, kos))
    return q_out, k_out


def rotary(q, k, rope, positions=None, cu_seqlens=None, q_out=None, k_out=None, stream=None):
    """Packed rows q [rows, H, D] and k [rows, Hk, D] (bf16; k may be None) turned to
    positions ([rows] int32) or, without them, to their places in the segments of
    cu_seqlens; returns (q_out, k_out), allocated when None; an output may be its
    own input.  Rows outside every segment are not written."""
    return _rotary(q, k, rope, positions, cu_seqlens, q_out, k_out, stream, 0)


def rotary_bwd(dq, dk, rope, positions=None, cu_seqlens=None, dq_out=None, dk_out=None, stream=None):
    """The gradient of rotary: that with respect to its inputs from that with respect
    to its outputs (turned back; the arguments are rotary's)."""
    return _rotary(dq, dk, rope, positions, cu_seqlens, dq_out, dk_out, stream, 1)


def rotary_cache_write(cache, q, k, v, rope, positions, slots, q_out=None, stream=None):
    """A step's new rows on their way into the cache, in one kernel: q (or None)
    turned and returned (q_out, allocated when None, may be q), k turned and
    written with v to the places that slots ([rows] int64) name; positions and slots
    as StepPlan has them."""
    if NATIVE is not None and stream is None:
        got = NATIVE.rotary_cache_write(cache.at, q, k, v, rope.at, positions, slots, q_out)
        if got is not NotImplemented:
            return _native(got, "varlen_attn_rotary_cache_write")
    total, dim = k.shape[0], cache.head_dim
    fresh = []
    if q is None:
        q_out, H, qp, qs, qop, qos = None, 0, None, _NO_STRIDE, None, _NO_STRIDE
    else:
        q_out, H, qp, qs, qop, qos = _turned(cache, q, q_out, "q", dim, total, fresh)
    if rope.device != cache.device:
        raise ValueError("the frequencies must be on the cache's device")
    _, kp, ks = _rows(cache, k, "k", dim, total, cache.num_kv_heads)
    _, vp, vs = _rows(cache, v, "v", dim, total, cache.num_kv_heads)
    _paged_call(LIB.varlen_attn_rotary_cache_write, cache, stream, fresh,
                (qp, qs, kp, ks, vp, vs, _list(cache, positions, total, "positions", "rows"),
                 _list(cache, slots, total, "slots", "rows", torch.int64), total, H, cache.ref, rope.ref, qop, qos))
    return q_out
