"""Python binding of the GB300 DFlash draft block-attention library.

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``libdflash_attn.so`` (C ABI in ``include/dflash_attn.h``), called
through ctypes or, for the short calls of the serving step, through a compiled
module (``csrc/binding.cpp``).
PyTorch supplies device memory and the current stream.  There is no CPU
fallback: if the shared library has not been built, every call raises.

The functions carry the C names:
  dflash_attn_dense, dflash_attn_anchored, dflash_attn_ragged,
  dflash_attn_dense_backward, dflash_attn_anchored_backward,
  dflash_attn_workspace_size, dflash_build_schedule_host, dflash_scan_mask,
  dflash_last_device_error, dflash_status_string,
  dflash_qk_norm_rope, dflash_qk_norm_rope_backward, dflash_cache_append,
  dflash_attn_paged, dflash_verify, dflash_attn_tree, dflash_sample,
  dflash_tree_accept, dflash_cache_compact, dflash_cache_copy,
  dflash_pages_resize, dflash_pages_fork.
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np

from . import build as _build

LIB_PATH = _build.LIB_PATH

DFLASH_BF16, DFLASH_FP32 = 0, 1
MODE_DENSE, MODE_ANCHORED, MODE_RAGGED = 0, 1, 2
MODE_DENSE_BACKWARD, MODE_ANCHORED_BACKWARD = 3, 4
TILE_M = TILE_N = 128
TILE_SKIP, TILE_PARTIAL, TILE_FULL = 0, 1, 2

STATUS = {0: "DFLASH_OK", 1: "DFLASH_ERR_INVALID", 2: "DFLASH_ERR_SHAPE", 3: "DFLASH_ERR_DTYPE",
          4: "DFLASH_ERR_ALIGN", 5: "DFLASH_ERR_UNSUPPORTED", 6: "DFLASH_ERR_WORKSPACE", 7: "DFLASH_ERR_CUDA",
          8: "DFLASH_ERR_TIMEOUT"}

EXPORTS = ("dflash_attn_dense", "dflash_attn_anchored", "dflash_attn_ragged", "dflash_attn_workspace_size",
           "dflash_build_schedule_host", "dflash_scan_mask", "dflash_status_string", "dflash_last_device_error",
           "dflash_kernel_launches", "dflash_attn_dense_noalloc", "dflash_build_mask",
           "dflash_attn_anchored_backward", "dflash_attn_dense_backward", "dflash_test_inject_stall",
           "dflash_test_limit_tile_flags",
           "dflash_attn_latent_ragged", "dflash_attn_latent_workspace_size",
           "dflash_qk_norm_rope", "dflash_qk_norm_rope_workspace_size", "dflash_qk_norm_rope_backward",
           "dflash_cache_append", "dflash_attn_paged", "dflash_attn_paged_workspace_size", "dflash_verify",
           "dflash_attn_tree", "dflash_sample", "dflash_tree_accept", "dflash_cache_compact", "dflash_cache_copy",
           "dflash_pages_workspace_size", "dflash_pages_resize", "dflash_pages_fork")


class DFlashError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {STATUS.get(status, status)} ({dflash_status_string(status)})")


class _Dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("S", ctypes.c_int), ("Q", ctypes.c_int),
                ("d_nope", ctypes.c_int), ("d_rope", ctypes.c_int), ("d_v", ctypes.c_int),
                ("scale", ctypes.c_float)]


class _RopeDims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("H_q", ctypes.c_int), ("H_kv", ctypes.c_int), ("D", ctypes.c_int),
                ("rot_dim", ctypes.c_int), ("max_pos", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("eps", ctypes.c_float), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64)]


class _PagedDims(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int), ("H_q", ctypes.c_int), ("H_kv", ctypes.c_int), ("D", ctypes.c_int),
                ("total_q", ctypes.c_int), ("max_q_len", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int), ("k_page_stride", ctypes.c_int64),
                ("v_page_stride", ctypes.c_int64)]


class _VerifyDims(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int), ("V", ctypes.c_int), ("total_draft", ctypes.c_int),
                ("max_draft", ctypes.c_int), ("target_stride", ctypes.c_int64), ("draft_stride", ctypes.c_int64)]


class _SampleDims(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int), ("V", ctypes.c_int), ("logits_stride", ctypes.c_int64),
                ("probs_stride", ctypes.c_int64)]


class _AcceptDims(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int), ("total", ctypes.c_int), ("max_path", ctypes.c_int)]


class _Layers(ctypes.Structure):
    _fields_ = [("L", ctypes.c_int), ("k_layer_stride", ctypes.c_int64), ("v_layer_stride", ctypes.c_int64)]


class _PoolDims(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int), ("max_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("num_pages", ctypes.c_int)]


_lock = threading.Lock()
_lib_handle = None
_lib_path = None


def load_library(path: str | None = None):
    """Load libdflash_attn.so (built by ``__graft_entry__.build()``); raises if absent."""
    global _lib_handle, _lib_path
    if _lib_handle is not None:
        return _lib_handle
    with _lock:
        if _lib_handle is not None:
            return _lib_handle
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"DFlash CUDA library not built ({p} missing): run "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(p)
        P, I, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        DP = ctypes.POINTER(_Dims)
        lib.dflash_attn_dense.argtypes = [DP, I, P, P, P, P, P, P, P, P, S, P]
        lib.dflash_attn_anchored.argtypes = [DP, I, P, P, P, P, P, I, I, P, P, P, S, P]
        lib.dflash_attn_ragged.argtypes = [I, I, I, I, I, F, I, P, P, P, P, P, P, P, I, I, I, I, P, P, P, S, P]
        lib.dflash_attn_workspace_size.argtypes = [I, DP, I, I, I, I, I, I, I, I, I]
        lib.dflash_attn_workspace_size.restype = S
        lib.dflash_build_schedule_host.argtypes = [I, I, I, P, I, I, P]
        lib.dflash_scan_mask.argtypes = [I, I, I, I, P, P, P]
        lib.dflash_status_string.argtypes = [I]
        lib.dflash_status_string.restype = ctypes.c_char_p
        lib.dflash_last_device_error.argtypes = [P]
        lib.dflash_attn_dense_noalloc.argtypes = [DP, I, P, P, P, P, P, P, P, P]
        lib.dflash_build_mask.argtypes = [I, I, I, P, I, I, I, P, P]
        lib.dflash_build_mask.restype = ctypes.c_int
        lib.dflash_attn_dense_noalloc.restype = ctypes.c_int
        lib.dflash_attn_anchored_backward.argtypes = [DP, I, P, P, P, P, P, I, I, P, P, P, P, P, P, P, P, S, P]
        lib.dflash_attn_dense_backward.argtypes = [DP, I, P, P, P, P, P, P, P, P, P, P, P, P, P, S, P]
        lib.dflash_attn_anchored_backward.restype = ctypes.c_int
        lib.dflash_attn_dense_backward.restype = ctypes.c_int
        lib.dflash_attn_latent_ragged.argtypes = [I, I, I, I, I, I, F, I, P, P, P, P, P, P, P, I, I, I, I, P, P, P,
                                                  S, P]
        lib.dflash_attn_latent_ragged.restype = ctypes.c_int
        lib.dflash_attn_latent_workspace_size.argtypes = [I, I, I, I, I, I, I, I, I, I]
        lib.dflash_attn_latent_workspace_size.restype = S
        lib.dflash_test_inject_stall.argtypes = [ctypes.c_ulonglong, I]
        lib.dflash_test_inject_stall.restype = None
        lib.dflash_test_limit_tile_flags.argtypes = [I]
        lib.dflash_test_limit_tile_flags.restype = None
        lib.dflash_kernel_launches.argtypes = []
        lib.dflash_kernel_launches.restype = ctypes.c_uint64
        RD, PD, VD, L = (ctypes.POINTER(_RopeDims), ctypes.POINTER(_PagedDims), ctypes.POINTER(_VerifyDims),
                         ctypes.c_int64)
        lib.dflash_qk_norm_rope.argtypes = [RD, I, P, P, P, P, P, P, P, P, P]
        lib.dflash_qk_norm_rope_backward.argtypes = [RD, I, P, P, P, P, P, P, P, P, P, P, P, P, P, S, P]
        lib.dflash_cache_append.argtypes = [PD, RD, I, P, P, P, L, P, P, P, P, P, P, P, P, P, P]
        lib.dflash_attn_paged.argtypes = [PD, I, P, P, P, P, P, P, I, F, P, P, P, S, P]
        lib.dflash_verify.argtypes = [VD, P, P, P, P, P, P, P, P, P]
        SD, AD, LD, OD = (ctypes.POINTER(_SampleDims), ctypes.POINTER(_AcceptDims), ctypes.POINTER(_Layers),
                          ctypes.POINTER(_PoolDims))
        lib.dflash_attn_tree.argtypes = [PD, I, P, P, P, P, P, P, P, F, P, P, P, S, P]
        lib.dflash_sample.argtypes = [SD, I, P, P, P, P, P, P, P, P, P]
        lib.dflash_tree_accept.argtypes = [AD, P, P, P, P, P, P, P, P]
        lib.dflash_cache_compact.argtypes = [PD, LD, I, P, P, P, P, I, P, P, P, P, P]
        lib.dflash_cache_copy.argtypes = [PD, LD, I, I, P, P, P, P, P, P]
        lib.dflash_pages_resize.argtypes = [OD, P, P, P, P, P, P, S, P]
        lib.dflash_pages_fork.argtypes = [OD, P, P, I, P, P, P, P, P, P, P, P, S, P]
        lib.dflash_pages_workspace_size.argtypes = [OD]
        lib.dflash_pages_workspace_size.restype = S
        for name in ("dflash_qk_norm_rope", "dflash_qk_norm_rope_backward", "dflash_cache_append",
                     "dflash_attn_paged", "dflash_verify", "dflash_attn_tree", "dflash_sample", "dflash_tree_accept",
                     "dflash_cache_compact", "dflash_cache_copy", "dflash_pages_resize", "dflash_pages_fork"):
            getattr(lib, name).restype = ctypes.c_int
        lib.dflash_qk_norm_rope_workspace_size.argtypes = [RD]
        lib.dflash_qk_norm_rope_workspace_size.restype = S
        lib.dflash_attn_paged_workspace_size.argtypes = [PD, I]
        lib.dflash_attn_paged_workspace_size.restype = S
        for name in ("dflash_attn_dense", "dflash_attn_anchored", "dflash_attn_ragged",
                     "dflash_build_schedule_host", "dflash_scan_mask", "dflash_last_device_error"):
            getattr(lib, name).restype = ctypes.c_int
        _lib_handle, _lib_path = lib, os.path.realpath(p)
        return lib


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------
def _torch():
    import torch
    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return DFLASH_BF16
    if t.dtype == torch.float32:
        return DFLASH_FP32
    raise TypeError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


def _dev_ptr(t, name, dtype=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(fn, st):
    if st != 0:
        raise DFlashError(fn, st)


def _workspace(nbytes, workspace, device):
    torch = _torch()
    if workspace is None:
        workspace = torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)
    elif workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError(f"workspace too small: need {nbytes} bytes")
    return workspace


def _dims(B, H, S, Q, dn, dr, dv, scale):
    return _Dims(B, H, S, Q, dn, dr, dv, float(scale or 0.0))


# ---------------------------------------------------------------------------
# public API
# ---------------------------------------------------------------------------
def dflash_status_string(status: int) -> str:
    try:
        return load_library().dflash_status_string(int(status)).decode()
    except RuntimeError:
        return STATUS.get(status, "unknown")


def dflash_attn_workspace_size(mode, B=0, H=0, S=0, Q=0, d_nope=0, d_rope=0, d_v=0, dtype=DFLASH_BF16, R=0,
                               total_q=0, total_kv=0, max_q_len=0) -> int:
    lib = load_library()
    if mode == MODE_RAGGED:
        return int(lib.dflash_attn_workspace_size(mode, None, dtype, R, H, d_nope, d_rope, d_v, total_q, total_kv,
                                                  max_q_len))
    d = _dims(B, H, S, Q, d_nope, d_rope, d_v, 0.0)
    return int(lib.dflash_attn_workspace_size(mode, ctypes.byref(d), dtype, 0, 0, 0, 0, 0, 0, 0, 0))


def _batched_shapes(q, k_nope, k_rope, v):
    B, Q, H, dqk = q.shape
    K = k_nope.shape[1]
    dn, dr, dv = k_nope.shape[3], k_rope.shape[2], v.shape[3]
    if (k_nope.shape[0], k_nope.shape[2]) != (B, H) or k_rope.shape[:2] != (B, K) or v.shape[:3] != (B, K, H):
        raise ValueError("inconsistent q/k/v shapes")
    if dn + dr != dqk:
        raise ValueError("q head dim must be d_nope + d_rope")
    return B, H, K - Q, Q, dn, dr, dv


def dflash_attn_dense(q, k_nope, k_rope, v, mask, out=None, lse=None, scale=0.0, workspace=None, stream=None):
    """Dense additive-mask block attention.  q [B,Q,H,dn+dr], k_nope [B,S+Q,H,dn],
    k_rope [B,S+Q,dr], v [B,S+Q,H,dv], mask [B,1,Q,S+Q] (q's dtype).
    Returns out [B,Q,H,dv]; fills lse [B,H,Q] fp32 if given."""
    torch = _torch()
    lib = load_library()
    B, H, S, Q, dn, dr, dv = _batched_shapes(q, k_nope, k_rope, v)
    dt = _dtype_code(q)
    if tuple(mask.shape) != (B, 1, Q, S + Q):
        raise ValueError("mask must be [B,1,Q,S+Q]")
    if out is None:
        out = torch.empty((B, Q, H, dv), dtype=q.dtype, device=q.device)
    nbytes = dflash_attn_workspace_size(MODE_DENSE, B, H, S, Q, dn, dr, dv, dt)
    ws = _workspace(nbytes, workspace, q.device)
    d = _dims(B, H, S, Q, dn, dr, dv, scale)
    st = lib.dflash_attn_dense(ctypes.byref(d), dt, _dev_ptr(q, "q"), _dev_ptr(k_nope, "k_nope", q.dtype),
                               _dev_ptr(k_rope, "k_rope", q.dtype), _dev_ptr(v, "v", q.dtype),
                               _dev_ptr(mask, "mask", q.dtype), _dev_ptr(out, "out", q.dtype),
                               _dev_ptr(lse, "lse", torch.float32), _dev_ptr(ws, "workspace"), nbytes,
                               _stream(stream))
    _check("dflash_attn_dense", st)
    return out


def dflash_attn_dense_noalloc(q, k_nope, k_rope, v, mask, out=None, lse=None, scale=0.0, stream=None):
    """dflash_attn_dense without a workspace: the library's own fixed device
    array holds the mask-tile classes (see include/dflash_attn.h).  For callers
    that cannot allocate device scratch memory; concurrent calls on one device
    must not overlap on the GPU."""
    torch = _torch()
    lib = load_library()
    B, H, S, Q, dn, dr, dv = _batched_shapes(q, k_nope, k_rope, v)
    dt = _dtype_code(q)
    if tuple(mask.shape) != (B, 1, Q, S + Q):
        raise ValueError("mask must be [B,1,Q,S+Q]")
    if out is None:
        out = torch.empty((B, Q, H, dv), dtype=q.dtype, device=q.device)
    d = _dims(B, H, S, Q, dn, dr, dv, scale)
    st = lib.dflash_attn_dense_noalloc(ctypes.byref(d), dt, _dev_ptr(q, "q"), _dev_ptr(k_nope, "k_nope", q.dtype),
                                       _dev_ptr(k_rope, "k_rope", q.dtype), _dev_ptr(v, "v", q.dtype),
                                       _dev_ptr(mask, "mask", q.dtype), _dev_ptr(out, "out", q.dtype),
                                       _dev_ptr(lse, "lse", torch.float32), _stream(stream))
    _check("dflash_attn_dense_noalloc", st)
    return out


def dflash_attn_anchored(q, k_nope, k_rope, v, anchors, block_size, out=None, lse=None, scale=0.0, workspace=None,
                         stream=None):
    """Anchored block attention: anchors [B,nb] int32 (device), Q = nb*block_size."""
    torch = _torch()
    lib = load_library()
    B, H, S, Q, dn, dr, dv = _batched_shapes(q, k_nope, k_rope, v)
    dt = _dtype_code(q)
    nb = anchors.shape[1]
    if out is None:
        out = torch.empty((B, Q, H, dv), dtype=q.dtype, device=q.device)
    nbytes = dflash_attn_workspace_size(MODE_ANCHORED, B, H, S, Q, dn, dr, dv, dt)
    ws = _workspace(nbytes, workspace, q.device)
    d = _dims(B, H, S, Q, dn, dr, dv, scale)
    st = lib.dflash_attn_anchored(ctypes.byref(d), dt, _dev_ptr(q, "q"), _dev_ptr(k_nope, "k_nope", q.dtype),
                                  _dev_ptr(k_rope, "k_rope", q.dtype), _dev_ptr(v, "v", q.dtype),
                                  _dev_ptr(anchors, "anchors", torch.int32), nb, int(block_size),
                                  _dev_ptr(out, "out", q.dtype), _dev_ptr(lse, "lse", torch.float32),
                                  _dev_ptr(ws, "workspace"), nbytes, _stream(stream))
    _check("dflash_attn_anchored", st)
    return out


def dflash_attn_ragged(q, k_nope, k_rope, v, q_offsets, kv_offsets, anchors, block_size, max_q_len, out=None,
                       lse=None, scale=0.0, workspace=None, stream=None):
    """Ragged (row-offset) block attention.  q [total_q,H,dn+dr], k_nope
    [total_kv,H,dn], k_rope [total_kv,dr], v [total_kv,H,dv]; offsets int32
    [R+1] and anchors int32 [total_q/block_size] on the device.  lse is [H,total_q]."""
    torch = _torch()
    lib = load_library()
    total_q, H, dqk = q.shape
    total_kv, dn, dr, dv = k_nope.shape[0], k_nope.shape[2], k_rope.shape[1], v.shape[2]
    if dn + dr != dqk:
        raise ValueError("q head dim must be d_nope + d_rope")
    R = q_offsets.shape[0] - 1
    dt = _dtype_code(q)
    if out is None:
        out = torch.empty((total_q, H, dv), dtype=q.dtype, device=q.device)
    nbytes = dflash_attn_workspace_size(MODE_RAGGED, H=H, d_nope=dn, d_rope=dr, d_v=dv, dtype=dt, R=R,
                                        total_q=total_q, total_kv=total_kv, max_q_len=int(max_q_len))
    ws = _workspace(nbytes, workspace, q.device)
    st = lib.dflash_attn_ragged(R, H, dn, dr, dv, float(scale or 0.0), dt, _dev_ptr(q, "q"),
                                _dev_ptr(k_nope, "k_nope", q.dtype), _dev_ptr(k_rope, "k_rope", q.dtype),
                                _dev_ptr(v, "v", q.dtype), _dev_ptr(q_offsets, "q_offsets", torch.int32),
                                _dev_ptr(kv_offsets, "kv_offsets", torch.int32),
                                _dev_ptr(anchors, "anchors", torch.int32), int(block_size), total_q, total_kv,
                                int(max_q_len), _dev_ptr(out, "out", q.dtype), _dev_ptr(lse, "lse", torch.float32),
                                _dev_ptr(ws, "workspace"), nbytes, _stream(stream))
    _check("dflash_attn_ragged", st)
    return out


def dflash_attn_latent_workspace_size(R, H, d_nope, d_rope, d_v, kv_rank, dtype=DFLASH_BF16, total_q=0,
                                      total_kv=0, max_q_len=0) -> int:
    return int(load_library().dflash_attn_latent_workspace_size(R, H, d_nope, d_rope, d_v, kv_rank, dtype, total_q,
                                                                 total_kv, max_q_len))


def dflash_attn_latent_ragged(q, c_kv, k_rope, w_kv_b, q_offsets, kv_offsets, anchors, block_size, max_q_len,
                              out=None, lse=None, scale=0.0, workspace=None, stream=None):
    """Ragged block attention over compressed KV latents.  q [total_q,H,dn+dr],
    c_kv [total_kv,kv_rank], k_rope [total_kv,dr], w_kv_b [H,dn+dv,kv_rank]
    (kv_b_proj per head: key rows, then value rows); offsets int32 [R+1] and
    anchors int32 [total_q/block_size] on the device.  lse is [H,total_q]."""
    torch = _torch()
    lib = load_library()
    total_q, H, dqk = q.shape
    total_kv, rank = c_kv.shape
    dr = k_rope.shape[1]
    dn = dqk - dr
    if w_kv_b.shape[0] != H or w_kv_b.shape[2] != rank or w_kv_b.shape[1] <= dn or k_rope.shape[0] != total_kv:
        raise ValueError("inconsistent q / c_kv / k_rope / w_kv_b shapes")
    dv = w_kv_b.shape[1] - dn
    R = q_offsets.shape[0] - 1
    dt = _dtype_code(q)
    if out is None:
        out = torch.empty((total_q, H, dv), dtype=q.dtype, device=q.device)
    nbytes = dflash_attn_latent_workspace_size(R, H, dn, dr, dv, rank, dt, total_q, total_kv, int(max_q_len))
    ws = _workspace(nbytes, workspace, q.device)
    st = lib.dflash_attn_latent_ragged(R, H, dn, dr, dv, rank, float(scale or 0.0), dt, _dev_ptr(q, "q"),
                                       _dev_ptr(c_kv, "c_kv", q.dtype), _dev_ptr(k_rope, "k_rope", q.dtype),
                                       _dev_ptr(w_kv_b, "w_kv_b", q.dtype),
                                       _dev_ptr(q_offsets, "q_offsets", torch.int32),
                                       _dev_ptr(kv_offsets, "kv_offsets", torch.int32),
                                       _dev_ptr(anchors, "anchors", torch.int32), int(block_size), total_q, total_kv,
                                       int(max_q_len), _dev_ptr(out, "out", q.dtype),
                                       _dev_ptr(lse, "lse", torch.float32), _dev_ptr(ws, "workspace"), nbytes,
                                       _stream(stream))
    _check("dflash_attn_latent_ragged", st)
    return out


def _backward_grads(q, k_nope, k_rope, v, grads):
    torch = _torch()
    if grads is None:
        grads = (torch.empty_like(q), torch.empty_like(k_nope), torch.empty_like(k_rope), torch.empty_like(v))
    dq, dkn, dkr, dvv = grads
    for name, g, ref in (("dq", dq, q), ("dk_nope", dkn, k_nope), ("dk_rope", dkr, k_rope), ("dv", dvv, v)):
        if g.shape != ref.shape or g.dtype != ref.dtype:
            raise ValueError(f"{name} must match its input's shape and dtype")
    return dq, dkn, dkr, dvv


def dflash_attn_anchored_backward(q, k_nope, k_rope, v, anchors, block_size, out, lse, dout, grads=None, scale=0.0,
                                  workspace=None, stream=None):
    """Gradients (dq, dk_nope, dk_rope, dv) of sum(dout * out) for the anchored
    forward; out and lse [B,H,Q] fp32 are that forward's outputs.  grads: optional
    preallocated (dq, dk_nope, dk_rope, dv) shaped like (q, k_nope, k_rope, v)."""
    torch = _torch()
    lib = load_library()
    B, H, S, Q, dn, dr, dv = _batched_shapes(q, k_nope, k_rope, v)
    dt = _dtype_code(q)
    nb = anchors.shape[1]
    dq, dkn, dkr, dvv = _backward_grads(q, k_nope, k_rope, v, grads)
    nbytes = dflash_attn_workspace_size(MODE_ANCHORED_BACKWARD, B, H, S, Q, dn, dr, dv, dt)
    ws = _workspace(nbytes, workspace, q.device)
    d = _dims(B, H, S, Q, dn, dr, dv, scale)
    st = lib.dflash_attn_anchored_backward(
        ctypes.byref(d), dt, _dev_ptr(q, "q"), _dev_ptr(k_nope, "k_nope", q.dtype), _dev_ptr(k_rope, "k_rope", q.dtype),
        _dev_ptr(v, "v", q.dtype), _dev_ptr(anchors, "anchors", torch.int32), nb, int(block_size),
        _dev_ptr(out, "out", q.dtype), _dev_ptr(lse, "lse", torch.float32), _dev_ptr(dout, "dout", q.dtype),
        _dev_ptr(dq, "dq"), _dev_ptr(dkn, "dk_nope"), _dev_ptr(dkr, "dk_rope"), _dev_ptr(dvv, "dv"),
        _dev_ptr(ws, "workspace"), nbytes, _stream(stream))
    _check("dflash_attn_anchored_backward", st)
    return dq, dkn, dkr, dvv


def dflash_attn_dense_backward(q, k_nope, k_rope, v, mask, out, lse, dout, grads=None, scale=0.0, workspace=None,
                               stream=None):
    """Gradients (dq, dk_nope, dk_rope, dv) of sum(dout * out) for the dense
    forward with additive mask [B,1,Q,S+Q] (the mask gets no gradient)."""
    torch = _torch()
    lib = load_library()
    B, H, S, Q, dn, dr, dv = _batched_shapes(q, k_nope, k_rope, v)
    dt = _dtype_code(q)
    if tuple(mask.shape) != (B, 1, Q, S + Q):
        raise ValueError("mask must be [B,1,Q,S+Q]")
    dq, dkn, dkr, dvv = _backward_grads(q, k_nope, k_rope, v, grads)
    nbytes = dflash_attn_workspace_size(MODE_DENSE_BACKWARD, B, H, S, Q, dn, dr, dv, dt)
    ws = _workspace(nbytes, workspace, q.device)
    d = _dims(B, H, S, Q, dn, dr, dv, scale)
    st = lib.dflash_attn_dense_backward(
        ctypes.byref(d), dt, _dev_ptr(q, "q"), _dev_ptr(k_nope, "k_nope", q.dtype), _dev_ptr(k_rope, "k_rope", q.dtype),
        _dev_ptr(v, "v", q.dtype), _dev_ptr(mask, "mask", q.dtype), _dev_ptr(out, "out", q.dtype),
        _dev_ptr(lse, "lse", torch.float32), _dev_ptr(dout, "dout", q.dtype), _dev_ptr(dq, "dq"),
        _dev_ptr(dkn, "dk_nope"), _dev_ptr(dkr, "dk_rope"), _dev_ptr(dvv, "dv"), _dev_ptr(ws, "workspace"), nbytes,
        _stream(stream))
    _check("dflash_attn_dense_backward", st)
    return dq, dkn, dkr, dvv


# ---------------------------------------------------------------------------
# the grouped-query draft's serving step
# ---------------------------------------------------------------------------
_binding_handle = None


def _binding():
    """The compiled module of the serving step's calls (built with the library); raises if absent.

    It is taken from the folder of the loaded library and links to the one there, so that all calls
    share one library with one error word, wherever load_library() found it."""
    global _binding_handle
    if _binding_handle is None:
        import importlib.util
        _torch()
        load_library()
        folder = os.path.dirname(_lib_path)
        path = os.path.join(folder, os.path.basename(_build.BINDING_PATH))
        beside = os.path.join(folder, os.path.basename(_build.LIB_PATH))
        if os.path.exists(path) and not (os.path.exists(beside) and os.path.samefile(beside, _lib_path)):
            raise RuntimeError(f"DFlash Python binding {path} belongs to {beside}, but {_lib_path} is loaded")
        if not os.path.exists(path):
            raise RuntimeError(f"DFlash Python binding not built ({path} missing): run "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        spec = importlib.util.spec_from_file_location("_dflash_binding", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _binding_handle = module
    return _binding_handle


def dflash_qk_norm_rope(q, k, positions, cos_sin, q_norm=None, k_norm=None, eps=1e-6, interleaved=False, q_out=None,
                        k_out=None, stream=None):
    """Norm (where a weight [D] is given) and rotation of q [T,H_q,D] and k
    [T,H_kv,D] at positions [T] int32.  Either of q and k may be None; their
    tokens may be strided.  cos_sin [max_pos, rot_dim] fp32 (rot_dim/2 cosines,
    then sines; None: no rotation).  Returns (q_out, k_out), contiguous."""
    r = (_binding_handle or _binding()).qk_norm_rope(q, k, positions, cos_sin, q_norm, k_norm, eps, interleaved, q_out,
                                                     k_out, stream)
    if r.__class__ is int:
        raise DFlashError("dflash_qk_norm_rope", r)
    return r


def dflash_qk_norm_rope_backward(q, k, positions, cos_sin, dq_out, dk_out, q_norm=None, k_norm=None, eps=1e-6,
                                 interleaved=False, grads=None, workspace=None, stream=None):
    """Gradients (dq, dk, dq_norm, dk_norm) of sum(dq_out * q_out) + sum(dk_out *
    k_out); the norm gradients are fp32 [D], None without a weight.  grads:
    optional preallocated (dq, dk, dq_norm, dk_norm)."""
    dq, dk, dwq, dwk = grads or (None, None, None, None)
    r = (_binding_handle or _binding()).qk_norm_rope_backward(q, k, positions, cos_sin, dq_out, dk_out, q_norm, k_norm,
                                                              eps, interleaved, dq, dk, dwq, dwk, workspace, stream)
    if r.__class__ is int:
        raise DFlashError("dflash_qk_norm_rope_backward", r)
    return r


def dflash_cache_append(k, v, k_cache, v_cache, page_table, kv_lens, q_offsets, q=None, cos_sin=None, q_norm=None,
                        k_norm=None, eps=1e-6, interleaved=False, q_out=None, stream=None):
    """Writes the new tokens' k (normed and rotated) and v [total_q,H_kv,D] into the
    pages of k_cache and v_cache [num_pages,page_size,H_kv,D]: request r's tokens
    [q_offsets[r], q_offsets[r+1]) are the last of its kv_lens[r] positions, and
    position p lies in page page_table[r, p // page_size].  With q [total_q,H_q,D]
    its heads are normed and rotated too; returns q_out (None without q)."""
    r = (_binding_handle or _binding()).cache_append(k, v, k_cache, v_cache, page_table, kv_lens, q_offsets, q,
                                                     cos_sin, q_norm, k_norm, eps, interleaved, q_out, stream)
    if r.__class__ is int:
        raise DFlashError("dflash_cache_append", r)
    return r


def dflash_attn_paged_workspace_size(H_q, H_kv, D, max_q_len, page_size, dtype=DFLASH_BF16) -> int:
    """Workspace bytes of dflash_attn_paged; they depend on neither the requests nor their lengths."""
    d = _PagedDims(1, H_q, H_kv, D, 1, int(max_q_len), 1, page_size, 1, 0, 0)
    return int(load_library().dflash_attn_paged_workspace_size(d, dtype))


def dflash_attn_paged(q, k_cache, v_cache, page_table, kv_lens, q_offsets, max_q_len, causal=True, out=None, lse=None,
                      scale=0.0, workspace=None, stream=None):
    """Attention of the new tokens q [total_q,H_q,D] over their requests' pages (see
    dflash_cache_append): all positions below kv_lens[r], or, causal, those up to
    the token's own.  Returns out [total_q,H_q,D]; fills lse [H_q,total_q] fp32 if given."""
    r = (_binding_handle or _binding()).attn_paged(q, k_cache, v_cache, page_table, kv_lens, q_offsets, max_q_len,
                                                   causal, out, lse, scale, workspace, stream)
    if r.__class__ is int:
        raise DFlashError("dflash_attn_paged", r)
    return r


def dflash_verify(target_probs, draft_probs, draft_tokens, draft_offsets, accept_u, sample_u, max_draft,
                  out_tokens=None, num_accepted=None, stream=None):
    """Accepts or replaces drafted tokens.  Request r drafted draft_tokens
    [draft_offsets[r], draft_offsets[r+1]) (int32) from draft_probs
    [total_draft, V] fp32 (None: it took its most likely token); target_probs fp32
    has its n + 1 rows from draft_offsets[r] + r on.  accept_u [total_draft] and
    sample_u [R] are fp32 in [0, 1).  Returns out_tokens [R, max_draft + 1] (the
    accepted tokens, the drawn one, then -1) and num_accepted [R], int32."""
    r = (_binding_handle or _binding()).verify(target_probs, draft_probs, draft_tokens, draft_offsets, accept_u,
                                               sample_u, max_draft, out_tokens, num_accepted, stream)
    if r.__class__ is int:
        raise DFlashError("dflash_verify", r)
    return r


def dflash_attn_tree(q, k_cache, v_cache, page_table, kv_lens, q_offsets, parents, max_q_len, out=None, lse=None,
                     scale=0.0, workspace=None, stream=None):
    """Attention of drafted trees: the new tokens of dflash_attn_paged are the nodes of a
    tree, each behind its parent parents [total_q] int32 (index within the request; -1: a
    root), and see the positions in front of the tree, themselves and their ancestors.
    All keys and values have to be finite, those that a node does not see too.  Workspace
    as dflash_attn_paged_workspace_size says."""
    r = (_binding_handle or _binding()).attn_tree(q, k_cache, v_cache, page_table, kv_lens, q_offsets, parents,
                                                  max_q_len, out, lse, scale, workspace, stream)
    if r.__class__ is int:
        raise DFlashError("dflash_attn_tree", r)
    return r


def dflash_sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, probs=None, tokens=None,
                  stream=None):
    """A token [N] int32 of every row of logits [N,V] (bf16 or fp32, rows may be
    strided) with given random numbers u [N] fp32 in [0, 1).  Per row, each optional:
    temperature [N] fp32 (0: the most likely token), top_k [N] int32 (<= 0: all), top_p
    [N] fp32 (>= 1: all), min_p [N] fp32 (<= 0: all), applied in this order.  Fills
    probs [N,V] fp32 with the distributions drawn from, if given."""
    r = (_binding_handle or _binding()).sample(logits, u, temperature, top_k, top_p, min_p, probs, tokens, stream)
    if r.__class__ is int:
        raise DFlashError("dflash_sample", r)
    return r


def dflash_tree_accept(sampled, tokens, parents, q_offsets, max_path, path=None, out_tokens=None, num_accepted=None,
                       stream=None):
    """Walks down every request's drafted tree (see dflash_attn_tree) from node 0 to the
    first child whose tokens [total] entry is the node's sampled [total] one, and so on, over
    at most max_path nodes.  Returns path [R,max_path] (the nodes, then -1),
    out_tokens [R,max_path] (the sampled tokens along it, then -1) and num_accepted [R]."""
    r = (_binding_handle or _binding()).tree_accept(sampled, tokens, parents, q_offsets, max_path, path, out_tokens,
                                                    num_accepted, stream)
    if r.__class__ is int:
        raise DFlashError("dflash_tree_accept", r)
    return r


def dflash_cache_compact(k_cache, v_cache, page_table, kv_lens, q_offsets, path, num_accepted, new_lens=None,
                         stream=None):
    """Moves the accepted nodes' keys and values together: with b the position of request
    r's first new token, position b + path[r, j] goes to b + j for j < num_accepted[r].
    k_cache and v_cache [num_pages,page_size,H_kv,D], or with an axis of layers in front.
    Returns the new lengths b + num_accepted."""
    r = (_binding_handle or _binding()).cache_compact(k_cache, v_cache, page_table, kv_lens, q_offsets, path,
                                                      num_accepted, new_lens, stream)
    if r.__class__ is int:
        raise DFlashError("dflash_cache_compact", r)
    return r


def dflash_cache_copy(k_cache, v_cache, src_pages, dst_pages, rows=None, stream=None):
    """Copies the first rows [n] positions (None: all) of pages src_pages [n] to pages
    dst_pages [n], int32; pairs with a -1 are left out.  Caches as for dflash_cache_compact."""
    r = (_binding_handle or _binding()).cache_copy(k_cache, v_cache, src_pages, dst_pages, rows, stream)
    if r is not None:
        raise DFlashError("dflash_cache_copy", r)


def dflash_pages_workspace_size(num_pages) -> int:
    """Workspace bytes of dflash_pages_resize and dflash_pages_fork."""
    return int(load_library().dflash_pages_workspace_size(_PoolDims(0, 0, 1, int(num_pages))))


def dflash_pages_resize(page_table, old_lens, new_lens, refs, page_size, missing=None, workspace=None, stream=None):
    """Gives back and takes pages so that row r of page_table [R,max_pages] holds
    ceil(new_lens[r] / page_size) of them where it held ceil(old_lens[r] / page_size).
    refs [num_pages] int32 counts the rows that hold a page, 0: free.  Returns
    missing [1]: pages that could not be had (their entries are -1)."""
    r = (_binding_handle or _binding()).pages_resize(page_table, old_lens, new_lens, refs, page_size, missing,
                                                     workspace, stream)
    if r.__class__ is int:
        raise DFlashError("dflash_pages_resize", r)
    return r


def dflash_pages_fork(page_table, lens, src, dst, refs, page_size, copy_src=None, copy_dst=None, copy_rows=None,
                      missing=None, workspace=None, stream=None):
    """Forks rows src [n] of page_table into the empty rows dst [n]: whole pages are
    shared, of the last one a page of its own is taken.  Updates lens [R]; returns
    copy_src, copy_dst, copy_rows [n], for dflash_cache_copy, and missing [1]."""
    r = (_binding_handle or _binding()).pages_fork(page_table, lens, src, dst, refs, page_size, copy_src, copy_dst,
                                                   copy_rows, missing, workspace, stream)
    if r.__class__ is int:
        raise DFlashError("dflash_pages_fork", r)
    return r


def dflash_build_schedule_host(B, S, Q, anchors, block_size) -> np.ndarray:
    """Host tile classes [B, ceil(Q/128), ceil((S+Q)/128)] of the anchored rule (numpy in, numpy out)."""
    lib = load_library()
    an = np.ascontiguousarray(anchors, np.int32)
    nb = an.shape[1] if an.ndim == 2 else 0
    out = np.zeros((B, -(-Q // TILE_M), -(-(S + Q) // TILE_N)), np.uint8)
    st = lib.dflash_build_schedule_host(B, S, Q, an.ctypes.data_as(ctypes.c_void_p), nb, int(block_size),
                                        out.ctypes.data_as(ctypes.c_void_p))
    _check("dflash_build_schedule_host", st)
    return out


def dflash_build_mask(anchors, block_size, S, dtype=None, mask=None, stream=None):
    """Device additive mask [B,1,Q,S+Q] (0 visible, -inf hidden) of the anchored
    rule from anchors [B,nb] int32 (CUDA).  dtype: torch.bfloat16 or torch.float32."""
    torch = _torch()
    lib = load_library()
    B, nb = anchors.shape
    Q = nb * int(block_size)
    dtype = dtype or torch.bfloat16
    if mask is None:
        mask = torch.empty((B, 1, Q, S + Q), dtype=dtype, device=anchors.device)
    st = lib.dflash_build_mask(B, S, Q, _dev_ptr(anchors, "anchors", torch.int32), nb, int(block_size),
                               _dtype_code(mask), _dev_ptr(mask, "mask"), _stream(stream))
    _check("dflash_build_mask", st)
    return mask


def dflash_scan_mask(mask, classes=None, stream=None):
    """Device tile classes of a dense mask [B,1,Q,S+Q]; returns a uint8 CUDA tensor."""
    torch = _torch()
    lib = load_library()
    B, _, Q, K = mask.shape
    S = K - Q
    if classes is None:
        classes = torch.empty((B, -(-Q // TILE_M), -(-K // TILE_N)), dtype=torch.uint8, device=mask.device)
    st = lib.dflash_scan_mask(B, S, Q, _dtype_code(mask), _dev_ptr(mask, "mask"),
                              _dev_ptr(classes, "classes", torch.uint8), _stream(stream))
    _check("dflash_scan_mask", st)
    return classes


def dflash_kernel_launches() -> int:
    """Kernels launched by the library in this process so far."""
    return int(load_library().dflash_kernel_launches())


def dflash_last_device_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error word."""
    return int(load_library().dflash_last_device_error(_stream(stream)))


def dflash_test_inject_stall(wait_budget_ns: int = 0, stall_cta: int = -1) -> None:
    """Test export: set the bounded-wait budget (0 = the 2 s default) and the CTA
    whose producer leaves its first work item's key tiles unloaded (-1 = none),
    for every later forward call in this process."""
    load_library().dflash_test_inject_stall(int(wait_budget_ns), int(stall_cta))


def dflash_test_limit_tile_flags(n: int = 0) -> None:
    """Test export: cap the backward kernels' shared-memory table of tile flags
    at n entries (0 = the full table), for every later call in this process."""
    load_library().dflash_test_limit_tile_flags(int(n))
