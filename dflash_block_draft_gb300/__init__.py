"""Python binding of the GB300 DFlash draft block-attention library.

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``libdflash_attn.so`` (C ABI in ``include/dflash_attn.h``).
PyTorch supplies device memory and the current stream.  There is no CPU
fallback: if the shared library has not been built, every call raises.

The functions carry the C names:
  dflash_attn_dense, dflash_attn_anchored, dflash_attn_ragged,
  dflash_attn_dense_backward, dflash_attn_anchored_backward,
  dflash_attn_workspace_size, dflash_build_schedule_host, dflash_scan_mask,
  dflash_last_device_error, dflash_status_string,
  dflash_qk_norm_rope, dflash_qk_norm_rope_backward, dflash_cache_append,
  dflash_attn_paged, dflash_verify.
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
           "dflash_cache_append", "dflash_attn_paged", "dflash_attn_paged_workspace_size", "dflash_verify")


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


_lock = threading.Lock()
_lib_handle = None


def load_library(path: str | None = None):
    """Load libdflash_attn.so (built by ``__graft_entry__.build()``); raises if absent."""
    global _lib_handle
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
        for name in ("dflash_qk_norm_rope", "dflash_qk_norm_rope_backward", "dflash_cache_append",
                     "dflash_attn_paged", "dflash_verify"):
            getattr(lib, name).restype = ctypes.c_int
        lib.dflash_qk_norm_rope_workspace_size.argtypes = [RD]
        lib.dflash_qk_norm_rope_workspace_size.restype = S
        lib.dflash_attn_paged_workspace_size.argtypes = [PD, I]
        lib.dflash_attn_paged_workspace_size.restype = S
        for name in ("dflash_attn_dense", "dflash_attn_anchored", "dflash_attn_ragged",
                     "dflash_build_schedule_host", "dflash_scan_mask", "dflash_last_device_error"):
            getattr(lib, name).restype = ctypes.c_int
        _lib_handle = lib
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
# These calls are short (a few microseconds on the device), so what the binding
# checks it checks with the cheapest tensor methods, and says what is wrong only
# once something is.
def _call(name, fn, index, stream, *args):
    """fn(*args, stream handle) with device `index` current; raises on a status."""
    torch = _torch()
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(index)
    else:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if torch._C._cuda_getDevice() == index:
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, handle)
    if rc:
        raise DFlashError(name, rc)


def _refuse(t, name, index, dtype, shape, form):
    if t.device.type != "cuda" or t.get_device() != index:
        raise ValueError(f"{name} must be a CUDA tensor" + (f" on device {index}" if index >= 0 else ""))
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous" if form is None else form)


def _arg(t, name, index, dtype, shape=None):
    """Data pointer of a contiguous tensor on CUDA device `index`, checked; None for None."""
    if t is None:
        return None
    if not (t.is_cuda and t.get_device() == index and t.dtype is dtype and t.is_contiguous() and
            (shape is None or t.shape == shape)):
        _refuse(t, name, index, dtype, shape, None)
    return t.data_ptr()


def _token_arg(t, name, index, dtype, shape):
    """Data pointer and token stride of [tokens, heads, D] whose tokens are each contiguous."""
    if t.is_cuda and t.get_device() == index and t.dtype is dtype and t.shape == shape:
        T, H, D = shape
        s0, s1, s2 = t.stride()
        if (s2 == 1 or D <= 1) and (s1 == D or H <= 1) and (s0 >= H * D or T <= 1):
            return t.data_ptr(), s0 if T > 1 else 0
    _refuse(t, name, index, dtype, shape, f"the heads of a token of {name} must be contiguous")


def _cache_arg(t, name, index, dtype, shape):
    """Data pointer and page stride of [pages, page_size, H_kv, D] whose pages are each contiguous."""
    if t.is_cuda and t.get_device() == index and t.dtype is dtype and t.shape == shape:
        n, P, H, D = shape
        s0, s1, s2, s3 = t.stride()
        if (s3 == 1 or D <= 1) and (s2 == D or H <= 1) and (s1 == H * D or P <= 1) and (s0 >= P * H * D or n <= 1):
            return t.data_ptr(), s0 if n > 1 else 0
    _refuse(t, name, index, dtype, shape, f"the pages of {name} must be contiguous")


def _rope_args(q, k, positions, cos_sin):
    torch = _torch()
    one = q if q is not None else k
    if one is None:
        raise ValueError("q or k must be given")
    if one.dim() != 3:
        raise ValueError("q and k must be [tokens, heads, D]")
    T, _, D = one.shape
    dev = one.get_device()
    Hq, Hk = 0 if q is None else q.shape[1], 0 if k is None else k.shape[1]
    if cos_sin is None:
        return one.dtype, dev, T, Hq, Hk, D, 0, 0, None, None
    if positions is None or cos_sin.dim() != 2:
        raise ValueError("cos_sin must be [max_pos, rot_dim] and comes with positions")
    max_pos, rot = cos_sin.shape
    cs = _arg(cos_sin, "cos_sin", dev, torch.float32)
    return one.dtype, dev, T, Hq, Hk, D, rot, max_pos, cs, _arg(positions, "positions", dev, torch.int32, (T,))


def dflash_qk_norm_rope(q, k, positions, cos_sin, q_norm=None, k_norm=None, eps=1e-6, interleaved=False, q_out=None,
                        k_out=None, stream=None):
    """Norm (where a weight [D] is given) and rotation of q [T,H_q,D] and k
    [T,H_kv,D] at positions [T] int32.  Either of q and k may be None; their
    tokens may be strided.  cos_sin [max_pos, rot_dim] fp32 (rot_dim/2 cosines,
    then sines; None: no rotation).  Returns (q_out, k_out), contiguous."""
    torch = _torch()
    lib = load_library()
    dt, dev, T, Hq, Hk, D, rot, max_pos, cs, ps = _rope_args(q, k, positions, cos_sin)
    code = _dtype_code(q if q is not None else k)
    qp, qs = (None, 0) if q is None else _token_arg(q, "q", dev, dt, (T, Hq, D))
    kp, ks = (None, 0) if k is None else _token_arg(k, "k", dev, dt, (T, Hk, D))
    if q is None:
        q_out = None
    elif q_out is None:
        q_out = torch.empty((T, Hq, D), dtype=dt, device=q.device)
    if k is None:
        k_out = None
    elif k_out is None:
        k_out = torch.empty((T, Hk, D), dtype=dt, device=k.device)
    d = _RopeDims(T, Hq, Hk, D, rot, max_pos, int(interleaved), eps, qs, ks)
    _call("dflash_qk_norm_rope", lib.dflash_qk_norm_rope, dev, stream, d, code, qp, kp,
          _arg(q_norm, "q_norm", dev, dt, (D,)), _arg(k_norm, "k_norm", dev, dt, (D,)), cs, ps,
          _arg(q_out, "q_out", dev, dt, (T, Hq, D)), _arg(k_out, "k_out", dev, dt, (T, Hk, D)))
    return q_out, k_out


def dflash_qk_norm_rope_backward(q, k, positions, cos_sin, dq_out, dk_out, q_norm=None, k_norm=None, eps=1e-6,
                                 interleaved=False, grads=None, workspace=None, stream=None):
    """Gradients (dq, dk, dq_norm, dk_norm) of sum(dq_out * q_out) + sum(dk_out *
    k_out); the norm gradients are fp32 [D], None without a weight.  grads:
    optional preallocated (dq, dk, dq_norm, dk_norm)."""
    torch = _torch()
    lib = load_library()
    dt, dev, T, Hq, Hk, D, rot, max_pos, cs, ps = _rope_args(q, k, positions, cos_sin)
    code = _dtype_code(q if q is not None else k)
    qp, qs = (None, 0) if q is None else _token_arg(q, "q", dev, dt, (T, Hq, D))
    kp, ks = (None, 0) if k is None else _token_arg(k, "k", dev, dt, (T, Hk, D))
    device = (q if q is not None else k).device
    if grads is None:
        grads = (None if q is None else torch.empty((T, Hq, D), dtype=dt, device=device),
                 None if k is None else torch.empty((T, Hk, D), dtype=dt, device=device),
                 None if q_norm is None else torch.empty(D, dtype=torch.float32, device=device),
                 None if k_norm is None else torch.empty(D, dtype=torch.float32, device=device))
    dq, dk, dwq, dwk = grads
    d = _RopeDims(T, Hq, Hk, D, rot, max_pos, int(interleaved), eps, qs, ks)
    nbytes = int(lib.dflash_qk_norm_rope_workspace_size(d))
    ws = _workspace(nbytes, workspace, device)
    _call("dflash_qk_norm_rope_backward", lib.dflash_qk_norm_rope_backward, dev, stream, d, code, qp, kp,
          _arg(q_norm, "q_norm", dev, dt, (D,)), _arg(k_norm, "k_norm", dev, dt, (D,)), cs, ps,
          _arg(dq_out if q is not None else None, "dq_out", dev, dt, (T, Hq, D)),
          _arg(dk_out if k is not None else None, "dk_out", dev, dt, (T, Hk, D)),
          _arg(dq, "dq", dev, dt, (T, Hq, D)), _arg(dk, "dk", dev, dt, (T, Hk, D)),
          _arg(dwq, "dq_norm", dev, torch.float32, (D,)), _arg(dwk, "dk_norm", dev, torch.float32, (D,)),
          _arg(ws, "workspace", dev, ws.dtype), nbytes)
    return dq, dk, dwq, dwk


def _paged_args(k_cache, v_cache, page_table, kv_lens, q_offsets, dt, dev):
    torch = _torch()
    shape = k_cache.shape
    if len(shape) != 4:
        raise ValueError("k_cache and v_cache must be [num_pages, page_size, H_kv, D]")
    kp, ks = _cache_arg(k_cache, "k_cache", dev, dt, shape)
    vp, vs = _cache_arg(v_cache, "v_cache", dev, dt, shape)
    if page_table.dim() != 2 or q_offsets.dim() != 1:
        raise ValueError("page_table must be [R, max_pages] and q_offsets [R + 1]")
    R, max_pages = page_table.shape
    tp = _arg(page_table, "page_table", dev, torch.int32)
    lp = _arg(kv_lens, "kv_lens", dev, torch.int32, (R,))
    op = _arg(q_offsets, "q_offsets", dev, torch.int32, (R + 1,))
    return shape, R, max_pages, kp, ks, vp, vs, tp, lp, op


def dflash_cache_append(k, v, k_cache, v_cache, page_table, kv_lens, q_offsets, q=None, cos_sin=None, q_norm=None,
                        k_norm=None, eps=1e-6, interleaved=False, q_out=None, stream=None):
    """Writes the new tokens' k (normed and rotated) and v [total_q,H_kv,D] into the
    pages of k_cache and v_cache [num_pages,page_size,H_kv,D]: request r's tokens
    [q_offsets[r], q_offsets[r+1]) are the last of its kv_lens[r] positions, and
    position p lies in page page_table[r, p // page_size].  With q [total_q,H_q,D]
    its heads are normed and rotated too; returns q_out (None without q)."""
    torch = _torch()
    lib = load_library()
    dt, dev = k.dtype, k.get_device()
    code = _dtype_code(k)
    (n, P, Hk, D), R, max_pages, kcp, kcs, vcp, vcs, tp, lp, op = _paged_args(k_cache, v_cache, page_table, kv_lens,
                                                                              q_offsets, dt, dev)
    T = k.shape[0]
    kp, ks = _token_arg(k, "k", dev, dt, (T, Hk, D))
    vp, vs = _token_arg(v, "v", dev, dt, (T, Hk, D))
    Hq, qp, qs = Hk, None, 0
    if q is not None:
        if q.dim() != 3:
            raise ValueError("q must be [total_q, H_q, D]")
        Hq = q.shape[1]
        qp, qs = _token_arg(q, "q", dev, dt, (T, Hq, D))
        if q_out is None:
            q_out = torch.empty((T, Hq, D), dtype=dt, device=q.device)
    else:
        q_out = None
    max_pos, rot = (0, 0) if cos_sin is None else cos_sin.shape
    pd = _PagedDims(R, Hq, Hk, D, T, 0, n, P, max_pages, kcs, vcs)
    rd = _RopeDims(T, Hq, Hk, D, rot, max_pos, int(interleaved), eps, qs, ks)
    _call("dflash_cache_append", lib.dflash_cache_append, dev, stream, pd, rd, code, qp, kp, vp, vs,
          _arg(q_norm, "q_norm", dev, dt, (D,)), _arg(k_norm, "k_norm", dev, dt, (D,)),
          _arg(cos_sin, "cos_sin", dev, torch.float32), tp, lp, op, _arg(q_out, "q_out", dev, dt, (T, Hq, D)), kcp,
          vcp)
    return q_out


def dflash_attn_paged_workspace_size(H_q, H_kv, D, max_q_len, page_size, dtype=DFLASH_BF16) -> int:
    """Workspace bytes of dflash_attn_paged; they depend on neither the requests nor their lengths."""
    d = _PagedDims(1, H_q, H_kv, D, 1, int(max_q_len), 1, page_size, 1, 0, 0)
    return int(load_library().dflash_attn_paged_workspace_size(d, dtype))


def dflash_attn_paged(q, k_cache, v_cache, page_table, kv_lens, q_offsets, max_q_len, causal=True, out=None, lse=None,
                      scale=0.0, workspace=None, stream=None):
    """Attention of the new tokens q [total_q,H_q,D] over their requests' pages (see
    dflash_cache_append): all positions below kv_lens[r], or, causal, those up to
    the token's own.  Returns out [total_q,H_q,D]; fills lse [H_q,total_q] fp32 if given."""
    torch = _torch()
    lib = load_library()
    dt, dev = q.dtype, q.get_device()
    code = _dtype_code(q)
    if q.dim() != 3:
        raise ValueError("q must be [total_q, H_q, D]")
    T, Hq, _ = q.shape
    (n, P, Hk, D), R, max_pages, kcp, kcs, vcp, vcs, tp, lp, op = _paged_args(k_cache, v_cache, page_table, kv_lens,
                                                                              q_offsets, dt, dev)
    qp = _arg(q, "q", dev, dt, (T, Hq, D))
    if out is None:
        out = torch.empty((T, Hq, D), dtype=dt, device=q.device)
    d = _PagedDims(R, Hq, Hk, D, T, int(max_q_len), n, P, max_pages, kcs, vcs)
    nbytes = lib.dflash_attn_paged_workspace_size(d, code)
    ws = _workspace(nbytes, workspace, q.device)
    _call("dflash_attn_paged", lib.dflash_attn_paged, dev, stream, d, code, qp, kcp, vcp, tp, lp, op, int(causal),
          float(scale or 0.0), _arg(out, "out", dev, dt, (T, Hq, D)),
          _arg(lse, "lse", dev, torch.float32, (Hq, T)), _arg(ws, "workspace", dev, ws.dtype), nbytes)
    return out


def dflash_verify(target_probs, draft_probs, draft_tokens, draft_offsets, accept_u, sample_u, max_draft,
                  out_tokens=None, num_accepted=None, stream=None):
    """Accepts or replaces drafted tokens.  Request r drafted draft_tokens
    [draft_offsets[r], draft_offsets[r+1]) (int32) from draft_probs
    [total_draft, V] fp32 (None: it took its most likely token); target_probs fp32
    has its n + 1 rows from draft_offsets[r] + r on.  accept_u [total_draft] and
    sample_u [R] are fp32 in [0, 1).  Returns out_tokens [R, max_draft + 1] (the
    accepted tokens, the drawn one, then -1) and num_accepted [R], int32."""
    torch = _torch()
    lib = load_library()
    dev, f32, i32 = target_probs.get_device(), torch.float32, torch.int32
    if target_probs.dim() != 2 or target_probs.stride(1) != 1 or draft_offsets.dim() != 1:
        raise ValueError("target_probs must be [rows, V] with contiguous rows, draft_offsets [R + 1]")
    rows, V = target_probs.shape
    T, R = draft_tokens.shape[0], draft_offsets.shape[0] - 1
    if rows < T + R:
        raise ValueError("target_probs needs a row for every drafted token and one more for every request")
    if not target_probs.is_cuda or target_probs.dtype is not f32:
        raise ValueError("target_probs must be a float32 CUDA tensor")
    ps, qp, qs = target_probs.stride(0) if rows > 1 else 0, None, 0
    if draft_probs is not None:
        if (draft_probs.shape != (T, V) or draft_probs.dtype is not f32 or draft_probs.get_device() != dev or
                (V > 1 and draft_probs.stride(1) != 1)):
            raise ValueError("draft_probs must be a float32 [total_draft, V] tensor with contiguous rows on the "
                             "device of target_probs")
        if T > 0:
            qp, qs = draft_probs.data_ptr(), draft_probs.stride(0) if T > 1 else 0
    if out_tokens is None:
        out_tokens = torch.empty((R, max_draft + 1), dtype=i32, device=target_probs.device)
    if num_accepted is None:
        num_accepted = torch.empty(R, dtype=i32, device=target_probs.device)
    d = _VerifyDims(R, V, T, int(max_draft), ps, qs)
    _call("dflash_verify", lib.dflash_verify, dev, stream, d, target_probs.data_ptr(), qp,
          _arg(draft_tokens, "draft_tokens", dev, i32, (T,)), _arg(draft_offsets, "draft_offsets", dev, i32),
          _arg(accept_u, "accept_u", dev, f32, (T,)), _arg(sample_u, "sample_u", dev, f32, (R,)),
          _arg(out_tokens, "out_tokens", dev, i32, (R, max_draft + 1)),
          _arg(num_accepted, "num_accepted", dev, i32, (R,)))
    return out_tokens, num_accepted


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
