"""Thin ctypes binding over libmaxsim.so, with the C entry points' names.

Only argument marshalling happens here: tensors become device pointers, the
current torch stream becomes the hipStream_t, and a non-zero status becomes a
``MaxSimError``.  Every step of the computation runs in the HIP kernels; there
is no CPU fallback: if the library was not built, importing this module raises.
PyTorch is used for device memory (outputs the caller does not pass are
allocated with torch) and streams.
"""
import ctypes
import functools
import os
import types
import warnings

import numpy as np
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmaxsim.so")

MAXSIM_OK = 0
MAXSIM_ERR_NULL = 1
MAXSIM_ERR_SHAPE = 2
MAXSIM_ERR_UNSUPPORTED = 3
MAXSIM_ERR_ALIGN = 4
MAXSIM_ERR_WORKSPACE = 5
MAXSIM_ERR_HIP = 6
MAXSIM_ERR_SCRATCH = 7
MAXSIM_F16 = 0
MAXSIM_BF16 = 1
MAXSIM_F32 = 2
MAXSIM_I8 = 3
MAXSIM_E4M3 = 4
QBLOCK = 128  # values that share a scale

# name -> (restype, argtypes); must match include/maxsim.h and include/maxsim_encoder.h
_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_F32 = ctypes.c_float
_F64 = ctypes.c_double
SIGNATURES = {
    "maxsim_fwd": (ctypes.c_int, [_P, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32, _P, _P, _P]),
    "maxsim_fwd_varlen": (ctypes.c_int, [_P, _P, _P, _I32, _I32, _I32, _I64, _I32, _I32, _I32, _P, _P, _P]),
    "maxsim_fwd_i8": (ctypes.c_int, [_P, _P, _P, _P, _P, _I32, _I32, _I32, _I64, _I32, _I32, _P, _P, _P]),
    "maxsim_bwd_workspace_bytes": (ctypes.c_size_t, [_I32, _I32, _I32, _I32]),
    "maxsim_bwd": (ctypes.c_int, [_P, _P, _I32, _P, _P, _I32, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P,
                                  ctypes.c_size_t, _P]),
    "maxsim_bwd_noalloc_scratch_bytes": (ctypes.c_size_t, []),
    "maxsim_bwd_noalloc": (ctypes.c_int, [_P, _P, _I32, _P, _P, _I32, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P]),
    "maxsim_bwd_varlen_workspace_bytes": (ctypes.c_size_t, [_I32, _I32, _I32, _I32]),
    "maxsim_bwd_varlen": (ctypes.c_int, [_P, _P, _P, _I32, _P, _P, _I32, _I32, _I32, _I64, _I32, _I32, _P, _P,
                                         _P, _P, _P, ctypes.c_size_t, _P]),
    "maxsim_bwd_scatter_workspace_bytes": (ctypes.c_size_t, [_I32, _I32, _I32]),
    "maxsim_bwd_scatter": (ctypes.c_int, [_P, _P, _P, _I32, _P, _P, _I32, _I32, _I32, _I32, _I64, _I32, _P, _P,
                                          _P, ctypes.c_size_t, _P]),
    "maxsim_bwd_prefer_scatter": (ctypes.c_int, [_I32, _I32, _I32, _I64]),
    "maxsim_fwd_host_stream_staging_bytes": (ctypes.c_size_t, [_I32, _I32, _I32, _I32, _I32]),
    "maxsim_fwd_host_stream": (ctypes.c_int, [_P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _P,
                                              ctypes.c_size_t, _P, _P, _P]),
    "maxsim_chamfer_fwd_workspace_bytes": (ctypes.c_size_t, [_I32, _I32, _I32]),
    "maxsim_chamfer_fwd": (ctypes.c_int, [_P, _P, _I32, _I32, _I32, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "maxsim_chamfer_bwd_workspace_bytes": (ctypes.c_size_t, [_I32, _I32, _I32]),
    "maxsim_chamfer_bwd": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _P,
                                          ctypes.c_size_t, _P]),
    "maxsim_fwd_pairs": (ctypes.c_int, [_P, _P, _P, _I32, _P, _P, _I32, _I32, _I32, _I32, _I64, _I32, _P, _P, _P]),
    "maxsim_topk": (ctypes.c_int, [_P, _P, _I32, _I32, _I32, _P, _P, _P]),
    "maxsim_two_stage_workspace_bytes": (ctypes.c_size_t, [_I32, _I32, _I32]),
    "maxsim_two_stage_topk": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _I64, _I32, _I32,
                                             _I32, _I32, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "maxsim_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "maxsim_rmsnorm_fwd": (ctypes.c_int, [_P, _I64, _P, _I64, _P, _I32, _I32, _I32, _I32, _F32, _I32, _P, _I64, _P,
                                          _P, _I64, _P, _P]),
    "maxsim_rmsnorm_bwd_workspace_bytes": (ctypes.c_size_t, [_I32, _I32]),
    "maxsim_rmsnorm_bwd": (ctypes.c_int, [_P, _I64, _P, _I64, _P, _P, _I32, _P, _I64, _I32, _I32, _I32, _P, _I64, _P,
                                          _P, ctypes.c_size_t, _P]),
    "maxsim_quant_fp8": (ctypes.c_int, [_P, _I64, _I32, _I32, _I32, _I32, _P, _I64, _P, _P, _I64, _P, _P]),
    "maxsim_gemm_fp8_workspace_bytes": (ctypes.c_size_t, [_I32, _I32, _I32]),
    "maxsim_gemm_fp8": (ctypes.c_int, [_P, _I64, _P, _P, _I64, _P, _I32, _I32, _I32, _I32, _I32, _P, _I64, _P,
                                       ctypes.c_size_t, _P]),
    "maxsim_adamw": (ctypes.c_int, [_P, _I32, _I32, _I32, _I32, _F64, _F64, _F64, _F64, _F64, _I32, _P, _P]),
}


class MaxSimError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = lib().maxsim_status_string(status).decode()
        super().__init__("%s: %s (status %d)" % (where, msg, status))


_lib = None


def lib():
    """The loaded libmaxsim.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libmaxsim.so is not built; run `python -m late_interaction_retrieval_amd.build` "
                              "(or __graft_entry__.build())")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(l, name)
            f.restype = res
            f.argtypes = args
        _lib = l
    return _lib


lib()  # fail loudly at import time if the native library is missing
try:  # the usual calls of the embedding head's operators, natively (fast_binding.cpp)
    from . import _fast
except ImportError as e:  # not built, or built against another torch: all of them go through ctypes
    warnings.warn("late_interaction_retrieval_amd: no _fast.so (%s): calls take some microseconds more" % e, RuntimeWarning)
    _fast = types.SimpleNamespace(**{name: lambda *args: None for name in ("rmsnorm_fwd", "rmsnorm_bwd", "quant_fp8",
                                                                         "gemm_fp8", "adamw")})


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t, stream):
    if stream is None:
        stream = torch.cuda.current_stream(t.device)
    return ctypes.c_void_p(stream.cuda_stream)


def _check(status, where):
    if status != MAXSIM_OK:
        raise MaxSimError(status, where)


def _dtype_code(t):
    if t.dtype == torch.float16:
        return MAXSIM_F16
    if t.dtype == torch.bfloat16:
        return MAXSIM_BF16
    raise TypeError("Q and D must be float16 or bfloat16, got %s" % t.dtype)


def _need(t, name, dtype=None, device=None):
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))


def maxsim_fwd(Q, D, d_lens=None, scores=None, argmax=None, with_argmax=True, stream=None):
    """Padded forward.  Q [Nq, Lq, 128], D [B, Ld, 128] (fp16/bf16), d_lens [B] int32 or None.

    Returns (scores [Nq, B] fp32, argmax [Nq, B, Lq] int32 or None).
    """
    Nq, Lq, d = Q.shape
    B, Ld, d2 = D.shape
    if d2 != d or Q.dtype != D.dtype:
        raise ValueError("Q and D must share dtype and width")
    _need(Q, "Q")
    _need(D, "D", device=Q.device)
    if d_lens is not None:
        _need(d_lens, "d_lens", torch.int32, Q.device)
    if scores is None:
        scores = torch.empty((Nq, B), dtype=torch.float32, device=Q.device)
    _need(scores, "scores", torch.float32, Q.device)
    if argmax is None and with_argmax:
        argmax = torch.empty((Nq, B, Lq), dtype=torch.int32, device=Q.device)
    if argmax is not None:
        _need(argmax, "argmax", torch.int32, Q.device)
    st = lib().maxsim_fwd(_ptr(Q), _ptr(D), _ptr(d_lens), Nq, Lq, B, Ld, d, _dtype_code(Q),
                          _ptr(scores), _ptr(argmax), _stream(Q, stream))
    _check(st, "maxsim_fwd")
    return scores, argmax


def maxsim_fwd_varlen(Q, D_packed, cu_seqlens, max_Ld, scores=None, argmax=None, with_argmax=True,
                      stream=None):
    """Padding-free forward.  D_packed [T, 128], cu_seqlens [B+1] int32 on the device."""
    Nq, Lq, d = Q.shape
    T, d2 = D_packed.shape
    B = cu_seqlens.shape[0] - 1
    if d2 != d or Q.dtype != D_packed.dtype:
        raise ValueError("Q and D_packed must share dtype and width")
    _need(Q, "Q")
    _need(D_packed, "D_packed", device=Q.device)
    _need(cu_seqlens, "cu_seqlens", torch.int32, Q.device)
    if scores is None:
        scores = torch.empty((Nq, B), dtype=torch.float32, device=Q.device)
    _need(scores, "scores", torch.float32, Q.device)
    if argmax is None and with_argmax:
        argmax = torch.empty((Nq, B, Lq), dtype=torch.int32, device=Q.device)
    if argmax is not None:
        _need(argmax, "argmax", torch.int32, Q.device)
    st = lib().maxsim_fwd_varlen(_ptr(Q), _ptr(D_packed), _ptr(cu_seqlens), Nq, Lq, B, T, int(max_Ld), d,
                                 _dtype_code(Q), _ptr(scores), _ptr(argmax), _stream(Q, stream))
    _check(st, "maxsim_fwd_varlen")
    return scores, argmax


def maxsim_fwd_i8(Q, q_scale, D_packed, d_scale, cu_seqlens, max_Ld, scores=None, argmax=None,
                  with_argmax=True, stream=None):
    """INT8 x INT8 padding-free forward (int8 rows, fp32 per-token scales)."""
    Nq, Lq, d = Q.shape
    T, d2 = D_packed.shape
    B = cu_seqlens.shape[0] - 1
    if d2 != d:
        raise ValueError("Q and D_packed must share the width")
    _need(Q, "Q", torch.int8)
    _need(D_packed, "D_packed", torch.int8, Q.device)
    _need(q_scale, "q_scale", torch.float32, Q.device)
    _need(d_scale, "d_scale", torch.float32, Q.device)
    _need(cu_seqlens, "cu_seqlens", torch.int32, Q.device)
    if scores is None:
        scores = torch.empty((Nq, B), dtype=torch.float32, device=Q.device)
    _need(scores, "scores", torch.float32, Q.device)
    if argmax is None and with_argmax:
        argmax = torch.empty((Nq, B, Lq), dtype=torch.int32, device=Q.device)
    if argmax is not None:
        _need(argmax, "argmax", torch.int32, Q.device)
    st = lib().maxsim_fwd_i8(_ptr(Q), _ptr(q_scale), _ptr(D_packed), _ptr(d_scale), _ptr(cu_seqlens), Nq, Lq,
                             B, T, int(max_Ld), d, _ptr(scores), _ptr(argmax), _stream(Q, stream))
    _check(st, "maxsim_fwd_i8")
    return scores, argmax


def maxsim_bwd_workspace_bytes(Nq, B, Lq, Ld):
    return int(lib().maxsim_bwd_workspace_bytes(Nq, B, Lq, Ld))


def maxsim_bwd(Q, D, argmax, grad_scores, dQ=None, dD=None, row_ptr=None, col_idx=None, workspace=None,
               stream=None):
    """Backward over padded documents.  Returns (dQ, dD, row_ptr, col_idx)."""
    Nq, Lq, d = Q.shape
    B, Ld, _ = D.shape
    dev = Q.device
    _need(Q, "Q")
    _need(D, "D", device=dev)
    _need(argmax, "argmax", torch.int32, dev)
    _need(grad_scores, "grad_scores", torch.float32, dev)
    if dQ is None:
        dQ = torch.empty((Nq, Lq, d), dtype=torch.float32, device=dev)
    if dD is None:
        dD = torch.empty((B, Ld, d), dtype=torch.float32, device=dev)
    if row_ptr is None:
        row_ptr = torch.empty(B * Ld + 1, dtype=torch.int32, device=dev)
    if col_idx is None:
        col_idx = torch.empty(Nq * B * Lq, dtype=torch.int32, device=dev)
    nbytes = maxsim_bwd_workspace_bytes(Nq, B, Lq, Ld)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
    for t, n in ((dQ, "dQ"), (dD, "dD"), (row_ptr, "row_ptr"), (col_idx, "col_idx"), (workspace, "workspace")):
        _need(t, n, device=dev)
    st = lib().maxsim_bwd(_ptr(Q), _ptr(D), _dtype_code(Q), _ptr(argmax), _ptr(grad_scores), Nq, Lq, B, Ld, d,
                          _ptr(dQ), _ptr(dD), _ptr(row_ptr), _ptr(col_idx), _ptr(workspace),
                          workspace.numel() * workspace.element_size(), _stream(Q, stream))
    _check(st, "maxsim_bwd")
    return dQ, dD, row_ptr, col_idx


def maxsim_bwd_noalloc(Q, D, argmax, grad_scores, dQ, dD, row_ptr, col_idx, stream=None):
    """maxsim_bwd without a workspace and without allocating: the library's own
    per-device scratch array serves as the workspace, and every output is the
    caller's.  Returns (dQ, dD, row_ptr, col_idx)."""
    Nq, Lq, d = Q.shape
    B, Ld, _ = D.shape
    dev = Q.device
    _need(Q, "Q")
    _need(D, "D", device=dev)
    _need(argmax, "argmax", torch.int32, dev)
    _need(grad_scores, "grad_scores", torch.float32, dev)
    for t, n, dt, numel in ((dQ, "dQ", torch.float32, Nq * Lq * d), (dD, "dD", torch.float32, B * Ld * d),
                            (row_ptr, "row_ptr", torch.int32, B * Ld + 1),
                            (col_idx, "col_idx", torch.int32, Nq * B * Lq)):
        _need(t, n, dt, dev)
        if t.numel() < numel:
            raise ValueError("%s holds %d elements, needs %d" % (n, t.numel(), numel))
    st = lib().maxsim_bwd_noalloc(_ptr(Q), _ptr(D), _dtype_code(Q), _ptr(argmax), _ptr(grad_scores), Nq, Lq, B, Ld,
                                  d, _ptr(dQ), _ptr(dD), _ptr(row_ptr), _ptr(col_idx), _stream(Q, stream))
    _check(st, "maxsim_bwd_noalloc")
    return dQ, dD, row_ptr, col_idx


def maxsim_bwd_varlen_workspace_bytes(Nq, B, Lq, max_Ld):
    return int(lib().maxsim_bwd_varlen_workspace_bytes(Nq, B, Lq, max_Ld))


def maxsim_bwd_varlen(Q, D_packed, cu_seqlens, max_Ld, argmax, grad_scores, dQ=None, dD=None, row_ptr=None,
                      col_idx=None, workspace=None, stream=None):
    """Backward over a packed corpus.  Returns (dQ [Nq, Lq, d], dD [T, d], row_ptr [T+1], col_idx
    [Nq*B*Lq], of which the first row_ptr[T] entries are defined)."""
    Nq, Lq, d = Q.shape
    T, d2 = D_packed.shape
    B = cu_seqlens.shape[0] - 1
    if d2 != d or Q.dtype != D_packed.dtype:
        raise ValueError("Q and D_packed must share dtype and width")
    dev = Q.device
    _need(Q, "Q")
    _need(D_packed, "D_packed", device=dev)
    _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
    _need(argmax, "argmax", torch.int32, dev)
    _need(grad_scores, "grad_scores", torch.float32, dev)
    if dQ is None:
        dQ = torch.empty((Nq, Lq, d), dtype=torch.float32, device=dev)
    if dD is None:
        dD = torch.empty((T, d), dtype=torch.float32, device=dev)
    if row_ptr is None:
        row_ptr = torch.empty(T + 1, dtype=torch.int32, device=dev)
    if col_idx is None:
        col_idx = torch.empty(Nq * B * Lq, dtype=torch.int32, device=dev)
    nbytes = maxsim_bwd_varlen_workspace_bytes(Nq, B, Lq, int(max_Ld))
    if workspace is None:
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
    for t, n in ((dQ, "dQ"), (dD, "dD"), (row_ptr, "row_ptr"), (col_idx, "col_idx"), (workspace, "workspace")):
        _need(t, n, device=dev)
    st = lib().maxsim_bwd_varlen(_ptr(Q), _ptr(D_packed), _ptr(cu_seqlens), _dtype_code(Q), _ptr(argmax),
                                 _ptr(grad_scores), Nq, Lq, B, T, int(max_Ld), d, _ptr(dQ), _ptr(dD), _ptr(row_ptr),
                                 _ptr(col_idx), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream(Q, stream))
    _check(st, "maxsim_bwd_varlen")
    return dQ, dD, row_ptr, col_idx


def maxsim_bwd_prefer_scatter(Nq, Lq, B, rows):
    return bool(lib().maxsim_bwd_prefer_scatter(Nq, Lq, B, rows))


def maxsim_bwd_scatter_workspace_bytes(Nq, B, Lq):
    return int(lib().maxsim_bwd_scatter_workspace_bytes(Nq, B, Lq))


def maxsim_bwd_scatter(Q, D, argmax, grad_scores, cu_seqlens=None, max_Ld=None, dQ=None, dD=None, workspace=None,
                       stream=None):
    """Backward with dD by atomic scatter (no CSR).  D is [B, Ld, d] (padded) or, with cu_seqlens,
    D_packed [T, d] with max_Ld the longest document.  Returns (dQ, dD)."""
    Nq, Lq, d = Q.shape
    dev = Q.device
    _need(Q, "Q")
    _need(D, "D", device=dev)
    _need(argmax, "argmax", torch.int32, dev)
    _need(grad_scores, "grad_scores", torch.float32, dev)
    if D.dtype != Q.dtype or D.shape[-1] != d:
        raise ValueError("Q and D must share dtype and width")
    if cu_seqlens is None:
        B, Ld, _ = D.shape
        T = 0
    else:
        _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
        B = cu_seqlens.shape[0] - 1
        T = D.shape[0]
        Ld = int(max_Ld)
    if dQ is None:
        dQ = torch.empty((Nq, Lq, d), dtype=torch.float32, device=dev)
    if dD is None:
        dD = torch.empty(D.shape, dtype=torch.float32, device=dev)
    _need(dQ, "dQ", torch.float32, dev)
    _need(dD, "dD", torch.float32, dev)
    if workspace is None:
        workspace = torch.empty(max(256, maxsim_bwd_scatter_workspace_bytes(Nq, B, Lq)), dtype=torch.uint8,
                                device=dev)
    _need(workspace, "workspace", device=dev)
    st = lib().maxsim_bwd_scatter(_ptr(Q), _ptr(D), _ptr(cu_seqlens), _dtype_code(Q), _ptr(argmax),
                                  _ptr(grad_scores), Nq, Lq, B, Ld, T, d, _ptr(dQ), _ptr(dD), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream(Q, stream))
    _check(st, "maxsim_bwd_scatter")
    return dQ, dD


class MaxSimFunction(torch.autograd.Function):
    """score = MaxSim(Q, D) as an autograd op: the forward saves the argmax and the
    backward builds the inverse-grid CSR and the gradients (paper Section 4.2).
    With deterministic=False the backward may take the atomic-scatter dD instead,
    where the dispatch rule (maxsim_bwd_prefer_scatter) expects it to be faster."""

    @staticmethod
    def forward(ctx, Q, D, cu_seqlens, max_Ld, deterministic):
        if cu_seqlens is None:
            scores, argmax = maxsim_fwd(Q, D)
        else:
            scores, argmax = maxsim_fwd_varlen(Q, D, cu_seqlens, max_Ld)
        ctx.save_for_backward(Q, D, argmax, cu_seqlens)
        ctx.max_Ld = max_Ld
        ctx.deterministic = deterministic
        return scores

    @staticmethod
    def backward(ctx, grad_scores):
        Q, D, argmax, cu = ctx.saved_tensors
        g = grad_scores.float().contiguous()
        Nq, Lq, _ = Q.shape
        B = argmax.shape[1]
        rows = D.shape[0] * D.shape[1] if cu is None else D.shape[0]
        if not ctx.deterministic and maxsim_bwd_prefer_scatter(Nq, Lq, B, rows):
            dQ, dD = maxsim_bwd_scatter(Q, D, argmax, g, cu_seqlens=cu, max_Ld=ctx.max_Ld)
        elif cu is None:
            dQ, dD, _, _ = maxsim_bwd(Q, D, argmax, g)
        else:
            dQ, dD, _, _ = maxsim_bwd_varlen(Q, D, cu, ctx.max_Ld, argmax, g)
        return dQ.to(Q.dtype), dD.to(D.dtype), None, None, None


def maxsim(Q, D, cu_seqlens=None, max_Ld=None, deterministic=True):
    """MaxSim scores [Nq, B] of every query against every document, with autograd
    support.  D is [B, Ld, d], or packed [T, d] with cu_seqlens [B+1] and max_Ld."""
    if cu_seqlens is not None and max_Ld is None:
        raise ValueError("max_Ld is required with cu_seqlens")
    return MaxSimFunction.apply(Q, D, cu_seqlens, max_Ld, deterministic)


def maxsim_fwd_host_stream_staging_bytes(Nq, Lq, Ld, block_docs, with_argmax):
    return int(lib().maxsim_fwd_host_stream_staging_bytes(Nq, Lq, Ld, block_docs, int(bool(with_argmax))))


def maxsim_fwd_host_stream(Q, D_host, block_docs, cu_seqlens_host=None, cu_seqlens=None, max_Ld=None, d_lens=None,
                           scores=None, argmax=None, with_argmax=False, staging=None, stream=None):
    """Score a corpus held in host memory (a CPU tensor, pinned for full speed) block by block.
    Padded: D_host [B, Ld, 128].  Packed: D_host [T, 128], cu_seqlens_host (CPU int32 [B+1]),
    cu_seqlens (the same on the device) and max_Ld.  Returns (scores [Nq, B], argmax or None).
    The copies run after this returns: keep D_host alive until the stream has finished."""
    Nq, Lq, d = Q.shape
    dev = Q.device
    _need(Q, "Q")
    if D_host.is_cuda or not D_host.is_contiguous():
        raise ValueError("D_host must be a contiguous host tensor")
    if D_host.dtype != Q.dtype or D_host.shape[-1] != d:
        raise ValueError("Q and D_host must share dtype and width")
    if cu_seqlens_host is None:
        B, Ld, _ = D_host.shape
    else:
        if cu_seqlens_host.is_cuda or cu_seqlens_host.dtype != torch.int32 or not cu_seqlens_host.is_contiguous():
            raise ValueError("cu_seqlens_host must be a contiguous host int32 tensor")
        if cu_seqlens is None or max_Ld is None:
            raise ValueError("a packed corpus needs cu_seqlens on the device and max_Ld")
        _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
        B = cu_seqlens_host.shape[0] - 1
        Ld = int(max_Ld)
    if d_lens is not None:
        _need(d_lens, "d_lens", torch.int32, dev)
    if scores is None:
        scores = torch.empty((Nq, B), dtype=torch.float32, device=dev)
    _need(scores, "scores", torch.float32, dev)
    if argmax is None and with_argmax:
        argmax = torch.empty((Nq, B, Lq), dtype=torch.int32, device=dev)
    if argmax is not None:
        _need(argmax, "argmax", torch.int32, dev)
    nbytes = maxsim_fwd_host_stream_staging_bytes(Nq, Lq, Ld, block_docs, argmax is not None)
    if staging is None:
        staging = torch.empty(max(256, nbytes), dtype=torch.uint8, device=dev)
    _need(staging, "staging", device=dev)
    st = lib().maxsim_fwd_host_stream(_ptr(Q), ctypes.c_void_p(D_host.data_ptr()),
                                      None if cu_seqlens_host is None else ctypes.c_void_p(cu_seqlens_host.data_ptr()),
                                      _ptr(cu_seqlens), _ptr(d_lens), Nq, Lq, B, Ld, d, _dtype_code(Q),
                                      int(block_docs), _ptr(staging), staging.numel(), _ptr(scores), _ptr(argmax),
                                      _stream(Q, stream))
    _check(st, "maxsim_fwd_host_stream")
    return scores, argmax


def _clouds(P, Q):
    if P.dim() == 2:
        P = P.unsqueeze(0)
    if Q.dim() == 2:
        Q = Q.unsqueeze(0)
    _need(P, "P", torch.float32)
    _need(Q, "Q", torch.float32, P.device)
    if P.shape[0] != Q.shape[0] or P.shape[2] != 3 or Q.shape[2] != 3:
        raise ValueError("P [Bt, N, 3] and Q [Bt, M, 3] must share Bt")
    return P, Q


def maxsim_chamfer_fwd(P, Q, workspace=None, stream=None):
    """Nearest neighbours both ways between P [Bt, N, 3] and Q [Bt, M, 3] (fp32):
    (dist_p [Bt, N], idx_p, dist_q [Bt, M], idx_q); squared distances."""
    P, Q = _clouds(P, Q)
    Bt, N, _ = P.shape
    M = Q.shape[1]
    dev = P.device
    dist_p = torch.empty((Bt, N), dtype=torch.float32, device=dev)
    idx_p = torch.empty((Bt, N), dtype=torch.int32, device=dev)
    dist_q = torch.empty((Bt, M), dtype=torch.float32, device=dev)
    idx_q = torch.empty((Bt, M), dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = torch.empty(max(256, int(lib().maxsim_chamfer_fwd_workspace_bytes(Bt, N, M))), dtype=torch.uint8,
                                device=dev)
    st = lib().maxsim_chamfer_fwd(_ptr(P), _ptr(Q), Bt, N, M, _ptr(dist_p), _ptr(idx_p), _ptr(dist_q), _ptr(idx_q),
                                  _ptr(workspace), workspace.numel(), _stream(P, stream))
    _check(st, "maxsim_chamfer_fwd")
    return dist_p, idx_p, dist_q, idx_q


def maxsim_chamfer_bwd(P, Q, idx_p, idx_q, grad_p, grad_q, workspace=None, stream=None):
    """Gradients of sum grad_p*dist_p + sum grad_q*dist_q through the saved selections:
    (dP, dQ, row_ptr_p, col_idx_p, row_ptr_q, col_idx_q)."""
    P, Q = _clouds(P, Q)
    Bt, N, _ = P.shape
    M = Q.shape[1]
    dev = P.device
    for t, n in ((idx_p, "idx_p"), (idx_q, "idx_q")):
        _need(t, n, torch.int32, dev)
    for t, n in ((grad_p, "grad_p"), (grad_q, "grad_q")):
        _need(t, n, torch.float32, dev)
    dP = torch.empty((Bt, N, 3), dtype=torch.float32, device=dev)
    dQ = torch.empty((Bt, M, 3), dtype=torch.float32, device=dev)
    rp_p = torch.empty(Bt * N + 1, dtype=torch.int32, device=dev)
    ci_p = torch.empty(max(1, Bt * M), dtype=torch.int32, device=dev)
    rp_q = torch.empty(Bt * M + 1, dtype=torch.int32, device=dev)
    ci_q = torch.empty(max(1, Bt * N), dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = torch.empty(max(256, int(lib().maxsim_chamfer_bwd_workspace_bytes(Bt, N, M))), dtype=torch.uint8,
                                device=dev)
    st = lib().maxsim_chamfer_bwd(_ptr(P), _ptr(Q), _ptr(idx_p), _ptr(idx_q), _ptr(grad_p), _ptr(grad_q), Bt, N, M,
                                  _ptr(dP), _ptr(dQ), _ptr(rp_p), _ptr(ci_p), _ptr(rp_q), _ptr(ci_q),
                                  _ptr(workspace), workspace.numel(), _stream(P, stream))
    _check(st, "maxsim_chamfer_bwd")
    return dP, dQ, rp_p, ci_p, rp_q, ci_q


class ChamferFunction(torch.autograd.Function):
    """(dist_p, dist_q) with autograd: the forward saves the nearest-neighbour
    indices, the backward inverts them (paper Section 4.2, Chamfer distance)."""

    @staticmethod
    def forward(ctx, P, Q):
        dist_p, idx_p, dist_q, idx_q = maxsim_chamfer_fwd(P, Q)
        ctx.save_for_backward(P, Q, idx_p, idx_q)
        return dist_p, dist_q

    @staticmethod
    def backward(ctx, grad_p, grad_q):
        P, Q, idx_p, idx_q = ctx.saved_tensors
        dP, dQ, _, _, _, _ = maxsim_chamfer_bwd(P, Q, idx_p, idx_q, grad_p.float().contiguous(),
                                                grad_q.float().contiguous())
        return dP.reshape(P.shape), dQ.reshape(Q.shape)


def chamfer_distance(P, Q):
    """The page's Chamfer distance per batch item, mean_p min_q |p-q|^2 +
    mean_q min_p |q-p|^2, for P [Bt, N, 3] and Q [Bt, M, 3] fp32, with autograd.

    Caller-side convenience, not a library operation: the nearest-neighbour
    distances and their gradients come from maxsim_chamfer_fwd and
    maxsim_chamfer_bwd; the mean over points that turns them into the loss
    is a torch reduction here (its backward hands the per-point weights 1/N
    and 1/M to maxsim_chamfer_bwd)."""
    dist_p, dist_q = ChamferFunction.apply(P, Q)
    return dist_p.mean(dim=-1) + dist_q.mean(dim=-1)


def maxsim_fwd_pairs(Q, D_packed, cu_seqlens, pair_q, pair_b, scores=None, argmax=None, with_argmax=False,
                     stream=None):
    """Scores [P] (and argmax [P, Lq]) of the listed (query, document) pairs over a packed corpus."""
    Nq, Lq, d = Q.shape
    T, d2 = D_packed.shape
    B = cu_seqlens.shape[0] - 1
    P = pair_q.shape[0]
    if d2 != d or Q.dtype != D_packed.dtype:
        raise ValueError("Q and D_packed must share dtype and width")
    dev = Q.device
    _need(Q, "Q")
    _need(D_packed, "D_packed", device=dev)
    _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
    _need(pair_q, "pair_q", torch.int32, dev)
    _need(pair_b, "pair_b", torch.int32, dev)
    if pair_b.shape[0] != P:
        raise ValueError("pair_q and pair_b must have the same length")
    if scores is None:
        scores = torch.empty(P, dtype=torch.float32, device=dev)
    _need(scores, "scores", torch.float32, dev)
    if argmax is None and with_argmax:
        argmax = torch.empty((P, Lq), dtype=torch.int32, device=dev)
    if argmax is not None:
        _need(argmax, "argmax", torch.int32, dev)
    st = lib().maxsim_fwd_pairs(_ptr(Q), _ptr(D_packed), _ptr(cu_seqlens), _dtype_code(Q), _ptr(pair_q),
                                _ptr(pair_b), P, Nq, Lq, B, T, d, _ptr(scores), _ptr(argmax), _stream(Q, stream))
    _check(st, "maxsim_fwd_pairs")
    return scores, argmax


def maxsim_topk(scores, K, ids=None, top_idx=None, top_score=None, stream=None):
    """Per row of scores [Nq, B] fp32: (top_idx [Nq, K] int32, top_score [Nq, K]), best first,
    equal scores by ascending id (ids [Nq, B] int32 if given, else the column)."""
    Nq, B = scores.shape
    dev = scores.device
    _need(scores, "scores", torch.float32)
    if ids is not None:
        _need(ids, "ids", torch.int32, dev)
        if ids.shape != scores.shape:
            raise ValueError("ids must have the shape of scores")
    if top_idx is None:
        top_idx = torch.empty((Nq, K), dtype=torch.int32, device=dev)
    if top_score is None:
        top_score = torch.empty((Nq, K), dtype=torch.float32, device=dev)
    _need(top_idx, "top_idx", torch.int32, dev)
    _need(top_score, "top_score", torch.float32, dev)
    st = lib().maxsim_topk(_ptr(scores), _ptr(ids), Nq, B, K, _ptr(top_idx), _ptr(top_score),
                           _stream(scores, stream))
    _check(st, "maxsim_topk")
    return top_idx, top_score


def maxsim_two_stage_workspace_bytes(Nq, B, K1):
    return int(lib().maxsim_two_stage_workspace_bytes(Nq, B, K1))


def maxsim_two_stage_topk(Q8, q_scale, D8, d_scale, Q16, D16, cu_seqlens, max_Ld, K1, K2, workspace=None,
                          stream=None):
    """INT8 scan of the whole corpus, each query's K1 best re-scored in fp16 / bf16 from Q16 / D16,
    the K2 best kept.  Returns (cand [Nq, K1], cand_score8, top_idx [Nq, K2], top_score)."""
    Nq, Lq, d = Q8.shape
    T = D8.shape[0]
    B = cu_seqlens.shape[0] - 1
    dev = Q8.device
    _need(Q8, "Q8", torch.int8)
    _need(D8, "D8", torch.int8, dev)
    _need(q_scale, "q_scale", torch.float32, dev)
    _need(d_scale, "d_scale", torch.float32, dev)
    _need(Q16, "Q16", device=dev)
    _need(D16, "D16", device=dev)
    _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
    if Q16.shape != Q8.shape or D16.shape != D8.shape or Q16.dtype != D16.dtype:
        raise ValueError("Q16 / D16 must be the fp16 or bf16 rows of Q8 / D8")
    nbytes = maxsim_two_stage_workspace_bytes(Nq, B, K1)
    if workspace is None:
        workspace = torch.empty(max(256, nbytes), dtype=torch.uint8, device=dev)
    cand = torch.empty((Nq, K1), dtype=torch.int32, device=dev)
    cand8 = torch.empty((Nq, K1), dtype=torch.float32, device=dev)
    top_idx = torch.empty((Nq, K2), dtype=torch.int32, device=dev)
    top_score = torch.empty((Nq, K2), dtype=torch.float32, device=dev)
    st = lib().maxsim_two_stage_topk(_ptr(Q8), _ptr(q_scale), _ptr(D8), _ptr(d_scale), _ptr(Q16), _ptr(D16),
                                     _ptr(cu_seqlens), _dtype_code(Q16), Nq, Lq, B, T, int(max_Ld), d, K1, K2,
                                     _ptr(cand), _ptr(cand8), _ptr(top_idx), _ptr(top_score), _ptr(workspace),
                                     workspace.numel(), _stream(Q8, stream))
    _check(st, "maxsim_two_stage_topk")
    return cand, cand8, top_idx, top_score


# ---------------------------------------------------------------- the embedding head and its training step
# (include/maxsim_encoder.h)

_CODES = {torch.float16: MAXSIM_F16, torch.bfloat16: MAXSIM_BF16, torch.float32: MAXSIM_F32, torch.int8: MAXSIM_I8,
          torch.float8_e4m3fn: MAXSIM_E4M3}


def _on_its_device(f):
    """Runs f on the device of its first argument, and on `stream` where one is given: what f allocates then belongs
    to the stream that uses it."""

    @functools.wraps(f)
    def call(first, *args, stream=None, **kw):
        dev = first.device
        if dev.type != "cuda":
            raise ValueError("%s: the tensors must be on the device" % f.__name__)
        if stream is None and dev.index == torch._C._cuda_getDevice():
            return f(first, *args, **kw)
        if stream is None:
            with torch.cuda.device(dev):
                return f(first, *args, **kw)
        if stream.device != dev:
            raise ValueError("%s: the stream is on %s, the tensors on %s" % (f.__name__, stream.device, dev))
        with torch.cuda.stream(stream):
            return f(first, *args, **kw)

    return call


def _raw_stream(dev):
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _code(dtype, allowed, name):
    c = _CODES.get(dtype, -1)
    if c not in allowed:
        raise TypeError("%s may not be %s" % (name, dtype))
    return c


_FLOATS = (MAXSIM_F16, MAXSIM_BF16, MAXSIM_F32)
_ALL = _FLOATS + (MAXSIM_I8, MAXSIM_E4M3)


def _rows(t, name, shape, dtype, dev):
    """The pitch of t as rows of its last dimension; t has `shape` and `dtype` and lies on `dev`."""
    if t.dtype is dtype and t.is_contiguous() and t.shape == shape and t.device == dev:
        return shape[-1]
    if t.device != dev:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    width = shape[-1]
    # rows one pitch apart through all leading dimensions, neighbours within a row
    pitch, rows = None, 1
    for d in range(len(shape) - 2, -1, -1):
        if shape[d] == 1:
            continue
        if pitch is None:
            pitch = t.stride(d)
        elif t.stride(d) != pitch * rows:
            raise ValueError("%s: the rows must be one pitch apart" % name)
        rows *= shape[d]
    if t.stride(-1) != 1 and width > 1:
        raise ValueError("%s: the values of a row must be neighbours" % name)
    if pitch is None:
        return width
    if pitch < width:
        raise ValueError("%s: the rows overlap" % name)
    return pitch


def _flat(t, name, n, dtype, dev):
    """t holds n values of `dtype` back to back on `dev`."""
    if t.dtype is dtype and t.is_contiguous() and t.numel() == n and t.device == dev:
        return
    if t.device != dev:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.numel() != n or not t.is_contiguous():
        raise ValueError("%s must hold %d contiguous values" % (name, n))


def _empty_e4m3(like, shape):
    """[..., width] e4m3 with rows a multiple of 16 bytes apart, as the product reads them."""
    width = shape[-1]
    pad = -width % 16
    if pad == 0:
        return like.new_empty(shape, dtype=torch.float8_e4m3fn)
    return like.new_empty(tuple(shape[:-1]) + (width + pad,), dtype=torch.float8_e4m3fn)[..., :width]


def _size(n):
    """A size or step for the C entry points' 32 bits, to which ctypes would cut it silently."""
    if not -0x80000000 <= n <= 0x7FFFFFFF:
        raise ValueError("%d does not fit 32 bits" % n)
    return n


def _row_count(shape):
    n = 1
    for s in shape[:-1]:
        n *= s
    return _size(n)


def _gain(weight, H, dtype, dev):
    if weight is None:
        return None, MAXSIM_F32
    if weight.dtype != dtype and weight.dtype != torch.float32:
        raise TypeError("weight must be %s or float32, got %s" % (dtype, weight.dtype))
    _flat(weight, "weight", H, weight.dtype, dev)
    return weight.data_ptr(), _CODES[weight.dtype]


def maxsim_rmsnorm_fwd(x, weight=None, eps=1e-6, residual=None, out_dtype=None, with_rstd=False, y=None, scale=None,
                       sum=None, rstd=None, stream=None):
    """RMS norm of the rows of x [..., H] (fp16, bf16, fp32), of x + residual where one is given.

    out_dtype: x's (the default), float16, bfloat16, float32, int8 (a scale for each row: the operand of
    maxsim_fwd_i8) or float8_e4m3fn (a scale for each 128 columns: the operand of maxsim_gemm_fp8).
    Returns (y, scale or None, sum or None, rstd or None); sum = x + residual in x's type, rstd [...] fp32.
    """
    if y is None and scale is None and sum is None and rstd is None and stream is None:
        got = _fast.rmsnorm_fwd(x, weight, eps, residual, out_dtype, with_rstd)
        if got is not None:
            return got
    return _rmsnorm_fwd(x, weight, eps, residual, out_dtype, with_rstd, y, scale, sum, rstd, stream=stream)


@_on_its_device
def _rmsnorm_fwd(x, weight, eps, residual, out_dtype, with_rstd, y, scale, sum, rstd):
    dev, shape, dtype = x.device, x.shape, x.dtype
    H, R = _size(shape[-1]), _row_count(shape)
    code = _code(dtype, _FLOATS, "x")
    out_dtype = dtype if out_dtype is None else out_dtype
    out = _code(out_dtype, _ALL, "out_dtype")
    ldx = _rows(x, "x", shape, dtype, dev)
    w, w_code = _gain(weight, H, dtype, dev)
    ldr = lds = ldy = H
    residual_at = sum_at = rstd_at = scale_at = None
    if residual is not None:
        ldr = _rows(residual, "residual", shape, dtype, dev)
        residual_at = residual.data_ptr()
        if sum is None:
            sum = x.new_empty(shape)
            sum_at = sum.data_ptr()
    if sum is not None and sum_at is None:
        lds = _rows(sum, "sum", shape, dtype, dev)
        sum_at = sum.data_ptr()
    if y is not None or out == MAXSIM_E4M3:
        if y is None:
            y = _empty_e4m3(x, shape)
        ldy = _rows(y, "y", shape, out_dtype, dev)
    else:
        y = x.new_empty(shape, dtype=out_dtype)
    if out >= MAXSIM_I8:
        want = shape[:-1] if out == MAXSIM_I8 else shape[:-1] + (-(-H // QBLOCK),)
        if scale is None:
            scale = x.new_empty(want, dtype=torch.float32)
        else:
            _flat(scale, "scale", R * (1 if out == MAXSIM_I8 else want[-1]), torch.float32, dev)
        scale_at = scale.data_ptr()
    elif scale is not None:
        raise ValueError("scale goes with an 8-bit output")
    if rstd is not None:
        _flat(rstd, "rstd", R, torch.float32, dev)
    elif with_rstd:
        rstd = x.new_empty(shape[:-1], dtype=torch.float32)
    if rstd is not None:
        rstd_at = rstd.data_ptr()
    st = _lib.maxsim_rmsnorm_fwd(x.data_ptr(), ldx, residual_at, ldr, w, w_code, R, H, code, eps, out, y.data_ptr(),
                                 ldy, scale_at, sum_at, lds, rstd_at, _raw_stream(dev))
    if st:
        _check(st, "maxsim_rmsnorm_fwd")
    return y, scale, sum, rstd


def maxsim_rmsnorm_bwd_workspace_bytes(R, H):
    return int(lib().maxsim_rmsnorm_bwd_workspace_bytes(R, H))


def maxsim_rmsnorm_bwd(dy, h, rstd, weight=None, dsum=None, with_dweight=True, dx=None, dweight=None, workspace=None,
                       stream=None):
    """Backward of the norm.  dy [..., H] is the gradient of y, h the forward's sum (x without a residual), rstd its
    rstd, dsum the gradient that arrives at sum itself.  Returns (dx, dweight [H] fp32 or None); dx is the gradient
    of x and of residual alike."""
    if dx is None and dweight is None and workspace is None and stream is None:
        got = _fast.rmsnorm_bwd(dy, h, rstd, weight, dsum, with_dweight)
        if got is not None:
            return got
    return _rmsnorm_bwd(dy, h, rstd, weight, dsum, with_dweight, dx, dweight, workspace, stream=stream)


@_on_its_device
def _rmsnorm_bwd(dy, h, rstd, weight, dsum, with_dweight, dx, dweight, workspace):
    dev, shape, dtype = h.device, h.shape, h.dtype
    H, R = _size(shape[-1]), _row_count(shape)
    code = _code(dtype, _FLOATS, "h")
    ldh = _rows(h, "h", shape, dtype, dev)
    lddy = _rows(dy, "dy", shape, dtype, dev)
    _flat(rstd, "rstd", R, torch.float32, dev)
    w, w_code = _gain(weight, H, dtype, dev)
    ldds = H if dsum is None else _rows(dsum, "dsum", shape, dtype, dev)
    lddx = H
    if dx is None:
        dx = h.new_empty(shape)
    else:
        lddx = _rows(dx, "dx", shape, dtype, dev)
    nbytes = 0
    if dweight is None and with_dweight:
        dweight = h.new_empty(H, dtype=torch.float32)
    elif dweight is not None:
        _flat(dweight, "dweight", H, torch.float32, dev)
    if dweight is not None:
        if workspace is None:
            nbytes = _lib.maxsim_rmsnorm_bwd_workspace_bytes(R, H)
            workspace = h.new_empty(nbytes, dtype=torch.uint8) if nbytes else None
        else:
            _need(workspace, "workspace", device=dev)
            nbytes = workspace.numel() * workspace.element_size()
    st = _lib.maxsim_rmsnorm_bwd(dy.data_ptr(), lddy, h.data_ptr(), ldh, rstd.data_ptr(), w, w_code,
                                 None if dsum is None else dsum.data_ptr(), ldds, R, H, code, dx.data_ptr(), lddx,
                                 None if dweight is None else dweight.data_ptr(),
                                 None if workspace is None else workspace.data_ptr(), nbytes, _raw_stream(dev))
    if st:
        _check(st, "maxsim_rmsnorm_bwd")
    return dx, dweight


def maxsim_quant_fp8(x, block_rows=1, rows=True, transposed=False, stream=None):
    """x [R, C] (fp16, bf16, fp32) in e4m3 with a scale for each 128 columns of a row (block_rows 1) or each
    128 x 128 values (block_rows 128), for maxsim_gemm_fp8.  Returns (q [R, C], scale, qt [C, R], scale_t): qt is x
    transposed, with a scale for each 128 of x's rows; rows / transposed say which of the two are made (else None)."""
    if stream is None:
        got = _fast.quant_fp8(x, block_rows, rows, transposed)
        if got is not None:
            return got
    return _quant_fp8(x, block_rows, rows, transposed, stream=stream)


@_on_its_device
def _quant_fp8(x, block_rows, rows, transposed):
    if x.dim() != 2:
        raise ValueError("x must be [R, C]")
    dev = x.device
    R, C = map(_size, x.shape)
    code = _code(x.dtype, _FLOATS, "x")
    ldx = _rows(x, "x", x.shape, x.dtype, dev)
    if not rows and not transposed:
        raise ValueError("neither rows nor transposed: nothing to make")
    rb, cb = -(-R // QBLOCK), -(-C // QBLOCK)
    q = scale = qt = scale_t = None
    if rows:
        q = _empty_e4m3(x, (R, C))
        scale = x.new_empty((R if block_rows == 1 else rb, cb), dtype=torch.float32)
    if transposed:
        qt = _empty_e4m3(x, (C, R))
        scale_t = x.new_empty((C if block_rows == 1 else cb, rb), dtype=torch.float32)
    st = _lib.maxsim_quant_fp8(x.data_ptr(), ldx, R, C, code, block_rows,
                               None if q is None else q.data_ptr(), -(-C // 16) * 16,
                               None if scale is None else scale.data_ptr(),
                               None if qt is None else qt.data_ptr(), -(-R // 16) * 16,
                               None if scale_t is None else scale_t.data_ptr(), _raw_stream(dev))
    if st:
        _check(st, "maxsim_quant_fp8")
    return q, scale, qt, scale_t


def _operand(t, name, dev):
    """The pitch of an e4m3 operand [rows, K]; every row is readable up to K rounded up to 16."""
    rows, K = t.shape
    if K % 16 == 0 and t.is_contiguous() and t.dtype is torch.float8_e4m3fn and t.device == dev:
        return K
    ld = _rows(t, name, t.shape, torch.float8_e4m3fn, dev)
    k16 = -(-K // 16) * 16
    if ld < k16 and rows <= 1:
        ld = k16
    if K != k16 and rows > 0 and t.storage_offset() + (rows - 1) * ld + k16 > t.untyped_storage().nbytes():
        raise ValueError("%s: rows of %d bytes must be readable up to %d" % (name, K, k16))
    return ld


def maxsim_gemm_fp8_workspace_bytes(M, N, K):
    return int(lib().maxsim_gemm_fp8_workspace_bytes(M, N, K))


def maxsim_gemm_fp8(A, a_scale, B, b_scale, out_dtype=torch.bfloat16, out=None, workspace=None, stream=None):
    """A B^T of e4m3 A [M, K] and B [N, K] with a_scale [M, ceil(K/128)] and b_scale [N, ceil(K/128)] or
    [ceil(N/128), ceil(K/128)] (a scale for 128 rows of B); fp32 sums, rounded once to out_dtype."""
    if out is None and workspace is None and stream is None:
        got = _fast.gemm_fp8(A, a_scale, B, b_scale, out_dtype)
        if got is not None:
            return got
    return _gemm_fp8(A, a_scale, B, b_scale, out_dtype, out, workspace, stream=stream)


@_on_its_device
def _gemm_fp8(A, a_scale, B, b_scale, out_dtype, out, workspace):
    dev = A.device
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[1]:
        raise ValueError("A [M, K] and B [N, K] must share K")
    M, K = map(_size, A.shape)
    N = _size(B.shape[0])
    lda, ldb = _operand(A, "A", dev), _operand(B, "B", dev)
    kb = -(-K // QBLOCK)
    _flat(a_scale, "a_scale", M * kb, torch.float32, dev)
    block_rows = 1 if b_scale.shape[0] == N else QBLOCK
    _flat(b_scale, "b_scale", -(-N // block_rows) * kb, torch.float32, dev)
    ldc = N
    if out is None:
        code = _code(out_dtype, _FLOATS, "out_dtype")
        out = a_scale.new_empty((M, N), dtype=out_dtype)
    else:
        code = _code(out.dtype, _FLOATS, "out")
        ldc = _rows(out, "out", (M, N), out.dtype, dev)
    nbytes = _lib.maxsim_gemm_fp8_workspace_bytes(M, N, K)
    if workspace is not None:
        _need(workspace, "workspace", device=dev)
        nbytes = workspace.numel() * workspace.element_size()
    elif nbytes:
        workspace = a_scale.new_empty(nbytes, dtype=torch.uint8)
    st = _lib.maxsim_gemm_fp8(A.data_ptr(), lda, a_scale.data_ptr(), B.data_ptr(), ldb, b_scale.data_ptr(), block_rows,
                              M, N, K, code, out.data_ptr(), ldc, None if workspace is None else workspace.data_ptr(),
                              nbytes, _raw_stream(dev))
    if st:
        _check(st, "maxsim_gemm_fp8")
    return out


_TENSOR = np.dtype([("param", np.uint64), ("grad", np.uint64), ("master", np.uint64), ("m", np.uint64),
                    ("v", np.uint64), ("m_scale", np.uint64), ("v_scale", np.uint64), ("n", np.int64)])


class AdamWTensors:
    """The tensors that maxsim_adamw steps over: parameters (all fp16, bf16 or fp32), moments m and v, and for 16-bit
    parameters fp32 masters that they are rounded from (optional).  Moments are fp32, or float8_e4m3fn with m_scales
    and v_scales (fp32, one for each 128 values; v is then held as its square root).  zeros() makes them.  No two of
    them may share memory (a tied weight is listed once), and each has to keep its own (a step checks that)."""

    def __init__(self, params, m, v, m_scales=None, v_scales=None, masters=None):
        params = list(params)
        if not params:
            raise ValueError("no parameters")
        self.device = dev = params[0].device
        self.params, self.m, self.v = params, list(m), list(v)
        self.m_scales = None if m_scales is None else list(m_scales)
        self.v_scales = None if v_scales is None else list(v_scales)
        self.masters = None if masters is None else list(masters)
        self.param_code = _code(params[0].dtype, _FLOATS, "params")
        self.state_code = _code(self.m[0].dtype if self.m else None, (MAXSIM_F32, MAXSIM_E4M3), "m")
        if (self.state_code == MAXSIM_E4M3) != (m_scales is not None) or (m_scales is None) != (v_scales is None):
            raise ValueError("m_scales and v_scales go with 8-bit moments")
        if masters is not None and self.param_code == MAXSIM_F32:
            raise ValueError("masters go with 16-bit parameters")
        self.sizes = [p.numel() for p in params]
        state = self.m[0].dtype
        table = np.zeros(len(params), _TENSOR)
        table["n"] = self.sizes

        def put(field, tensors, dtype, per=1):
            if len(tensors) != len(params):
                raise ValueError("%s: %d tensors for %d parameters" % (field, len(tensors), len(params)))
            for i, t in enumerate(tensors):
                _flat(t, "%s[%d]" % (field, i), -(-self.sizes[i] // per), dtype, dev)
                table[field][i] = t.data_ptr()

        put("param", params, params[0].dtype)
        put("m", self.m, state)
        put("v", self.v, state)
        if m_scales is not None:
            put("m_scale", self.m_scales, torch.float32, QBLOCK)
            put("v_scale", self.v_scales, torch.float32, QBLOCK)
        if masters is not None:
            put("master", self.masters, torch.float32)
        self._table = table
        self._address = table.ctypes.data
        fields = [self.params, self.m, self.v] + ([self.m_scales, self.v_scales] if m_scales is not None else [])
        self._held = [t for of_one in zip(*(fields + ([self.masters] if masters is not None else []))) for t in of_one]
        self._held_at = [t.data_ptr() for t in self._held]
        ends = sorted((at, at + t.numel() * t.element_size()) for at, t in zip(self._held_at, self._held) if t.numel())
        if any(this[1] > following[0] for this, following in zip(ends, ends[1:])):
            raise ValueError("two of the tensors share memory")

    def __reduce__(self):
        # a copy, or one read back from a file, has tensors of its own, and so a table of its own
        return type(self), (self.params, self.m, self.v, self.m_scales, self.v_scales, self.masters)

    def _check_memory(self):
        # a tensor whose .data was replaced, or whose storage was freed, would be updated where it no longer is
        if any(t.data_ptr() != at for t, at in zip(self._held, self._held_at)):
            raise ValueError("a tensor's memory has moved since this AdamWTensors was made")

    @classmethod
    def zeros(cls, params, state_dtype=torch.float32, masters=True):
        """Moments at 0 for these parameters, and fp32 masters of 16-bit ones."""
        params = list(params)
        moments = lambda: [torch.zeros(p.numel(), dtype=torch.float32, device=p.device).to(state_dtype)  # noqa: E731
                           for p in params]
        scales = lambda: [torch.zeros(-(-p.numel() // QBLOCK), device=p.device) for p in params]  # noqa: E731
        eight = state_dtype == torch.float8_e4m3fn
        held = [p.detach().float() for p in params] if masters and params[0].dtype != torch.float32 else None
        return cls(params, moments(), moments(), scales() if eight else None,
                   scales() if eight else None, held)


def maxsim_adamw(tensors, grads, step, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step_dev=None,
                 stream=None):
    """One AdamW step of an AdamWTensors with these gradients (one tensor a parameter, all fp16, bf16 or fp32), in
    place.  step: the number of this step, from 1 on; or step_dev, a device int32 that holds it, for a step that is
    captured and replayed.  A graph that saved a parameter before the step refuses its backward after it, as after any
    change in place."""
    if step_dev is None and stream is None:
        st = _fast.adamw(tensors._address, len(tensors.sizes), tensors.device.index, tensors.param_code,
                         tensors.state_code, tensors._held, grads, lr, beta1, beta2, eps, weight_decay, step)
        if st is not None:  # the call was made: never make it again, the step is in place
            return _check(st, "maxsim_adamw")
    _adamw(tensors, grads, step, lr, beta1, beta2, eps, weight_decay, step_dev, stream=stream)


@_on_its_device
def _adamw(tensors, grads, step, lr, beta1, beta2, eps, weight_decay, step_dev):
    dev = tensors.device
    tensors._check_memory()
    if len(grads) != len(tensors.sizes):
        raise ValueError("%d gradients for %d parameters" % (len(grads), len(tensors.sizes)))
    dtype = grads[0].dtype
    code = _code(dtype, _FLOATS, "grads")
    for g, n in zip(grads, tensors.sizes):
        if g.dtype != dtype or g.numel() != n or g.device != dev or not g.is_contiguous():
            raise ValueError("gradients must be contiguous, of one type, on %s and of their parameters' sizes" % dev)
    if step_dev is not None:
        _flat(step_dev, "step_dev", 1, torch.int32, dev)
    _size(step)
    table = tensors._table.copy()
    table["grad"] = [g.data_ptr() for g in grads]
    st = _lib.maxsim_adamw(table.ctypes.data, len(grads), tensors.param_code, code, tensors.state_code, lr, beta1,
                           beta2, eps, weight_decay, step, None if step_dev is None else step_dev.data_ptr(),
                           _raw_stream(dev))
    if st in (MAXSIM_OK, MAXSIM_ERR_HIP):  # the parameters have changed, or some may have
        torch.autograd.graph.increment_version([p for p in tensors.params if not p.is_inference()])
    _check(st, "maxsim_adamw")


class RMSNormFunction(torch.autograd.Function):
    """RMS norm of x (+ residual) as an autograd op; with a residual the sum is an output too."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        ctx.set_materialize_grads(False)  # an output that nothing uses costs no tensor of zeros
        y, _, h, rstd = maxsim_rmsnorm_fwd(x, weight, eps, residual=residual, with_rstd=True)
        ctx.save_for_backward(x if residual is None else h, weight, rstd)
        return y if residual is None else (y, h)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dsum=None):
        h, weight, rstd = ctx.saved_tensors
        dw = None
        if dy is None:  # only the sum was used
            dx = dsum
            if weight is not None and ctx.needs_input_grad[1]:
                dw = torch.zeros_like(weight)
        else:
            dx, dw = maxsim_rmsnorm_bwd(dy.contiguous(), h, rstd, weight,
                                        dsum=None if dsum is None else dsum.contiguous(),
                                        with_dweight=weight is not None and ctx.needs_input_grad[1])
        return (dx if ctx.needs_input_grad[0] else None, None if dw is None else dw.to(weight.dtype).reshape(weight.shape),
                dx if ctx.needs_input_grad[2] else None, None)


def rms_norm(x, weight=None, residual=None, eps=1e-6):
    """x / sqrt(mean(x^2) + eps) * weight over the last dimension, with autograd support.  With a residual of x's shape: the norm
    of x + residual, and the sum itself, (y, sum)."""
    return RMSNormFunction.apply(x.contiguous(), weight, None if residual is None else residual.contiguous(), eps)


class LinearFP8Function(torch.autograd.Function):
    """x W^T with both operands in 8 bits, as an autograd op: x and dy with a scale for each 128 along the sum they
    take part in, W for each 128 x 128.  Of x only its 8-bit transpose is kept for dW."""

    @staticmethod
    def forward(ctx, x, weight):
        rows = x.reshape(_row_count(x.shape), x.shape[-1]).contiguous()
        need_x, need_w = ctx.needs_input_grad
        q, s, qt, st = maxsim_quant_fp8(rows, transposed=need_w)
        w, ws, wt, wst = maxsim_quant_fp8(weight.contiguous(), block_rows=QBLOCK, transposed=need_x)
        ctx.save_for_backward(qt, st, wt, wst)
        ctx.x_shape, ctx.x_dtype, ctx.w_dtype = x.shape, x.dtype, weight.dtype
        return maxsim_gemm_fp8(q, s, w, ws, out_dtype=x.dtype).reshape(x.shape[:-1] + (weight.shape[0],))

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        qt, st, wt, wst = ctx.saved_tensors
        need_x, need_w = ctx.needs_input_grad
        g, gs, gt, gst = maxsim_quant_fp8(dy.reshape(_row_count(dy.shape), dy.shape[-1]).contiguous(), rows=need_x,
                                          transposed=need_w)
        dx = dw = None
        if need_x:
            dx = maxsim_gemm_fp8(g, gs, wt, wst, out_dtype=ctx.x_dtype).reshape(ctx.x_shape)
        if need_w:
            dw = maxsim_gemm_fp8(gt, gst, qt, st, out_dtype=torch.float32).to(ctx.w_dtype)
        return dx, dw


_MOST_K = 1 << 22  # of maxsim_gemm_fp8


def _product_takes(M, N, K):
    """Sizes within maxsim_gemm_fp8's limits."""
    return K <= _MOST_K and -(-M // QBLOCK) * -(-N // QBLOCK) < 1 << 22


def linear_fp8(x, weight):
    """x [..., K] times weight [N, K] transposed, in 8-bit floating point with a scale for each block of 128, with
    autograd support (x, weight: fp16, bf16 or fp32; the result has x's type).  A gradient's product runs over the
    tokens (of weight) or over N (of x), of which it takes 2^22 at most."""
    if weight.dim() != 2 or x.shape[-1] != weight.shape[1]:
        raise ValueError("x [..., K] and weight [N, K] must share K")
    if torch.is_grad_enabled():  # refused here and not by the product in the backward
        T, (N, K) = _row_count(x.shape), weight.shape
        if weight.requires_grad and not _product_takes(N, K, T):
            raise ValueError("linear_fp8: no gradient of a weight [%d, %d] from %d tokens (at most %d)" % (N, K, T, _MOST_K))
        if x.requires_grad and not _product_takes(T, K, N):
            raise ValueError("linear_fp8: no gradient of x [%d, %d] through %d columns (at most %d)" % (T, K, N, _MOST_K))
    return LinearFP8Function.apply(x, weight)


def encode_tokens(hidden, gain, proj, proj_scale, residual=None, out_dtype=torch.int8, eps=1e-6):
    """Token rows for the MaxSim entry points from an encoder's last hidden rows [..., H]: their RMS norm (of
    hidden + residual where one is given) in 8 bits, the projection to 128 columns, and rows of length 1 --
    (rows int8 [..., 128], scale [...]) for maxsim_fwd_i8, or (rows fp16 / bf16, None) for the other forwards.
    proj [128, H] and proj_scale: maxsim_quant_fp8(weight, block_rows=128).  hidden has to be finite: the forwards take
    no NaN."""
    if proj.shape[0] != QBLOCK:
        raise ValueError("proj must have 128 rows, got %d" % proj.shape[0])
    q, s, _, _ = maxsim_rmsnorm_fwd(hidden, gain, eps, residual=residual, out_dtype=torch.float8_e4m3fn)
    H = hidden.shape[-1]
    # rows of one pitch: the leading dimensions collapse without a copy
    flat = q.as_strided((_row_count(q.shape), H), (-(-H // 16) * 16, 1))
    rows = maxsim_gemm_fp8(flat, s, proj, proj_scale, out_dtype=torch.float32)
    # rows of length 1: the norm with the gain 1 / sqrt(128)
    gain1 = torch.full((QBLOCK,), QBLOCK ** -0.5, dtype=torch.float32, device=rows.device)
    rows, scale, _, _ = maxsim_rmsnorm_fwd(rows, gain1, 1e-12, out_dtype=out_dtype)
    shape = hidden.shape[:-1]
    return rows.reshape(shape + (QBLOCK,)), None if scale is None else scale.reshape(shape)
