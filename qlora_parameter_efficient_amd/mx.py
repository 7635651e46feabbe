"""ctypes binding of the MX entry points (include/lq_mx.h) of liblq.so.

As in lq.py, each function has the name of the C entry point it calls: it
checks placement, dtypes and shapes, allocates outputs and workspace with
torch, passes raw pointers and the current HIP stream of the tensors' device,
and raises LqError on a negative status.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from dataclasses import dataclass

import torch

from . import lq
from .lq import LqError, LqWeightStruct, NF4Weight  # noqa: F401

HEADER = os.path.join(os.path.dirname(lq.HEADER), "lq_mx.h")

LQ_MX_BLOCK = 32
LQ_MX_FP4, LQ_MX_FP8 = 4, 8
LQ_MX_ROWS_BF16 = 64
LQ_MX_OP_FWD, LQ_MX_OP_BWD, LQ_MX_OP_BWD_CKPT = 0, 1, 2
FORMATS = {"fp4": LQ_MX_FP4, "fp8": LQ_MX_FP8}


class LqMxStruct(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


_vp, _i32, _i64, _f32, _sz = lq._vp, lq._i32, lq._i64, lq._f32, lq._sz
_QP = ctypes.POINTER(LqMxStruct)

_SIGS = {
    "lq_mx_codes_bytes": (_sz, [_i32, _i64, _i64]),
    "lq_mx_scales_bytes": (_sz, [_i64, _i64]),
    "lq_mx_quantize": (ctypes.c_int, [_vp, _i32, _i64, _i64, _i32, _vp, _vp, _vp]),
    "lq_mx_dequantize": (ctypes.c_int, [_QP, _vp, _i32, _vp]),
    "lq_mx_lora_fwd": (ctypes.c_int, [_vp, _QP, _i64, _QP, _vp, _vp, _i64, _f32, _vp, _vp, _vp,
                                      _sz, _vp]),
    "lq_mx_lora_bwd": (ctypes.c_int, [_vp, _QP, _i64, _QP, _vp, _vp, _i64, _f32, _vp, _vp, _vp,
                                      _vp, _i32, _vp, _sz, _vp]),
    "lq_lora_bwd_ckpt": (ctypes.c_int, [_vp, _QP, _i64, lq._WP, _vp, _vp, _i64, _f32, _vp, _vp,
                                        _vp, _vp, _i32, _vp, _sz, _vp]),
    "lq_mx_workspace_size": (_sz, [_i32, _i64, _i64, _i64, _i64]),
}

_lib = None


def lib():
    global _lib
    if _lib is None:
        L = lq.lib()
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


@dataclass
class MxTensor:
    """Device buffers of an MX tensor (rows x cols, blocks of 32 columns)."""
    codes: torch.Tensor            # uint8, rows x (padded columns / 2 or 1)
    scales: torch.Tensor           # uint8, rows x (padded columns / 32)
    rows: int
    cols: int
    format: str                    # "fp4" (E2M1) or "fp8" (E4M3)


def _check(rc):
    if rc != 0:
        raise LqError(rc, lib().lq_last_error().decode())


def _want(cond, msg):
    if not cond:
        raise ValueError(msg)


def _same_device(dev, *ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda or t.device != dev:
                raise ValueError("tensors must be on one GPU")
            if not t.is_contiguous():
                raise ValueError("tensors must be contiguous")


def _tensor(t, dtype, shape, what):
    if t is not None and (t.dtype != dtype or t.shape != shape):
        raise ValueError(f"{what}: expected {dtype} of shape {tuple(shape)}, got {t.dtype} "
                         f"{tuple(t.shape)}")


def _on(dev):
    """Context that makes dev the current device (nothing when it already is)."""
    if dev.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(dev)


@functools.lru_cache(maxsize=512)
def _buffer_bytes(fmt, rows, cols):
    return (lib().lq_mx_codes_bytes(fmt, rows, cols), lib().lq_mx_scales_bytes(rows, cols))


@functools.lru_cache(maxsize=1024)
def lq_mx_workspace_size(op, M, N, K, r):
    return int(lib().lq_mx_workspace_size(op, M, N, K, r))


def mx_struct(q: MxTensor, dev):
    _same_device(dev, q.codes, q.scales)
    fmt = FORMATS[q.format]
    if q.codes.dtype != torch.uint8 or q.scales.dtype != torch.uint8:
        raise ValueError("MX codes and scales are uint8 tensors")
    if (q.codes.numel(), q.scales.numel()) != _buffer_bytes(fmt, q.rows, q.cols):
        raise ValueError(f"MX buffers do not hold a {q.rows} x {q.cols} {q.format} tensor")
    return LqMxStruct(fmt, 0, q.rows, q.cols, q.codes.data_ptr(), q.scales.data_ptr())


def _workspace(ws, op, M, N, K, r, dev):
    """(tensor that keeps it alive, pointer, bytes); ``ws`` is the caller's, or None."""
    if ws is None:
        need = lq_mx_workspace_size(op, M, N, K, r)
        if need == 0:
            return None, None, 0
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _same_device(dev, ws)
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


# ------------------------------------------------------------------ calls

def lq_mx_quantize(X: torch.Tensor, format: str = "fp8") -> MxTensor:
    dev = X.device
    _same_device(dev, X)
    _want(X.dim() == 2, "X must be a matrix")
    rows, cols = X.shape
    kb = -(-cols // LQ_MX_BLOCK)
    fmt = FORMATS[format]
    with _on(dev):
        codes = torch.empty((rows, kb * 4 * fmt), dtype=torch.uint8, device=dev)
        scales = torch.empty((rows, kb), dtype=torch.uint8, device=dev)
        _check(lib().lq_mx_quantize(X.data_ptr(), lq._dt(X), rows, cols, fmt, codes.data_ptr(),
                                    scales.data_ptr(), lq._stream()))
    return MxTensor(codes, scales, rows, cols, format)


def lq_mx_dequantize(q: MxTensor, dtype=torch.bfloat16) -> torch.Tensor:
    dev = q.codes.device
    s = mx_struct(q, dev)
    _want(dtype in (torch.bfloat16, torch.float32), f"unsupported dtype {dtype}")
    with _on(dev):
        out = torch.empty((q.rows, q.cols), dtype=dtype, device=dev)
        _check(lib().lq_mx_dequantize(ctypes.byref(s), out.data_ptr(), lq._dt(out), lq._stream()))
    return out


def _adapter(A, B, N, K):
    r = 0 if A is None else A.shape[0]
    _tensor(A, torch.bfloat16, (r, K), "A")
    if (A is None) != (B is None):
        raise ValueError("A and B must both be given or both be None")
    _tensor(B, torch.bfloat16, (N, r), "B")
    return r


def lq_mx_lora_fwd(X, W0: MxTensor, A=None, B=None, scale=0.0, T_out=None, ws=None, Y=None):
    """X: a bf16 matrix (at most LQ_MX_ROWS_BF16 rows) or an MxTensor; A and B
    None: no adapter."""
    dev = W0.codes.device
    w = mx_struct(W0, dev)
    N, K = W0.rows, W0.cols
    if isinstance(X, MxTensor):
        M = X.rows
        xq, xp = ctypes.byref(mx_struct(X, dev)), None
        _want(X.cols == K, f"X has {X.cols} columns, W0 {K}")
    else:
        M = X.shape[0]
        _same_device(dev, X)
        _tensor(X, torch.bfloat16, (M, K), "X")
        xq, xp = None, X.data_ptr()
    r = _adapter(A, B, N, K)
    _same_device(dev, A, B, T_out, Y)
    _tensor(T_out, torch.float32, (M, r), "T_out")
    _tensor(Y, torch.bfloat16, (M, N), "Y")
    with _on(dev):
        if Y is None:
            Y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        ws, wp, wn = _workspace(ws, LQ_MX_OP_FWD, M, N, K, r, dev)
        _check(lib().lq_mx_lora_fwd(xp, xq, M, ctypes.byref(w), lq._ptr(A), lq._ptr(B), r, scale,
                                    Y.data_ptr(), lq._ptr(T_out), wp, wn, lq._stream()))
    return Y


def _backward(fn, op, w, N, K, dev, dY, Xq, A, B, scale, T_saved, need_dx, need_grads, dX, dA, dB,
              accumulate, ws):
    M = dY.shape[0]
    _same_device(dev, dY, A, B, T_saved, dX, dA, dB)
    _tensor(dY, torch.bfloat16, (M, N), "dY")
    r = _adapter(A, B, N, K)
    _want(r > 0, "the backward needs an adapter")
    _tensor(T_saved, torch.float32, (M, r), "T_saved")
    _tensor(dX, torch.bfloat16, (M, K), "dX")
    _tensor(dA, torch.float32, (r, K), "dA")
    _tensor(dB, torch.float32, (N, r), "dB")
    _want(not accumulate or not need_grads or (dA is not None and dB is not None),
          "accumulate needs dA and dB")
    xq = None
    if need_grads:
        _want((Xq.rows, Xq.cols) == (M, K), f"Xq is {Xq.rows} x {Xq.cols}, expected {M} x {K}")
        xq = ctypes.byref(mx_struct(Xq, dev))
    else:
        _want(dA is None and dB is None, "dA and dB given with need_grads=False")
    with _on(dev):
        if dX is None and need_dx:
            dX = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
        if need_grads and dA is None:
            dA = torch.empty((r, K), dtype=torch.float32, device=dev)
        if need_grads and dB is None:
            dB = torch.empty((N, r), dtype=torch.float32, device=dev)
        ws, wp, wn = _workspace(ws, op, M, N, K, r, dev)
        _check(fn(dY.data_ptr(), xq, M, ctypes.byref(w), A.data_ptr(), B.data_ptr(), r, scale,
                  lq._ptr(T_saved), lq._ptr(dX), lq._ptr(dA), lq._ptr(dB), int(accumulate), wp, wn,
                  lq._stream()))
    return dX, dA, dB


def lq_mx_lora_bwd(dY, Xq, W0: MxTensor, A, B, scale, T_saved=None, need_dx=True, need_grads=True,
                   dX=None, dA=None, dB=None, accumulate=False, ws=None):
    """Xq: the MxTensor the forward multiplied (None with need_grads=False)."""
    dev = W0.codes.device
    return _backward(lib().lq_mx_lora_bwd, LQ_MX_OP_BWD, mx_struct(W0, dev), W0.rows, W0.cols, dev,
                     dY, Xq, A, B, scale, T_saved, need_dx, need_grads, dX, dA, dB, accumulate, ws)


def lq_lora_bwd_ckpt(dY, Xq, W0, A, B, scale, T_saved=None, need_dx=True, need_grads=True,
                     dX=None, dA=None, dB=None, accumulate=False, ws=None):
    """W0: a dense bf16 matrix or an NF4Weight; Xq: the MxTensor of the layer's
    input (None with need_grads=False)."""
    dev = dY.device
    w = lq.weight_struct(W0, lq.LQ_BF16)
    for t in ((W0.codes, W0.q8, W0.c2, W0.absmax) if isinstance(W0, NF4Weight) else (W0,)):
        _same_device(dev, t)
    if not isinstance(W0, NF4Weight):
        _want(W0.dtype == torch.bfloat16, "a dense W0 is bf16")
    return _backward(lib().lq_lora_bwd_ckpt, LQ_MX_OP_BWD_CKPT, w, w.N, w.K, dev, dY, Xq, A, B,
                     scale, T_saved, need_dx, need_grads, dX, dA, dB, accumulate, ws)
