"""ctypes binding of the MX entry points (include/lq_mx.h) of liblq.so.

As in lq.py, each function has the name of the C entry point it calls: it
checks placement, dtypes and shapes, allocates outputs and workspace with
torch, passes raw pointers and the current HIP stream of the tensors' device,
and raises LqError on a negative status.
"""
from __future__ import annotations

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
LQ_MX_OP_FWD, LQ_MX_OP_BWD, LQ_MX_OP_BWD_CKPT, LQ_MX_OP_BWD_CKPT_FUSED = 0, 1, 2, 3
LQ_MX_NO_GRADS = 16
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
    "lq_lora_bwd_ckpt_workspace": (_sz, [_i64, lq._WP, _i64, _i32, _i32]),
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


_BF16, _F32, _U8 = torch.bfloat16, torch.float32, torch.uint8
_DT = {_BF16: lq.LQ_BF16, _F32: lq.LQ_F32}
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(
    torch._C, "_cuda_getCurrentRawStream") else lambda i: torch.cuda.current_stream(i).cuda_stream


def _is(t, dtype, shape, dev, what):
    """Checks an operand (decode calls are a few microseconds: no helper calls
    on the way that passes)."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        if t.dtype is not dtype or t.shape != shape:
            raise ValueError(f"{what}: expected {dtype} of shape {tuple(shape)}, got {t.dtype} "
                             f"{tuple(t.shape)}")
        raise ValueError(f"{what}: tensors must be contiguous and on one GPU")
    return t.data_ptr()


@functools.lru_cache(maxsize=512)
def _buffer_bytes(fmt, rows, cols):
    return (lib().lq_mx_codes_bytes(fmt, rows, cols), lib().lq_mx_scales_bytes(rows, cols))


@functools.lru_cache(maxsize=1024)
def lq_mx_workspace_size(op, M, N, K, r):
    return int(lib().lq_mx_workspace_size(op, M, N, K, r))


@functools.lru_cache(maxsize=1024)
def lq_lora_bwd_ckpt_workspace(M, kind, N, K, r, need_dx=True, need_grads=True):
    """kind: lq.LQ_WEIGHT_DENSE or lq.LQ_WEIGHT_NF4."""
    w = LqWeightStruct()
    w.kind, w.dtype, w.N, w.K = kind, lq.LQ_BF16, N, K
    return int(lib().lq_lora_bwd_ckpt_workspace(M, ctypes.byref(w), r, int(need_dx),
                                                int(need_grads)))


def mx_struct(q: MxTensor, dev: int):
    """C descriptor of q after checking its buffers (dev: the GPU's index)."""
    fmt, rows, cols = FORMATS[q.format], q.rows, q.cols
    codes, scales = q.codes, q.scales
    if (codes.dtype is not _U8 or scales.dtype is not _U8 or codes.get_device() != dev
            or scales.get_device() != dev or not codes.is_contiguous()
            or not scales.is_contiguous()):
        raise ValueError("MX codes and scales are contiguous uint8 tensors on one GPU")
    if (codes.numel(), scales.numel()) != _buffer_bytes(fmt, rows, cols):
        raise ValueError(f"MX buffers do not hold a {rows} x {cols} {q.format} tensor")
    return LqMxStruct(fmt, 0, rows, cols, codes.data_ptr(), scales.data_ptr())


def _workspace(ws, size, args, like, dev):
    """(tensor that keeps it alive, pointer, bytes); ``ws`` is the caller's, or
    None for one of size(*args) bytes."""
    if ws is None:
        need = size(*args)
        if need == 0:
            return None, None, 0
        ws = like.new_empty(need, dtype=_U8)
        return ws, ws.data_ptr(), need
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("ws: tensors must be contiguous and on one GPU")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


_current = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _elsewhere(dev, fn, *args):
    """fn(*args) with dev, the GPU its tensors are on, as the current device."""
    if dev < 0:
        raise ValueError("tensors must be on the GPU")
    with torch.cuda.device(dev):
        return fn(*args)


# ------------------------------------------------------------------ calls

def lq_mx_quantize(X: torch.Tensor, format: str = "fp8") -> MxTensor:
    dev = X.get_device()
    if dev != _current():
        return _elsewhere(dev, lq_mx_quantize, X, format)
    if X.dim() != 2 or X.dtype not in _DT or not X.is_contiguous():
        raise ValueError("X must be a contiguous bf16 or float32 matrix")
    rows, cols = X.shape
    kb = -(-cols // LQ_MX_BLOCK)
    fmt = FORMATS[format]
    codes = X.new_empty((rows, kb * 4 * fmt), dtype=_U8)
    scales = X.new_empty((rows, kb), dtype=_U8)
    if rows == 0 and cols:  # an empty batch: the layer's calls take it, the codec has no work
        return MxTensor(codes, scales, rows, cols, format)
    _check(lib().lq_mx_quantize(X.data_ptr(), _DT[X.dtype], rows, cols, fmt, codes.data_ptr(),
                                scales.data_ptr(), _raw_stream(dev)))
    return MxTensor(codes, scales, rows, cols, format)


def lq_mx_dequantize(q: MxTensor, dtype=torch.bfloat16) -> torch.Tensor:
    dev = q.codes.get_device()
    if dev != _current():
        return _elsewhere(dev, lq_mx_dequantize, q, dtype)
    s = mx_struct(q, dev)
    _want(dtype in _DT, f"unsupported dtype {dtype}")
    out = q.codes.new_empty((q.rows, q.cols), dtype=dtype)
    if q.rows == 0 and q.cols:
        return out
    _check(lib().lq_mx_dequantize(ctypes.byref(s), out.data_ptr(), _DT[dtype], _raw_stream(dev)))
    return out


def _adapter(A, B, N, K, dev):
    """(rank, pointers of A and B)"""
    if A is None or B is None:
        _want(A is None and B is None, "A and B must both be given or both be None")
        return 0, None, None
    r = A.shape[0]
    return r, _is(A, _BF16, (r, K), dev, "A"), _is(B, _BF16, (N, r), dev, "B")


def lq_mx_lora_fwd(X, W0: MxTensor, A=None, B=None, scale=0.0, T_out=None, ws=None, Y=None):
    """X: a bf16 matrix (at most LQ_MX_ROWS_BF16 rows) or an MxTensor; A and B
    None: no adapter."""
    dev = W0.codes.get_device()
    if dev != _current():
        return _elsewhere(dev, lq_mx_lora_fwd, X, W0, A, B, scale, T_out, ws, Y)
    w = mx_struct(W0, dev)
    N, K = W0.rows, W0.cols
    if isinstance(X, MxTensor):
        M, like = X.rows, X.codes
        xq, xp = ctypes.byref(mx_struct(X, dev)), None
        _want(X.cols == K, f"X has {X.cols} columns, W0 {K}")
    else:
        M, like = X.shape[0], X
        xq, xp = None, _is(X, _BF16, (M, K), dev, "X")
    r, ap, bp = _adapter(A, B, N, K, dev)
    tp = None if T_out is None else _is(T_out, _F32, (M, r), dev, "T_out")
    if Y is None:
        Y = like.new_empty((M, N), dtype=_BF16)
        yp = Y.data_ptr()
    else:
        yp = _is(Y, _BF16, (M, N), dev, "Y")
    ws, wp, wn = _workspace(ws, lq_mx_workspace_size, (LQ_MX_OP_FWD, M, N, K, r), like, dev)
    _check(lib().lq_mx_lora_fwd(xp, xq, M, ctypes.byref(w), ap, bp, r, scale, yp, tp, wp, wn,
                                _raw_stream(dev)))
    return Y


def _backward(fn, kind, w, N, K, dev, dY, Xq, A, B, scale, T_saved, need_dx, need_grads, dX, dA, dB,
              accumulate, ws):
    """kind: None on an MXFP4 base, else that of the base."""
    M = dY.shape[0]
    yp = _is(dY, _BF16, (M, N), dev, "dY")
    r, ap, bp = _adapter(A, B, N, K, dev)
    _want(r > 0, "the backward needs an adapter")
    tp = None if T_saved is None else _is(T_saved, _F32, (M, r), dev, "T_saved")
    _want(not accumulate or not need_grads or (dA is not None and dB is not None),
          "accumulate needs dA and dB")
    xq = None
    if need_grads:
        _want((Xq.rows, Xq.cols) == (M, K), f"Xq is {Xq.rows} x {Xq.cols}, expected {M} x {K}")
        xq = ctypes.byref(mx_struct(Xq, dev))
        if dA is None:
            dA = dY.new_empty((r, K), dtype=_F32)
        if dB is None:
            dB = dY.new_empty((N, r), dtype=_F32)
    else:
        _want(dA is None and dB is None, "dA and dB given with need_grads=False")
    if dX is None and need_dx:
        dX = dY.new_empty((M, K), dtype=_BF16)
    xp = None if dX is None else _is(dX, _BF16, (M, K), dev, "dX")
    gap = None if dA is None else _is(dA, _F32, (r, K), dev, "dA")
    gbp = None if dB is None else _is(dB, _F32, (N, r), dev, "dB")
    if kind is None:
        size, args = lq_mx_workspace_size, (LQ_MX_OP_BWD + (0 if need_grads else LQ_MX_NO_GRADS),
                                            M, N, K, r)
    else:
        size, args = lq_lora_bwd_ckpt_workspace, (M, kind, N, K, r, dX is not None, need_grads)
    ws, wp, wn = _workspace(ws, size, args, dY, dev)
    _check(fn(yp, xq, M, ctypes.byref(w), ap, bp, r, scale, tp, xp, gap, gbp, int(accumulate), wp,
              wn, _raw_stream(dev)))
    return dX, dA, dB


def lq_mx_lora_bwd(dY, Xq, W0: MxTensor, A, B, scale, T_saved=None, need_dx=True,
                   need_grads=True, dX=None, dA=None, dB=None, accumulate=False, ws=None):
    """Xq: the MxTensor the forward multiplied (None with need_grads=False)."""
    dev = dY.get_device()
    if dev != _current():
        return _elsewhere(dev, lq_mx_lora_bwd, dY, Xq, W0, A, B, scale, T_saved, need_dx,
                          need_grads, dX, dA, dB, accumulate, ws)
    return _backward(lib().lq_mx_lora_bwd, None, mx_struct(W0, dev), W0.rows, W0.cols, dev,
                     dY, Xq, A, B, scale, T_saved, need_dx, need_grads, dX, dA, dB, accumulate, ws)


def lq_lora_bwd_ckpt(dY, Xq, W0, A, B, scale, T_saved=None, need_dx=True, need_grads=True,
                     dX=None, dA=None, dB=None, accumulate=False, ws=None):
    """W0: a dense bf16 matrix or an NF4Weight; Xq: the MxTensor of the layer's
    input (None with need_grads=False)."""
    dev = dY.get_device()
    if dev != _current():
        return _elsewhere(dev, lq_lora_bwd_ckpt, dY, Xq, W0, A, B, scale, T_saved, need_dx,
                          need_grads, dX, dA, dB, accumulate, ws)
    nf4 = isinstance(W0, NF4Weight)
    for t in (W0.codes, W0.q8, W0.c2, W0.absmax) if nf4 else (W0,):
        _want(t is None or t.get_device() == dev, "W0: tensors must be on one GPU")
    _want(nf4 or W0.dtype is _BF16, "a dense W0 is bf16")
    w = lq.weight_struct(W0, lq.LQ_BF16)
    return _backward(lib().lq_lora_bwd_ckpt, w.kind, w, w.N, w.K, dev, dY, Xq, A, B,
                     scale, T_saved, need_dx, need_grads, dX, dA, dB, accumulate, ws)
