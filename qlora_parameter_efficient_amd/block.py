"""ctypes binding of the operators around an adapted projection
(include/lq_block.h) of liblq.so.

As in lq.py and mx.py, each function has the name of the C entry point it calls:
it checks placement, dtypes and shapes, allocates outputs and workspace with
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
from .lq import LqError, LqWeightStruct  # noqa: F401
from .mx import (FORMATS, LQ_MX_BLOCK, MxTensor, _BF16, _DT, _F32, _U8, _current, _elsewhere, _is, _raw_stream,
                 _want, _workspace)

HEADER = os.path.join(os.path.dirname(lq.HEADER), "lq_block.h")

LQ_ADAPTERS_MAX_SLOTS = 4096
LQ_ADAPTERS_OP_FWD, LQ_ADAPTERS_OP_BWD = 0, 1


class LqAdapterPoolStruct(ctypes.Structure):
    _fields_ = [("slots", ctypes.c_int32), ("r", ctypes.c_int32), ("N", ctypes.c_int64),
                ("K", ctypes.c_int64), ("A", ctypes.c_void_p), ("B", ctypes.c_void_p),
                ("ranks", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


_vp, _i32, _i64, _f32, _sz = lq._vp, lq._i32, lq._i64, lq._f32, lq._sz
_PP = ctypes.POINTER(LqAdapterPoolStruct)

_SIGS = {
    "lq_rmsnorm_fwd": (ctypes.c_int, [_vp, _vp, _i64, _i64, _i32, _vp, _i32, _f32, _vp, _vp, _i32, _vp,
                                      _vp, _vp, _vp]),
    "lq_rmsnorm_bwd": (ctypes.c_int, [_vp, _vp, _i64, _i64, _i32, _vp, _i32, _f32, _vp, _vp, _vp, _vp,
                                      _i32, _vp, _sz, _vp]),
    "lq_rmsnorm_bwd_workspace": (_sz, [_i64, _i64]),
    "lq_adapters_fwd": (ctypes.c_int, [_vp, _i64, _PP, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "lq_adapters_bwd": (ctypes.c_int, [_vp, _vp, _i64, _PP, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp,
                                       _sz, _vp]),
    "lq_adapters_workspace_size": (_sz, [_i32, _i64, _i64, _i64, _i64, _i32]),
    "lq_head_loss": (ctypes.c_int, [_vp, _i64, lq._WP, _vp, _vp, _i32, _vp, _f32, _vp, _vp, _vp, _vp,
                                    _sz, _vp]),
    "lq_head_loss_workspace": (_sz, [_i64, _i64, _i64, _i32, _i32]),
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


def _check(rc):
    if rc != 0:
        raise LqError(rc, lib().lq_last_error().decode())


# ------------------------------------------------------------------- norm

@functools.lru_cache(maxsize=1024)
def lq_rmsnorm_bwd_workspace(M, K):
    return int(lib().lq_rmsnorm_bwd_workspace(M, K))


def _matrix(X, what):
    """(rows, columns) of a contiguous bf16 or float32 matrix"""
    if X.dim() != 2 or X.dtype not in _DT or not X.is_contiguous():
        raise ValueError(f"{what} must be a contiguous bf16 or float32 matrix")
    return X.shape


def _gain(W, K, dev):
    if W.dtype not in _DT:
        raise ValueError("W must be bf16 or float32")
    return _is(W, W.dtype, (K,), dev, "W")


def lq_rmsnorm_fwd(X, W, eps=1e-6, R=None, need_y=True, format=None, H_out=None, Y=None,
                   rstd_out=None):
    """(H, Y, q): the residual stream H = X + R (X itself where R is None and no
    H_out is given), y in X's type (None with need_y=False) and as an MxTensor
    (None without a format, "fp8" or "fp4")."""
    dev = X.get_device()
    if dev != _current():
        return _elsewhere(dev, lq_rmsnorm_fwd, X, W, eps, R, need_y, format, H_out, Y, rstd_out)
    M, K = _matrix(X, "X")
    dt = X.dtype
    wp = _gain(W, K, dev)
    rp = None if R is None else _is(R, dt, (M, K), dev, "R")
    if H_out is None:
        if R is None:
            H_out, hp = X, None
        else:
            H_out = torch.empty_like(X)
            hp = H_out.data_ptr()
    else:
        hp = _is(H_out, dt, (M, K), dev, "H_out")
    if Y is None and need_y:
        Y = torch.empty_like(X)
    yp = None if Y is None else _is(Y, dt, (M, K), dev, "Y")
    tp = None if rstd_out is None else _is(rstd_out, _F32, (M,), dev, "rstd_out")
    q, fmt, cp, sp = None, 0, None, None
    if format is not None:
        fmt, kb = FORMATS[format], -(-K // LQ_MX_BLOCK)
        codes = X.new_empty((M, kb * 4 * fmt), dtype=_U8)
        scales = X.new_empty((M, kb), dtype=_U8)
        q, cp, sp = MxTensor(codes, scales, M, K, format), codes.data_ptr(), scales.data_ptr()
    _want(Y is not None or q is not None, "nothing to write: need_y or a format")
    if M:
        _check(lib().lq_rmsnorm_fwd(X.data_ptr(), rp, M, K, _DT[dt], wp, _DT[W.dtype], eps, hp, yp,
                                    fmt, cp, sp, tp, _raw_stream(dev)))
    return H_out, Y, q


def lq_rmsnorm_bwd(dY, H, W, eps=1e-6, rstd=None, dH=None, need_dx=True, need_dw=True, dX=None,
                   dW=None, accumulate=False, ws=None):
    """(dX, dW); dH: the gradient that reaches H by its other uses."""
    dev = dY.get_device()
    if dev != _current():
        return _elsewhere(dev, lq_rmsnorm_bwd, dY, H, W, eps, rstd, dH, need_dx, need_dw, dX, dW,
                          accumulate, ws)
    M, K = _matrix(dY, "dY")
    dt = dY.dtype
    hp, wp = _is(H, dt, (M, K), dev, "H"), _gain(W, K, dev)
    cp = None if rstd is None else _is(rstd, _F32, (M,), dev, "rstd")
    gp = None if dH is None else _is(dH, dt, (M, K), dev, "dH")
    _want(not accumulate or not need_dw or dW is not None, "accumulate needs dW")
    _want(need_dw or dW is None, "dW given with need_dw=False")
    if dX is None and need_dx:
        dX = torch.empty_like(dY)
    xp = None if dX is None else _is(dX, dt, (M, K), dev, "dX")
    if dW is None and need_dw:
        dW = dY.new_empty((K,), dtype=_F32)
    dwp = None if dW is None else _is(dW, _F32, (K,), dev, "dW")
    wsp, wsn = None, 0
    if dW is not None:
        ws, wsp, wsn = _workspace(ws, lq_rmsnorm_bwd_workspace, (M, K), dY, dev)
    _check(lib().lq_rmsnorm_bwd(dY.data_ptr(), hp, M, K, _DT[dt], wp, _DT[W.dtype], eps, cp, gp, xp,
                                dwp, int(accumulate), wsp, wsn, _raw_stream(dev)))
    return dX, dW


# --------------------------------------------------------------- adapters

@dataclass
class AdapterPool:
    """Device tensors of the adapters of one projection, each in a place of its own."""
    A: torch.Tensor                 # slots x r x K bf16
    B: torch.Tensor                 # slots x N x r bf16
    scales: torch.Tensor            # float32, slots
    ranks: torch.Tensor | None = None   # int32, slots: the ranks in use; None: r everywhere


@functools.lru_cache(maxsize=1024)
def lq_adapters_workspace_size(op, M, N, K, r, slots):
    return int(lib().lq_adapters_workspace_size(op, M, N, K, r, slots))


_I32 = torch.int32


def _pool(q: AdapterPool, dev):
    """C descriptor of the pool after checking its tensors."""
    if q.A.dim() != 3 or q.B.dim() != 3:
        raise ValueError("the pool's A is slots x r x K and B slots x N x r")
    slots, r, K = q.A.shape
    N = q.B.shape[1]
    s = LqAdapterPoolStruct(slots, r, N, K, _is(q.A, _BF16, (slots, r, K), dev, "A"),
                            _is(q.B, _BF16, (slots, N, r), dev, "B"),
                            None if q.ranks is None else _is(q.ranks, _I32, (slots,), dev, "ranks"),
                            _is(q.scales, _F32, (slots,), dev, "scales"))
    return s


def lq_adapters_fwd(X, pool: AdapterPool, rows, Y, out=None, T_out=None, ws=None):
    """Y plus each row's adapter (rows: int32, its place in the pool, or outside
    it for none); out=Y adds in place."""
    dev = X.get_device()
    if dev != _current():
        return _elsewhere(dev, lq_adapters_fwd, X, pool, rows, Y, out, T_out, ws)
    q = _pool(pool, dev)
    M, N, K, r = X.shape[0], q.N, q.K, q.r
    xp, ip = _is(X, _BF16, (M, K), dev, "X"), _is(rows, _I32, (M,), dev, "rows")
    yp = _is(Y, _BF16, (M, N), dev, "Y")
    tp = None if T_out is None else _is(T_out, _F32, (M, r), dev, "T_out")
    if out is None:
        out = torch.empty_like(Y)
    op = _is(out, _BF16, (M, N), dev, "out")
    ws, wp, wn = _workspace(ws, lq_adapters_workspace_size, (LQ_ADAPTERS_OP_FWD, M, N, K, r, q.slots),
                            X, dev)
    _check(lib().lq_adapters_fwd(xp, M, ctypes.byref(q), ip, yp, op, tp, wp, wn, _raw_stream(dev)))
    return out


def lq_adapters_bwd(dY, X, pool: AdapterPool, rows, dX=None, T_saved=None, need_grads=True, out=None,
                    dA=None, dB=None, accumulate=False, ws=None):
    """(dX + each row's share, dA, dB); dX: the gradient that came through the
    shared projection (None: only dA and dB); out=dX adds in place."""
    dev = dY.get_device()
    if dev != _current():
        return _elsewhere(dev, lq_adapters_bwd, dY, X, pool, rows, dX, T_saved, need_grads, out, dA, dB,
                          accumulate, ws)
    q = _pool(pool, dev)
    M, N, K, r, slots = dY.shape[0], q.N, q.K, q.r, q.slots
    gp, ip = _is(dY, _BF16, (M, N), dev, "dY"), _is(rows, _I32, (M,), dev, "rows")
    _want(dX is not None or out is None, "out without dX")
    dxp = op = None
    if dX is not None:
        dxp = _is(dX, _BF16, (M, K), dev, "dX")
        if out is None:
            out = torch.empty_like(dX)
        op = _is(out, _BF16, (M, K), dev, "out")
    xp = tp = None
    if need_grads:
        xp = _is(X, _BF16, (M, K), dev, "X")
        tp = None if T_saved is None else _is(T_saved, _F32, (M, r), dev, "T_saved")
        _want(not accumulate or (dA is not None and dB is not None), "accumulate needs dA and dB")
        if dA is None:
            dA = dY.new_empty((slots, r, K), dtype=_F32)
        if dB is None:
            dB = dY.new_empty((slots, N, r), dtype=_F32)
    else:
        _want(dA is None and dB is None, "dA and dB given with need_grads=False")
    ap = None if dA is None else _is(dA, _F32, (slots, r, K), dev, "dA")
    bp = None if dB is None else _is(dB, _F32, (slots, N, r), dev, "dB")
    ws, wp, wn = _workspace(ws, lq_adapters_workspace_size, (LQ_ADAPTERS_OP_BWD, M, N, K, r, slots), dY,
                            dev)
    _check(lib().lq_adapters_bwd(gp, xp, M, ctypes.byref(q), ip, tp, dxp, op, ap, bp, int(accumulate),
                                 wp, wn, _raw_stream(dev)))
    return out, dA, dB


# ------------------------------------------------------------------- head

@functools.lru_cache(maxsize=1024)
def lq_head_loss_workspace(M, V, K, kt, need_dh):
    return int(lib().lq_head_loss_workspace(M, V, K, kt, int(need_dh)))


def lq_head_loss(H, W0, targets, p=None, w=None, logit_scale=1.0, need_dh=True, dH=None, loss=None,
                 lse=None, ws=None):
    """(loss, lse, dH) of a frozen bf16 head W0 (V x K): targets int32, M (labels)
    or M x kt; p: their weights (None: 1); w: the rows' shares of the total whose
    gradient dH is (None: 1)."""
    dev = H.get_device()
    if dev != _current():
        return _elsewhere(dev, lq_head_loss, H, W0, targets, p, w, logit_scale, need_dh, dH, loss, lse,
                          ws)
    if H.dim() != 2 or W0.dim() != 2:
        raise ValueError("H and W0 are matrices")
    M, (V, K) = H.shape[0], W0.shape
    hp = _is(H, _BF16, (M, K), dev, "H")
    s = LqWeightStruct()
    s.kind, s.dtype, s.N, s.K = lq.LQ_WEIGHT_DENSE, lq.LQ_BF16, V, K
    s.dense = _is(W0, _BF16, (V, K), dev, "W0")
    kt = 1 if targets.dim() == 1 else targets.shape[1]
    tp = _is(targets, _I32, (M,) if targets.dim() == 1 else (M, kt), dev, "targets")
    pp = None if p is None else _is(p, _F32, targets.shape, dev, "p")
    sp = None if w is None else _is(w, _F32, (M,), dev, "w")
    if loss is None:
        loss = H.new_empty((M,), dtype=_F32)
    if lse is None:
        lse = H.new_empty((M,), dtype=_F32)
    if dH is None and need_dh:
        dH = torch.empty_like(H)
    lp, ep = _is(loss, _F32, (M,), dev, "loss"), _is(lse, _F32, (M,), dev, "lse")
    dp = None if dH is None else _is(dH, _BF16, (M, K), dev, "dH")
    ws, wp, wn = _workspace(ws, lq_head_loss_workspace, (M, V, K, kt, dH is not None), H, dev)
    _check(lib().lq_head_loss(hp, M, ctypes.byref(s), tp, pp, kt, sp, logit_scale, lp, ep, dp, wp, wn,
                              _raw_stream(dev)))
    return loss, lse, dH
