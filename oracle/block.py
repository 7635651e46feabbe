"""The operators around an adapted projection, in float64 from their formulas:
the RMS norm of a residual stream, adapters of many requests beside a shared
projection, the loss of a large-vocabulary head."""
import numpy as np


def rmsnorm(H, w, eps):
    """(y, c): y = H w c with c = 1 / sqrt(mean(H^2) + eps) of each row."""
    H = np.asarray(H, np.float64)
    c = 1.0 / np.sqrt((H * H).mean(axis=1) + eps)
    return H * c[:, None] * np.asarray(w, np.float64), c


def rmsnorm_backward(dY, H, w, c, dH=None):
    """(dX, dW) of rmsnorm; dH: the gradient that reaches H by its other uses."""
    dY, H = np.asarray(dY, np.float64), np.asarray(H, np.float64)
    c = np.asarray(c, np.float64)[:, None]
    g = dY * np.asarray(w, np.float64)
    dX = c * g - H * c**3 * (g * H).mean(axis=1, keepdims=True)
    if dH is not None:
        dX = dX + np.asarray(dH, np.float64)
    return dX, (dY * H * c).sum(axis=0)


def _members(rows, slot):
    return np.nonzero(np.asarray(rows) == slot)[0]


def adapters_forward(X, A, B, scales, ranks, rows, Y):
    """(Y plus each row's adapter, T); rows outside the pool have none."""
    X, Y = np.asarray(X, np.float64), np.array(Y, np.float64)
    T = np.zeros((X.shape[0], A.shape[1]))
    for a in range(A.shape[0]):
        i, k = _members(rows, a), max(0, min(int(ranks[a]), A.shape[1]))
        if len(i) == 0:
            continue
        T[i, :k] = X[i] @ A[a, :k].astype(np.float64).T
        Y[i] += float(scales[a]) * (T[i, :k] @ B[a, :, :k].astype(np.float64).T)
    return Y, T


def adapters_backward(dY, X, A, B, scales, ranks, rows, dX, T):
    """(dX plus each row's share, dA, dB, U)"""
    dY, X, dX = np.asarray(dY, np.float64), np.asarray(X, np.float64), np.array(dX, np.float64)
    dA, dB = np.zeros(A.shape), np.zeros(B.shape)
    U = np.zeros((dY.shape[0], A.shape[1]))
    for a in range(A.shape[0]):
        i, k = _members(rows, a), max(0, min(int(ranks[a]), A.shape[1]))
        if len(i) == 0:
            continue
        s = float(scales[a])
        U[i, :k] = dY[i] @ B[a, :, :k].astype(np.float64)
        dX[i] += s * (U[i, :k] @ A[a, :k].astype(np.float64))
        dA[a, :k] = s * (U[i, :k].T @ X[i])
        dB[a, :, :k] = s * (dY[i].T @ np.asarray(T, np.float64)[i, :k])
    return dX, dA, dB, U


def head_loss(H, W, targets, p, w, scale):
    """(loss, lse, dH): cross entropy of softmax(scale H W^T) against the weighted
    targets of each row (entries outside the vocabulary are none), its log sum of
    exponentials, and the gradient of sum(w loss)."""
    H, W = np.asarray(H, np.float64), np.asarray(W, np.float64)
    M, V = H.shape[0], W.shape[0]
    z = float(scale) * (H @ W.T)
    top = z.max(axis=1)
    e = np.exp(z - top[:, None])
    lse = top + np.log(e.sum(axis=1))
    hot = np.zeros((M, V))
    loss = np.zeros(M)
    for i in range(M):
        for j, t in enumerate(targets[i]):
            if 0 <= t < V:
                q = 1.0 if p is None else float(p[i][j])
                hot[i, t] += q
                loss[i] += q * (lse[i] - z[i, t])
    any_ = ((targets >= 0) & (targets < V)).any(axis=1)
    d = np.exp(z - lse[:, None]) * hot.sum(axis=1, keepdims=True) - hot
    d *= (float(scale) * np.asarray(w, np.float64))[:, None]
    dH = np.where(any_[:, None], np.where(any_[:, None], d, 0.0) @ W, 0.0)
    return np.where(any_, loss, 0.0), lse, dH
