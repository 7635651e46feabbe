"""Inputs and bounds shared by the tests of the operators around a projection."""
import numpy as np
import torch

from .gpu_helpers import DEV

U32 = 2.0**-24
HALF_BF16 = 2.0**-8


def host(x):
    """A device tensor as float64 in numpy (integers as they are)."""
    x = x.detach().cpu()
    return x.numpy() if not x.is_floating_point() else x.double().numpy()


def adapter_case(M, N, K, r, slots, ranks=None, rows="runs", seed=0):
    """A pool, rows and activations: numpy seeds, bf16 on the device.  Past the ranks
    in use the factors hold NaN."""
    rng = np.random.default_rng((M, N, K, r, slots, seed))
    t = lambda s, *shape: torch.from_numpy((rng.standard_normal(shape) * s).astype(np.float32)).to(torch.bfloat16)  # noqa: E731
    if ranks is None:
        ranks = np.where(rng.random(slots) < 0.5, r, rng.integers(1, r + 1, slots))
    ranks = np.asarray(ranks, np.int32)
    A, B = t(K**-0.5, slots, r, K), t(r**-0.5, slots, N, r)
    for a in range(slots):
        k = max(0, min(int(ranks[a]), r))
        A[a, k:] = float("nan")
        B[a, :, k:] = float("nan")
    if isinstance(rows, str):
        if rows == "runs":
            q = max(1, min(M, 7))
            rows = np.repeat(rng.integers(-1, slots, q), -(-M // q))[:M]
        elif rows == "random":
            rows = rng.integers(-1, slots + 1, M)
        else:
            rows = np.full(M, int(rows))
    c = dict(M=M, N=N, K=K, r=r, slots=slots, A=A, B=B, ranks=torch.from_numpy(ranks),
             scales=torch.from_numpy((0.5 + rng.random(slots)).astype(np.float32)),
             rows=torch.from_numpy(np.asarray(rows, np.int32).copy()), X=t(1.0, M, K), Y=t(1.3, M, N),
             dY=t(1.0, M, N), dX=t(1.3, M, K))
    return {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in c.items()}


def pool_arrays(c):
    """A, B (zeros past the ranks), scales, ranks, rows for the oracle."""
    A, B, ranks = host(c["A"]).copy(), host(c["B"]).copy(), host(c["ranks"])
    for a in range(c["slots"]):
        k = max(0, min(int(ranks[a]), c["r"]))
        A[a, k:] = 0.0
        B[a, :, k:] = 0.0
    return A, B, host(c["scales"]), ranks, host(c["rows"])


def within(got, want, slack, what, rel=0.0):
    err = np.abs(np.asarray(got, np.float64) - want)
    bad = ~(err <= rel * np.abs(want) + slack)
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(np.where(bad, err, 0.0))), bool(np.isnan(err).any()))
