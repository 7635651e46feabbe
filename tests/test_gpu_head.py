"""lq_head_loss against the oracle in float64.

Tolerances, u = 2^-24.  A logit is a float32 sum of K products, off by at most
e_z = K u scale |H||W|^T, and so are lse and a target's logit; exp, the sum over V
(a chain of at most V / 1024 + 32 additions per thread and across threads) and the
logarithm add (V / 1024 + 64) u relative to the sum and |z| u for the exponent's
product, taken twice.  D is rounded to bf16 (2^-8 of each entry) with an entry's
relative error 2 e_z before; dH is rounded once more."""
import numpy as np
import pytest
import torch

from oracle import block as oblock
from qlora_parameter_efficient_amd import block

from .block_helpers import HALF_BF16, U32, host, within
from .gpu_helpers import DEV, announce, bits

pytestmark = pytest.mark.gpu

SHAPES = [  # M, V, K, kt
    (1, 1, 64, 1), (1, 1000, 64, 1), (2, 255, 128, 3), (5, 256, 320, 1), (64, 257, 64, 2), (65, 500, 192, 1),
    (128, 1030, 256, 50), (129, 777, 576, 128), (130, 2000, 512, 1), (257, 1283, 64, 16), (300, 4096, 320, 1),
    (17, 20000, 128, 1), (9, 40001, 64, 5), (3, 70003, 64, 7), (1, 300001, 64, 2)]


def case(M, V, K, kt, seed=0):
    rng = np.random.default_rng((M, V, K, kt, seed))
    bf = lambda s, *shape: torch.from_numpy((rng.standard_normal(shape) * s).astype(np.float32)).to(torch.bfloat16).to(DEV)  # noqa: E731
    t = rng.integers(0, V, (M, kt))
    t[rng.random((M, kt)) < 0.1] = -1
    t[rng.random((M, kt)) < 0.05] = V + 7
    if M > 2:
        t[M // 2] = -1                      # a row without a target
        t[1] = t[1, 0] if V > 1 else t[1]   # one index kt times
    p = None if kt == 1 else rng.random((M, kt)).astype(np.float32)
    w = (rng.random(M) + 0.1).astype(np.float32)
    c = dict(H=bf(1.0, M, K), W=bf(2.0 * K**-0.5, V, K), t=t.astype(np.int32), p=p, w=w, scale=0.75)
    dev = lambda a: None if a is None else torch.from_numpy(a).to(DEV)  # noqa: E731
    c["dev"] = dict(targets=dev(c["t"]), p=dev(p), w=dev(w), logit_scale=0.75)
    return c


def check(c, loss, lse, dH):
    H, W, s = host(c["H"]), host(c["W"]), c["scale"]
    M, K, V = H.shape[0], H.shape[1], W.shape[0]
    want_loss, want_lse, want_d = oblock.head_loss(H, W, c["t"], c["p"], c["w"], s)
    z = s * (H @ W.T)
    e_z = (K * U32 * s * (np.abs(H) @ np.abs(W).T)).max(axis=1)
    e_lse = e_z + (V / 1024 + 64 + 4 * np.abs(z).max(axis=1)) * U32
    ok = (c["t"] >= 0) & (c["t"] < V)
    q = np.where(ok, 1.0 if c["p"] is None else c["p"], 0.0)
    if lse is not None:
        within(host(lse), want_lse, e_lse + np.abs(want_lse) * U32, "lse")
    if loss is not None:
        kt = q.shape[1]
        mag = (q * (np.abs(want_lse)[:, None] + np.abs(z).max(axis=1)[:, None])).sum(axis=1)
        within(host(loss), want_loss, q.sum(axis=1) * (e_lse + e_z) + (kt + 4) * U32 * mag, "loss")
    if dH is not None:
        soft = np.exp(z - want_lse[:, None])
        hot = np.zeros_like(z)
        for j in range(q.shape[1]):
            np.add.at(hot, (np.arange(M), np.where(ok[:, j], c["t"][:, j], 0)), q[:, j])
        share = np.where(ok.any(axis=1), c["w"] * s, 0.0)[:, None]
        d = np.abs(share) * np.abs(soft * q.sum(axis=1, keepdims=True) - hot)
        off = np.abs(share) * ((2 * e_lse[:, None] + (kt_terms(q) + 8) * U32) * (soft * q.sum(axis=1, keepdims=True))
                               + (kt_terms(q) + 8) * U32 * hot)
        slack = (d * (HALF_BF16 + V * U32) + off * (1 + HALF_BF16)) @ np.abs(W)
        within(host(dH), want_d, slack * (1 + HALF_BF16), "dH", HALF_BF16)
        assert (host(dH)[~ok.any(axis=1)] == 0).all()


def kt_terms(q):
    return q.shape[1]


@pytest.mark.parametrize("M,V,K,kt", SHAPES)
def test_loss_and_gradient(M, V, K, kt):
    announce(f"head M={M} V={V} K={K} kt={kt}")
    c = case(M, V, K, kt)
    loss, lse, dH = block.lq_head_loss(c["H"], c["W"], **c["dev"])
    check(c, loss, lse, dH)
    # the loss alone: the same bits
    loss2, lse2, none = block.lq_head_loss(c["H"], c["W"], **c["dev"], need_dh=False)
    assert none is None and np.array_equal(bits(loss2), bits(loss)) and np.array_equal(bits(lse2), bits(lse))


def test_labels_as_a_vector_and_defaults():
    c = case(70, 300, 128, 1)
    t = c["dev"]["targets"][:, 0].contiguous()
    loss, lse, dH = block.lq_head_loss(c["H"], c["W"], t)
    c.update(scale=1.0, w=np.ones(70, np.float32))
    check(c, loss, lse, dH)
    ref = torch.nn.functional.cross_entropy((c["H"].double() @ c["W"].double().t()), t.long().masked_fill(t >= 300, -1),
                                            ignore_index=-1, reduction="none")
    assert torch.allclose(loss.double(), ref, atol=1e-4)


def test_large_logits():
    """Logits far apart: the maximum carries the sum, nothing overflows."""
    c = case(40, 900, 64, 1)
    c["W"] = (c["W"].float() * 40).to(torch.bfloat16)
    loss, lse, dH = block.lq_head_loss(c["H"], c["W"], **c["dev"])
    assert torch.isfinite(loss).all() and torch.isfinite(dH).all()
    check(c, loss, lse, dH)


def test_rows_without_targets_hold_anything():
    c = case(50, 700, 128, 2)
    H, w = c["H"].clone(), c["dev"]["w"].clone()
    H[25] = float("nan")
    w[25] = float("inf")
    loss, lse, dH = block.lq_head_loss(H, c["W"], c["dev"]["targets"], c["dev"]["p"], w, 0.75)
    want = block.lq_head_loss(c["H"], c["W"], **c["dev"])
    keep = [i for i in range(50) if i != 25]
    assert loss[25] == 0 and (dH[25] == 0).all() and torch.isnan(lse[25])
    assert torch.equal(loss[keep], want[0][keep]) and torch.equal(dH[keep], want[2][keep])
    # a NaN in a row with a target stays in that row
    H[25] = 0
    H[3, 5] = float("nan")
    if bool((c["dev"]["targets"][3] < 0).all()):
        c["dev"]["targets"][3, 0] = 1
    loss, lse, dH = block.lq_head_loss(H, c["W"], **c["dev"])
    assert torch.isnan(loss[3]) and torch.isnan(dH[3]).all()
    keep = [i for i in range(50) if i not in (3, 25)]
    assert torch.equal(loss[keep], want[0][keep]) and torch.equal(dH[keep], want[2][keep])


def test_gradient_is_the_derivative():
    """Central differences of sum(w loss) in float64 through the oracle."""
    c = case(4, 130, 64, 3)
    _, _, dH = block.lq_head_loss(c["H"], c["W"], **c["dev"])
    H, W = host(c["H"]), host(c["W"])
    f = lambda H: float((c["w"] * oblock.head_loss(H, W, c["t"], c["p"], c["w"], 0.75)[0]).sum())  # noqa: E731
    top = np.abs(host(dH)).max()
    for i, k in [(0, 0), (1, 33), (3, 63)]:
        e = np.zeros_like(H)
        e[i, k] = 1e-4
        assert abs((f(H + e) - f(H - e)) / 2e-4 - float(dH[i, k])) <= 4 * HALF_BF16 * top


def test_several_pieces():
    """More logits than the workspace holds at a time: whole rows of pieces, and a
    last piece of another shape."""
    M, V, K = 700, 1 << 20, 64
    g = torch.Generator(device=DEV).manual_seed(3)
    H = torch.randn((M, K), generator=g, device=DEV).bfloat16()
    W = (torch.randn((V, K), generator=g, device=DEV) * 0.3).bfloat16()
    t = torch.randint(0, V, (M,), generator=g, device=DEV, dtype=torch.int32)
    assert block.lq_head_loss_workspace(M, V, K, 1, True) < 256 * V * 6 + (64 << 20)
    loss, lse, dH = block.lq_head_loss(H, W, t)
    for rows in (slice(0, 256), slice(256, 512), slice(512, 700)):
        part = block.lq_head_loss(H[rows].contiguous(), W, t[rows].contiguous())
        assert torch.equal(part[0], loss[rows]) and torch.equal(part[1], lse[rows]) and torch.equal(part[2], dH[rows])
    z = H[[0, 255, 256, 699]].double() @ W.double().t()
    assert torch.allclose(lse[[0, 255, 256, 699]].double(), torch.logsumexp(z, 1), atol=1e-4)


@pytest.mark.parametrize("M,V,K", [(1001, 50257, 192), (777, 33000, 320), (2048, 32000, 128), (200, 9999, 1024)])
def test_larger_shapes(M, V, K):
    """Several rounds of tiles, a second launch for a short last one, split
    reductions; the formulas in float64 on the GPU."""
    announce(f"head M={M} V={V} K={K}")
    g = torch.Generator(device=DEV).manual_seed(V)
    H = torch.randn((M, K), generator=g, device=DEV).bfloat16()
    W = (torch.randn((V, K), generator=g, device=DEV) * 2.0 * K**-0.5).bfloat16()
    t = torch.randint(0, V, (M,), generator=g, device=DEV, dtype=torch.int32)
    w = torch.rand(M, generator=g, device=DEV)
    loss, lse, dH = block.lq_head_loss(H, W, t, w=w)
    h, e = H.double(), W.double()
    z = h @ e.t()
    want = torch.logsumexp(z, 1)
    e_z = K * U32 * (h.abs() @ e.abs().t()).amax(1)
    e_lse = e_z + (V / 1024 + 64 + 4 * z.abs().amax(1)) * U32
    assert bool(((lse.double() - want).abs() <= e_lse + want.abs() * U32).all())
    zt = z.gather(1, t[:, None].long())[:, 0]
    assert bool(((loss.double() - (want - zt)).abs() <= e_lse + e_z + 8 * U32 * (want.abs() + zt.abs())).all())
    soft = torch.exp(z - want[:, None])
    d = soft.scatter_add(1, t[:, None].long(), -torch.ones_like(zt)[:, None]) * w[:, None].double()
    off = w[:, None].double() * (2 * e_lse[:, None] + 16 * U32) * (soft + 16 * U32)
    slack = (d.abs() * (HALF_BF16 + V * U32) + off * (1 + HALF_BF16)) @ e.abs()
    ref = d @ e
    assert bool(((dH.double() - ref).abs() <= HALF_BF16 * ref.abs() + slack * (1 + HALF_BF16)).all())
    # the errors above are worst cases; together the roundings are far smaller
    assert float((dH.double() - ref).norm() / ref.norm()) < 2 * HALF_BF16


@pytest.mark.parametrize("M,V", [(1, 256), (300, 256), (3, 2048), (130, 4096)])
def test_a_rows_largest_entry_is_not_rounded(M, V):
    """All logits 0 and one row of W not zero: dH = w (1 / V - 1) W_t, whose factor lies
    half a bf16 step off that type's values.  With the factor in bf16 dH would be
    off by up to two half steps; here it is rounded once, plus the float32
    factors' roundings."""
    g = torch.Generator(device=DEV).manual_seed(V)
    K = 256
    H = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    W = torch.zeros((V, K), dtype=torch.bfloat16, device=DEV)
    W[5] = torch.randn(K, generator=g, device=DEV).bfloat16()
    w = torch.full((M,), (1.0 + 2.0**-8 + 2.0**-13) * V / (V - 1), device=DEV)
    t = torch.full((M,), 5, dtype=torch.int32, device=DEV)
    _, _, dH = block.lq_head_loss(H, W, t, w=w)
    ref = w.double()[:, None] * (1.0 / V - 1.0) * W[5].double()
    assert bool(((dH.double() - ref).abs() <= (HALF_BF16 + (V + 32) * U32) * ref.abs()).all())
