"""lq_head_loss where logits are infinite: the log sum of exponentials is +inf with a
logit of +inf, -inf where all are -inf, and NaN with a NaN among them."""
import pytest
import torch

from qlora_parameter_efficient_amd import block

from .gpu_helpers import DEV, announce

pytestmark = pytest.mark.gpu
INF = float("inf")


def logits_by_row(M, V, K=64):
    """H and W whose logit of (i, v) is H[i, 0] W[v, 0] but for 63 zero products."""
    H = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    W = torch.zeros((V, K), dtype=torch.bfloat16, device=DEV)
    H[:, 0] = 1.0
    g = torch.Generator(device=DEV).manual_seed(V)
    W[:, 1:] = torch.randn((V, K - 1), generator=g, device=DEV).bfloat16()
    return H, W


# (rows of 70003 are longer than a workgroup keeps; 3 and 130 rows split their sums differently)
@pytest.mark.parametrize("M", [3, 130])
@pytest.mark.parametrize("V", [40, 2000, 70003])
def test_one_infinite_logit(M, V):
    announce(f"head with an infinite logit M={M} V={V}")
    H, W = logits_by_row(M, V)
    H[1, 0] = -1.0
    W[V - 1, 0] = INF  # rows 0, 2, ...: +inf; row 1: -inf
    t = torch.full((M,), 2, dtype=torch.int32, device=DEV)
    loss, lse, dH = block.lq_head_loss(H, W, t)
    plus = torch.arange(M, device=DEV) != 1
    assert bool((lse[plus] == INF).all()) and bool((loss[plus] == INF).all())
    # softmax of such a row is inf / inf
    assert bool(torch.isnan(dH[plus]).all())
    # row 1: V - 1 logits of 0
    want = torch.log(torch.tensor(float(V - 1), dtype=torch.float64)).item()
    assert abs(float(lse[1]) - want) <= (V / 1024 + 64) * 2.0**-24 * max(1.0, want)
    assert bool(torch.isfinite(loss[1])) and bool(torch.isfinite(dH[1, 1:]).all())
    # the infinite logit as the target
    t.fill_(V - 1)
    loss, lse2, dH = block.lq_head_loss(H, W, t)
    assert torch.equal(lse2, lse) and loss[1] == INF and bool(torch.isnan(loss[plus]).all())
    assert bool(torch.isnan(dH[plus]).all()) and bool(torch.isfinite(dH[1, 1:]).all())


@pytest.mark.parametrize("V", [40, 2000, 70003])
def test_all_logits_minus_infinity(V):
    announce(f"head with all logits -inf V={V}")
    H, W = logits_by_row(5, V)
    H[0, 0] = -1.0
    W[:, 0] = INF
    t = torch.zeros(5, dtype=torch.int32, device=DEV)
    t[4] = -1
    loss, lse, dH = block.lq_head_loss(H, W, t)
    assert lse[0] == -INF and bool(torch.isnan(loss[0])) and bool(torch.isnan(dH[0]).all())
    assert bool((lse[1:] == INF).all())
    # (without a target: loss 0 whatever the logits are)
    assert loss[4] == 0


@pytest.mark.parametrize("V", [40, 2000, 70003])
def test_a_nan_beside_an_infinite_logit(V):
    announce(f"head with NaN and inf V={V}")
    H, W = logits_by_row(3, V)
    W[7, 0] = INF
    W[V // 2 + 1, 0] = float("nan")
    loss, lse, dH = block.lq_head_loss(H, W, torch.full((3,), 5, dtype=torch.int32, device=DEV))
    assert bool(torch.isnan(lse).all()) and bool(torch.isnan(loss).all()) and bool(torch.isnan(dH).all())
