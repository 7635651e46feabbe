"""lq_head_loss over many short rows, and rows that are confident or not finite."""
import pytest
import torch

from qlora_parameter_efficient_amd import block

from .block_helpers import HALF_BF16, U32
from .gpu_helpers import DEV, announce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,V", [((1 << 21) + 77, 64), ((1 << 22) + 5, 3)])
def test_more_short_rows_than_a_launch_takes(M, V):
    """1024 threads a row: 2^22 rows would be 2^32 threads.  Logits of 64 products of bf16
    values, exact to 64 u of their magnitudes; at most 64 exponentials of a row in a
    chain of 32 additions."""
    announce(f"head M={M} V={V}")
    K = 64
    g = torch.Generator(device=DEV).manual_seed(V)
    H = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)
    for part in H.split(1 << 20):
        part.copy_(torch.randn(part.shape, generator=g, device=DEV))
    W = (torch.randn((V, K), generator=g, device=DEV) * 0.25).bfloat16()
    t = torch.randint(0, V, (M,), generator=g, device=DEV, dtype=torch.int32)
    loss, lse, dH = block.lq_head_loss(H, W, t)
    w = W.double()
    for i in torch.arange(M, device=DEV).split(1 << 18):
        h = H[i].double()
        z = h @ w.t()
        e_z = K * U32 * (h.abs() @ w.abs().t()).amax(1)
        want, zt = torch.logsumexp(z, 1), z.gather(1, t[i, None].long())[:, 0]
        e = e_z + (64 + 4 * z.abs().amax(1)) * U32
        assert bool(((lse[i].double() - want).abs() <= e + want.abs() * U32).all()), int(i[0])
        assert bool(((loss[i].double() - (want - zt)).abs() <= e + e_z + 8 * U32 * (want.abs() + zt.abs())).all()), int(i[0])
        soft = torch.exp(z - want[:, None])
        d = soft.scatter_add(1, t[i, None].long(), -torch.ones_like(zt)[:, None])
        slack = (d.abs() * (HALF_BF16 + V * U32) + (2 * e[:, None] + 16 * U32) * (soft + 16 * U32) * (1 + HALF_BF16)) @ w.abs()
        ref = d @ w
        assert bool(((dH[i].double() - ref).abs() <= HALF_BF16 * ref.abs() + slack * (1 + HALF_BF16)).all()), int(i[0])


@pytest.mark.parametrize("V", [300, 5000, 70001])
def test_lse_does_not_depend_on_the_targets(V):
    """The same bits with any target, among the largest logits or not, or several."""
    announce(f"lse of any target V={V}")
    g = torch.Generator(device=DEV).manual_seed(V)
    H = torch.randn((9, 64), generator=g, device=DEV).bfloat16()
    W = (torch.randn((V, 64), generator=g, device=DEV) * 0.5).bfloat16()
    top = (H.float() @ W.float().t()).topk(8, 1).indices.int()
    want = block.lq_head_loss(H, W, torch.full((9,), -1, dtype=torch.int32, device=DEV))[1]
    for t in (top[:, 0].contiguous(), top[:, 7].contiguous(), top.contiguous(), torch.full_like(top[:, 0], V - 1)):
        assert torch.equal(block.lq_head_loss(H, W, t)[1], want)
