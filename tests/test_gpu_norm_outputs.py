"""The RMS norm's outputs over its inputs' buffers, and its MX output of a residual sum."""
import pytest
import torch

from qlora_parameter_efficient_amd import block, mx

from .gpu_helpers import DEV, announce

pytestmark = pytest.mark.gpu
SHAPES = [(3, 15), (9, 64), (6, 1024), (700, 1100), (16, 4097), (1500, 4096), (3, 11008), (2, 16385), (300, 30000), (1, 65536)]


def draw(M, K, dt, n):
    g = torch.Generator(device=DEV).manual_seed(M * K)
    return [torch.randn((M, K), generator=g, device=DEV).to(dt) for _ in range(n)] + [1 + 0.2 * torch.randn(K, generator=g, device=DEV)]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", SHAPES)
def test_dx_over_each_input(M, K, dt):
    """dX may be dY, dH or H: the bits of a buffer of its own, and the others untouched."""
    announce(f"rmsnorm bwd over its inputs {M}x{K} {dt}")
    dY, H, dH, W = draw(M, K, dt, 3)
    want, dw = block.lq_rmsnorm_bwd(dY, H, W, 1e-5, dH=dH)
    for over in ("dY", "dH", "H"):
        b = dict(dY=dY.clone(), H=H.clone(), dH=dH.clone())
        got, dw2 = block.lq_rmsnorm_bwd(b["dY"], b["H"], W, 1e-5, dH=b["dH"], dX=b[over])
        assert got is b[over] and torch.equal(got, want) and torch.equal(dw2, dw), over
        for name, t in (("dY", dY), ("H", H), ("dH", dH)):
            assert name == over or torch.equal(b[name], t), (over, name)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", SHAPES)
def test_mx_output_of_a_residual_sum(M, K, dt, fmt):
    """The codes are the quantiser's of y = H c w in the kernel's two float32 products, with
    its H (the rounded sum) and its c; H over R and over X too."""
    announce(f"rmsnorm fwd residual {M}x{K} {dt} {fmt}")
    X, R, W = draw(M, K, dt, 2)
    c = torch.empty(M, device=DEV)
    H, Y, q = block.lq_rmsnorm_fwd(X, W, 1e-5, R=R, format=fmt, rstd_out=c)
    assert torch.equal(H, (X.float() + R.float()).to(dt))
    y = H.float() * c[:, None] * W
    want = mx.lq_mx_quantize(y, fmt)
    assert torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales)
    assert torch.equal(Y, y.to(dt))
    for over in (0, 1):
        b = [X.clone(), R.clone()]
        H2, none, q2 = block.lq_rmsnorm_fwd(b[0], W, 1e-5, R=b[1], format=fmt, need_y=False, H_out=b[over])
        assert none is None and H2 is b[over] and torch.equal(H2, H)
        assert torch.equal(q2.codes, q.codes) and torch.equal(q2.scales, q.scales)
