"""The operators around a projection together, as a step uses them: a training
step of several adapters on one base, a serving step captured into a graph, and
calls on several streams."""
import numpy as np
import pytest
import torch

from oracle import block as oblock
from oracle import lora as olora
from qlora_parameter_efficient_amd import block, lq, mx

from .block_helpers import adapter_case, host, pool_arrays
from .gpu_helpers import BF16_TOL, DEV, announce, rel_err

pytestmark = pytest.mark.gpu


def bf(seed, sigma, *shape):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * sigma).to(torch.bfloat16).to(DEV)


def pool(c):
    return block.AdapterPool(c["A"], c["B"], c["scales"], c["ranks"])


def test_training_step_of_several_adapters():
    """Norm, a projection with an adapter of its own, the requests' adapters, the
    loss, and all gradients, against the same chain in float64 (the framework's bar
    for bf16 results: every tensor of the chain is rounded to bf16 once)."""
    M, N, K, V, r = 300, 256, 320, 1000, 8
    c = adapter_case(M, N, K, r, 5, seed=7)
    X, R, G = bf(1, 1.0, M, K), bf(2, 1.0, M, K), bf(3, 1e-3, M, K)
    gain = torch.linspace(0.5, 1.5, K, device=DEV)
    W, A0, B0, head = bf(4, K**-0.5, N, K), bf(5, K**-0.5, 4, K), bf(6, 0.3, N, 4), bf(7, 2 * N**-0.5, V, N)
    t = torch.randint(0, V, (M,), device=DEV, dtype=torch.int32)
    t[::7] = -1
    w = torch.full((M,), 1.0 / M, device=DEV)
    announce("a training step")
    rstd, T0, T = torch.empty(M, device=DEV), torch.empty((M, 4), device=DEV), torch.empty((M, r), device=DEV)
    H, y, _ = block.lq_rmsnorm_fwd(X, gain, 1e-5, R=R, rstd_out=rstd)
    Y = lq.lq_lora_fwd(y, W, A0, B0, 0.5, T_out=T0)
    block.lq_adapters_fwd(y, pool(c), c["rows"], Y, out=Y, T_out=T)
    loss, lse, dY = block.lq_head_loss(Y, head, t, w=w)
    dy, dA0, dB0 = lq.lq_lora_bwd(dY, y, W, A0, B0, 0.5, T_saved=T0)
    dy, dA, dB = block.lq_adapters_bwd(dY, y, pool(c), c["rows"], dy, T_saved=T, out=dy)
    dX, dgain = block.lq_rmsnorm_bwd(dy, H, gain, 1e-5, rstd=rstd, dH=G)
    # the same in float64
    A, B, s, ranks, rows = pool_arrays(c)
    h = host(X) + host(R)
    oy, oc = oblock.rmsnorm(h, host(gain), 1e-5)
    oY, _, _ = olora.lora_forward(oy, host(W), host(A0), host(B0), 0.5)
    oY, oT = oblock.adapters_forward(oy, A, B, s, ranks, rows, oY)
    oloss, olse, odY = oblock.head_loss(oY, host(head), host(t)[:, None], None, host(w), 1.0)
    ody, odA0, odB0 = olora.lora_backward(odY, oy, host(W), host(A0), host(B0), 0.5)
    ody, odA, odB, _ = oblock.adapters_backward(odY, oy, A, B, s, ranks, rows, ody, oT)
    odX, odg = oblock.rmsnorm_backward(ody, h, host(gain), oc, host(G))
    for name, got, want in (("H", H, h), ("y", y, oy), ("Y", Y, oY), ("loss", loss, oloss), ("lse", lse, olse), ("dY", dY, odY),
                            ("dA0", dA0, odA0), ("dB0", dB0, odB0), ("dy", dy, ody), ("dA", dA, odA), ("dB", dB, odB),
                            ("dX", dX, odX), ("dgain", dgain, odg)):
        assert rel_err(host(got), want) <= BF16_TOL, (name, rel_err(host(got), want))
    # the factors of the places that have rows move, the others stay
    master = c["A"].float().nan_to_num(0.0)
    before = master.clone()
    m, v = torch.zeros_like(master), torch.zeros_like(master)
    lq.lq_adamw_step([(master, m, v, dA, None)], 1, 1e-2)
    used = sorted(set(rows.tolist()) & set(range(5)))
    for a in range(5):
        assert torch.equal(master[a], before[a]) == (a not in used), a


def test_serving_step_in_a_graph():
    """Norm to bf16 and MXFP8 at once, an MXFP4 base, adapters in place; replays
    follow the rows, ranks and activations that they find."""
    M, N, K, r = 24, 512, 256, 16
    c = adapter_case(M, N, K, r, 6, rows="random", seed=2)
    X, R, gain = bf(1, 1.0, M, K), bf(2, 1.0, M, K), torch.ones(K, device=DEV)
    W = mx.lq_mx_quantize(bf(3, K**-0.5, N, K), "fp4")

    def step():
        H, y, q = block.lq_rmsnorm_fwd(X, gain, 1e-5, R=R, format="fp8")
        Y = mx.lq_mx_lora_fwd(q, W)
        block.lq_adapters_fwd(y, pool(c), c["rows"], Y, out=Y)
        return H, y, q.codes, Y

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for k in range(4):
        X.copy_(bf(10 + k, 1.0 + k, M, K))
        c["rows"].copy_(torch.from_numpy(np.random.default_rng(k).integers(-1, 7, M).astype(np.int32)))
        c["ranks"].copy_(torch.tensor([1 + k, 16, 0, 16, 7, 16 - k], dtype=torch.int32))
        c["A"].nan_to_num_(0.0)
        c["B"].nan_to_num_(0.0)
        g.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in out]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k
        plain = mx.lq_mx_lora_fwd(block.lq_rmsnorm_fwd(X, gain, 1e-5, R=R, format="fp8")[2], W)
        bare = (c["rows"] < 0) | (c["rows"] >= 6) | (c["rows"] == 2)
        assert torch.equal(got[3][bare], plain[bare]) and not torch.equal(got[3][~bare], plain[~bare])


@pytest.mark.parametrize("M", [3, 20, 500])
def test_captured_calls_equal_eager_ones(M):
    """Every call on its own in one graph, replayed with other work between."""
    N, K, V, r = 192, 256, 3000, 12
    c = adapter_case(M, N, K, r, 4, rows="random", seed=M)
    gain, H = torch.ones(K, device=DEV), bf(1, 1.0, M, K)
    W, t = bf(2, 0.1, V, K), torch.randint(-1, V, (M, 3), device=DEV, dtype=torch.int32)
    p = torch.rand((M, 3), device=DEV)

    def calls():
        out = [*block.lq_rmsnorm_fwd(H, gain, R=c["X"], need_y=True)[:2], *block.lq_rmsnorm_bwd(c["X"], H, gain, dH=c["dX"]),
               block.lq_adapters_fwd(c["X"], pool(c), c["rows"], c["Y"]),
               *block.lq_adapters_bwd(c["dY"], c["X"], pool(c), c["rows"], c["dX"]), *block.lq_head_loss(H, W, t, p)]
        return out

    want = calls()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = calls()
    for k in range(3):
        for x in out:
            x.fill_(7.0)
        g.replay()
        calls()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(out, want)):
            assert torch.equal(a.nan_to_num(9.0), b.nan_to_num(9.0)), (k, i)


def test_calls_on_two_streams():
    """Calls that overlap on two streams, each on data of its own."""
    cs = [adapter_case(200, 512, 512, 16, 4, seed=s) for s in range(2)]
    W = bf(9, 0.1, 2000, 512)
    t = torch.randint(0, 2000, (200,), device=DEV, dtype=torch.int32)

    def work(c):
        Y = block.lq_adapters_fwd(c["X"], pool(c), c["rows"], c["Y"])
        out = [Y, *block.lq_adapters_bwd(c["dY"], c["X"], pool(c), c["rows"], c["dX"]), *block.lq_head_loss(Y, W, t)]
        return out + [*block.lq_rmsnorm_bwd(c["dY"], c["Y"], torch.ones(512, device=DEV))]

    want = [work(c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(3):
        got = []
        for c, s in zip(cs, streams):
            with torch.cuda.stream(s):
                got.append(work(c))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_refusals_leave_outputs_alone():
    c = adapter_case(20, 64, 64, 4, 2)
    Y = c["Y"].clone()
    with pytest.raises(lq.LqError):
        block.lq_adapters_fwd(c["X"], pool(c), c["rows"], Y, out=Y, ws=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        block.lq_adapters_fwd(c["X"], pool(c), c["rows"].long(), Y, out=Y)
    with pytest.raises(ValueError):
        block.lq_adapters_fwd(c["X"].t().contiguous().t(), pool(c), c["rows"], Y, out=Y)
    with pytest.raises(ValueError):
        block.lq_adapters_bwd(c["dY"], c["X"], pool(c), c["rows"], c["dX"], accumulate=True)
    with pytest.raises(ValueError):
        block.lq_rmsnorm_fwd(Y, torch.ones(32, device=DEV))
    with pytest.raises(ValueError):
        block.lq_rmsnorm_fwd(Y, torch.ones(64, device=DEV), need_y=False)
    with pytest.raises(lq.LqError):
        block.lq_rmsnorm_fwd(Y, torch.ones(64, device=DEV), float("nan"))
    with pytest.raises(ValueError):
        block.lq_head_loss(Y, c["X"], torch.zeros(20, device=DEV))
    with pytest.raises(lq.LqError):
        block.lq_head_loss(Y[:, :32].contiguous(), c["X"][:, :32].contiguous(), torch.zeros(20, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert torch.equal(Y, c["Y"])
