"""Backward from MX checkpoints against float64: the MXFP4 layer and the dense
and NF4 layers, with bounds derived in mx_helpers; a whole step; gradients
against differences; streams, graphs and shared leaves."""
import pytest
import torch

from qlora_parameter_efficient_amd import lq, mx
from tests.gpu_helpers import DEV, announce
from tests.mx_helpers import assert_within, gamma, make, ref_backward, ref_forward, values
from tests.mx_helpers import cancelling, expand_bound

pytestmark = pytest.mark.gpu

SHAPES = [(1, 64, 64, 1), (3, 128, 192, 5), (64, 256, 320, 8), (65, 320, 128, 64), (130, 64, 1088, 16),
          (300, 1088, 832, 33), (777, 512, 1920, 24), (1000, 2048, 2048, 16), (2048, 4096, 512, 11),
          (1001, 64, 11008, 8), (50, 512, 256, 28), (40, 832, 1152, 20), (4100, 320, 384, 48),
          (4100, 192, 192, 11), (4101, 256, 256, 16), (4130, 512, 512, 36)]


def out_buffers(M, N, K, r):
    """dX, dA, dB as views with guard rows on both sides."""
    X = torch.full((M + 2, K), 5.0, dtype=torch.bfloat16, device=DEV)
    a = torch.full((r + 2, K), 5.0, device=DEV)
    b = torch.full((N + 2, r), 5.0, device=DEV)
    return (X, a, b), (X[1:-1], a[1:-1], b[1:-1])


def compare(got, refs, names=("dX", "dA", "dB")):
    for g, (w, b), n in zip(got, refs, names):
        assert_within(g, w, b, n)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("saved", [True, False])
@pytest.mark.parametrize("M,N,K,r", SHAPES)
def test_mx_layer(M, N, K, r, fmt, saved):
    announce(f"mx bwd {fmt} M={M} N={N} K={K} r={r} saved={saved}")
    X, W, A, B, dY, s = make(M, N, K, r, fmt)
    x = values(X)
    T = (x @ A.double().t()).float() if saved else None
    whole, (dX, dA, dB) = out_buffers(M, N, K, r)
    got = mx.lq_mx_lora_bwd(dY, X, W, A, B, s, T_saved=T, dX=dX, dA=dA, dB=dB)
    torch.cuda.synchronize()
    Tr = T.double() if saved else x @ A.double().t()
    refs = ref_backward(dY, x, Tr, values(W), A, B, s)
    if not saved:  # T's own error
        _, _, _, bT = ref_forward(x, values(W), A, B, s, False)
        w, b = refs[2]
        refs = refs[:2] + ((w, b + abs(s) * (dY.double().abs().t() @ bT)),)
    compare(got, refs)
    for t in whole:
        assert (t[0] == 5.0).all() and (t[-1] == 5.0).all()


@pytest.mark.parametrize("base", ["dense", "nf4", "nf4_single"])
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("M,N,K,r", SHAPES)
def test_checkpoint_of_dense_and_nf4_layers(M, N, K, r, fmt, base):
    announce(f"ckpt bwd {base} {fmt} M={M} N={N} K={K} r={r}")
    X, _, A, B, dY, s = make(M, N, K, r, fmt)
    g = torch.Generator().manual_seed(9)
    Wd = (torch.randn((N, K), generator=g) * 0.02).to(torch.bfloat16).to(DEV)
    W = Wd
    if base != "dense":
        W = lq.lq_nf4_quantize(Wd, double_quant=base == "nf4")
        Wd = lq.lq_nf4_dequantize(W).view(N, K)
    x = values(X)
    T = (x @ A.double().t()).float()
    got = mx.lq_lora_bwd_ckpt(dY, X, W, A, B, s, T_saved=T)
    torch.cuda.synchronize()
    compare(got, ref_backward(dY, x, T.double(), Wd.double(), A, B, s))


@pytest.mark.parametrize("M,N,K,r", [(2, 3840, 384, 11), (1, 1024, 64, 1), (66, 5056, 320, 16),
                                     (16, 4096, 512, 8), (300, 1024, 4992, 5), (1001, 1088, 11072, 8),
                                     (2050, 1024, 4160, 16), (130, 1024, 512, 7), (512, 1024, 1024, 64)])
def test_dense_base_of_many_shapes(M, N, K, r):
    """dX of a dense base, alone and with the gradients: split reductions, every
    tile height, columns that end inside a tile, ranks that are no multiple of 4."""
    announce(f"ckpt dense M={M} N={N} K={K} r={r}")
    X, _, A, B, dY, s = make(M, N, K, r, "fp8")
    W = (torch.randn((N, K), generator=torch.Generator().manual_seed(9)) * 0.02)
    W = W.to(torch.bfloat16).to(DEV)
    x = values(X)
    T = (x @ A.double().t()).float()
    refs = ref_backward(dY, x, T.double(), W.double(), A, B, s)
    whole, (dX, dA, dB) = out_buffers(M, N, K, r)
    got = mx.lq_lora_bwd_ckpt(dY, X, W, A, B, s, T_saved=T, dX=dX, dA=dA, dB=dB)
    alone, _, _ = mx.lq_lora_bwd_ckpt(dY, None, W, A, B, s, need_grads=False)
    torch.cuda.synchronize()
    compare(got, refs)
    assert torch.equal(alone, dX)
    for t in whole:
        assert (t[0] == 5.0).all() and (t[-1] == 5.0).all()


@pytest.mark.parametrize("base", ["mxfp4", "dense"])
@pytest.mark.parametrize("M,N,K", [(70, 1024, 320), (300, 1088, 4992)])
def test_non_finite_rows_stay_in_their_rows(M, N, K, base):
    """A NaN in row m of dY makes row m of dX NaN, one in a weight its columns
    (a block of 32, or one of a dense base); nothing else."""
    announce(f"bwd NaN {base} {M} {N} {K}")
    X, W, A, B, dY, s = make(M, N, K, 8, "fp8")
    dY[5, 3] = float("nan")
    dY[M - 1, N - 1] = float("inf")
    want = torch.zeros((M, K), dtype=torch.bool, device=DEV)
    if base == "mxfp4":
        W.scales[N - 2, K // 32 - 1] = 255
        want[:, K - 32:] = True
        dX, _, _ = mx.lq_mx_lora_bwd(dY, None, W, A, B, s, need_grads=False)
    else:
        Wd = (torch.randn((N, K), generator=torch.Generator().manual_seed(9)) * 0.02)
        Wd = Wd.to(torch.bfloat16).to(DEV)
        Wd[N - 2, K - 1] = float("nan")
        want[:, K - 1] = True
        dX, _, _ = mx.lq_lora_bwd_ckpt(dY, None, Wd, A, B, s, need_grads=False)
    torch.cuda.synchronize()
    assert not torch.isfinite(dX[M - 1]).any()  # infinities of both signs, or their sums
    want[5] = True
    assert torch.equal(torch.isnan(dX[:-1]), want[:-1])


@pytest.mark.parametrize("base", ["mxfp4", "dense", "nf4"])
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("M,N,K,r", [(1, 64, 64, 4), (40, 512, 512, 8), (200, 256, 320, 12), (333, 192, 512, 40),
                                     (777, 512, 256, 64)])
def test_non_finite_gradients(M, N, K, r, fmt, base):
    """An infinity or NaN in dY, X, T or B makes the sums of dA and dB that it
    enters non-finite, and no other: in the first row, the last one before a
    range's end, and the last."""
    X, W, A, B, dY, s = make(M, N, K, r, fmt)
    w, fn = W, mx.lq_mx_lora_bwd
    if base != "mxfp4":
        fn = mx.lq_lora_bwd_ckpt
        w = (torch.randn((N, K), generator=torch.Generator().manual_seed(9)) * 0.02).to(torch.bfloat16).to(DEV)
        w = w if base == "dense" else lq.lq_nf4_quantize(w)
    T = (values(X) @ A.double().t()).float()
    inf, nan = float("inf"), float("nan")

    def run(what, need_dx=True, **kw):
        announce(f"bwd non-finite {what} {base} {fmt} M={M} N={N} K={K} r={r} dx={need_dx}")
        a = dict(dY=dY, Xq=X, B=B, T_saved=T)
        a.update(kw)
        _, dA, dB = fn(a["dY"], a["Xq"], w, A, a["B"], s, T_saved=a["T_saved"], need_dx=need_dx)
        torch.cuda.synchronize()
        return ~torch.isfinite(dA), ~torch.isfinite(dB)

    none_a = torch.zeros((r, K), dtype=torch.bool, device=DEV)
    none_b = torch.zeros((N, r), dtype=torch.bool, device=DEV)
    for m in sorted({0, min(63, M - 1), M - 1}):
        for v in (nan, inf, -inf):
            d = dY.clone()
            d[m, N - 2] = v
            for dx in (True, False):
                bad_a, bad_b = run(f"dY {v} in row {m}", dx, dY=d)
                assert bad_a.all()  # U's row m, every rank
                want = none_b.clone()
                want[N - 2] = True
                assert torch.equal(bad_b, want)
            t = T.clone()
            t[m, r - 1] = v
            bad_a, bad_b = run(f"T {v} in row {m}", T_saved=t)
            want = none_b.clone()
            want[:, r - 1] = True
            assert torch.equal(bad_a, none_a) and torch.equal(bad_b, want)
        q = mx.MxTensor(X.codes, X.scales.clone(), M, K, fmt)
        q.scales[m, K // 32 - 1] = 255
        want = none_a.clone()
        want[:, K - 32:] = True
        bad_a, bad_b = run(f"X NaN in row {m}", Xq=q)
        assert torch.equal(bad_a, want) and torch.equal(bad_b, none_b)
        bad_a, bad_b = run(f"X NaN in row {m}, T formed", Xq=q, T_saved=None)
        assert torch.equal(bad_a, want) and bad_b.all()
    for v in (nan, inf):
        b = B.clone()
        b[N - 1, 0] = v
        want = none_a.clone()
        want[0] = True
        for dx in (True, False):
            bad_a, bad_b = run(f"B {v}", dx, B=b)
            assert torch.equal(bad_a, want) and torch.equal(bad_b, none_b)


@pytest.mark.parametrize("base", ["mxfp4", "dense"])
@pytest.mark.parametrize("M,N,K,r", [(100, 1024, 512, 6), (3, 4096, 320, 16), (600, 1024, 11008, 8),
                                     (700, 1024, 4096, 6), (1030, 1024, 8192, 11), (4100, 1024, 4096, 61)])
def test_adapter_term_with_cancelling_ranks(M, N, K, r, base):
    """On a base of zeros dX is s U A alone, and its ranks cancel: U enters with
    more than one bf16's bits in every tile variant (a dense base on shapes that
    take the same kernel).  U's own sum is kept exact: dY is one element a row."""
    announce(f"bwd cancelling ranks {base} M={M} N={N} K={K} r={r}")
    even = r - r % 2
    B, A = cancelling(even, N, K, 5)
    B, A = B.t().contiguous(), A.t().contiguous()  # A cancels over ranks, B nearly equal in pairs
    if r % 2:
        A = torch.cat((A, torch.zeros((1, K), dtype=A.dtype, device=DEV)))
        B = torch.cat((B, torch.zeros((N, 1), dtype=B.dtype, device=DEV)), 1)
    g = torch.Generator().manual_seed(1)
    dY = torch.zeros((M, N))
    dY[torch.arange(M), torch.randint(0, N, (M,), generator=g)] = torch.randn(M, generator=g)
    dY = dY.to(torch.bfloat16).to(DEV)
    s = 1.375
    if base == "mxfp4":
        W = mx.lq_mx_quantize(torch.zeros(N, K, device=DEV), "fp4")
        dX, _, _ = mx.lq_mx_lora_bwd(dY, None, W, A, B.contiguous(), s, need_grads=False)
    else:
        W = torch.zeros((N, K), dtype=torch.bfloat16, device=DEV)
        dX, _, _ = mx.lq_lora_bwd_ckpt(dY, None, W, A, B.contiguous(), s, need_grads=False)
    torch.cuda.synchronize()
    U = dY.double() @ B.double()  # one product a row: exact in float32
    want = s * (U @ A.double())
    assert_within(dX, want, expand_bound(want, U, 0.0, A.double().t(), s), "dX")


def test_parts_and_accumulation():
    M, N, K, r = 200, 256, 320, 12
    X, W, A, B, dY, s = make(M, N, K, r, "fp8")
    Wd = mx.lq_mx_dequantize(W)
    for fn, w in ((mx.lq_mx_lora_bwd, W), (mx.lq_lora_bwd_ckpt, Wd)):
        announce(f"bwd parts {fn.__name__}")
        dX, dA, dB = fn(dY, X, w, A, B, s)
        only, na, nb = fn(dY, None, w, A, B, s, need_grads=False)
        assert na is None and nb is None and torch.equal(only, dX)
        nx, ga, gb = fn(dY, X, w, A, B, s, need_dx=False)
        assert nx is None
        # without dX, U = dY B comes from another kernel: equal up to its sum's rounding
        assert torch.allclose(ga, dA, rtol=0, atol=float(dA.abs().max()) * 1e-5)
        assert torch.equal(gb, dB)
        a0, b0 = torch.randn_like(dA), torch.randn_like(dB)
        a1, b1 = a0.clone(), b0.clone()
        fn(dY, X, w, A, B, s, dA=a1, dB=b1, accumulate=True)
        assert torch.equal(a1, a0 + dA) and torch.equal(b1, b0 + dB)
        # the same call again gives the same bits
        again = fn(dY, X, w, A, B, s)
        assert all(torch.equal(p, q) for p, q in zip(again, (dX, dA, dB)))


def test_no_rows():
    _, W, A, B, _, s = make(1, 128, 64, 4, "fp8")
    X = mx.MxTensor(torch.empty((0, 64), dtype=torch.uint8, device=DEV),
                    torch.empty((0, 2), dtype=torch.uint8, device=DEV), 0, 64, "fp8")
    dY = torch.empty((0, 128), dtype=torch.bfloat16, device=DEV)
    for fn, w in ((mx.lq_mx_lora_bwd, W), (mx.lq_lora_bwd_ckpt, mx.lq_mx_dequantize(W))):
        dX, dA, dB = fn(dY, X, w, A, B, s)
        assert dX.shape == (0, 64) and not dA.any() and not dB.any()
        a, b = torch.ones_like(dA), torch.ones_like(dB)
        fn(dY, X, w, A, B, s, dA=a, dB=b, accumulate=True)
        assert (a == 1).all() and (b == 1).all()


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_training_step_of_no_rows(fmt):
    """The whole recipe on an empty batch: empty outputs, zero gradients."""
    announce(f"mx step of no rows {fmt}")
    _, W, A, B, _, s = make(1, 128, 64, 4, fmt)
    X = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    dY = torch.empty((0, 128), dtype=torch.bfloat16, device=DEV)
    Y, dX, dA, dB = step(X, W, A, B, dY, s, fmt)
    assert Y.shape == (0, 128) and dX.shape == (0, 64) and not dA.any() and not dB.any()
    q = mx.lq_mx_quantize(X, fmt)
    assert mx.lq_mx_dequantize(q, torch.float32).shape == (0, 64)
    for x in (torch.empty((4, 0), device=DEV), torch.empty((0, 0), device=DEV)):
        with pytest.raises(mx.LqError):
            mx.lq_mx_quantize(x, fmt)


def test_gradients_against_differences():
    """L = sum(Y G): dA and dB of the step against float64 central differences
    of the formula (L is linear in A and in B alone), and dX against its own."""
    M, N, K, r = 48, 64, 128, 4
    X, W, A, B, G, s = make(M, N, K, r, "fp8")
    x, w = values(X), values(W)

    def loss(x, A, B):
        return ((x @ w.t() + s * (x @ A.t()) @ B.t()) * G.double()).sum()

    dX, dA, dB = mx.lq_mx_lora_bwd(G, X, W, A, B, s)
    (_, bX), (_, bA), (_, bB) = ref_backward(G, x, x @ A.double().t(), w, A, B, s)
    g = torch.Generator().manual_seed(2)
    for _ in range(6):
        for t, grad, bound, at in ((A.double(), dA, bA, 1), (B.double(), dB, bB, 2), (x, dX, bX, 0)):
            v = torch.randn(t.shape, generator=g, dtype=torch.float64).to(DEV)
            args = [x, A.double(), B.double()]
            hi, lo = list(args), list(args)
            hi[at], lo[at] = t + 0.5 * v, t - 0.5 * v
            diff = loss(*hi) - loss(*lo)
            slack = (bound * v.abs()).sum() * 1.01 + 1e-9 * diff.abs()
            if at == 2:  # T recomputed in float32
                slack = slack + (abs(s) * v.abs().t() @ (G.double().abs().t() @ (
                    (K / 16 + 32) * 2.0**-23 * (x.abs() @ A.double().abs().t())))).diagonal().sum()
            assert (diff - (grad.double() * v).sum()).abs() <= slack


def step(X, W, A, B, dY, s, fmt):
    q = mx.lq_mx_quantize(X, fmt)
    T = torch.empty((X.shape[0], A.shape[0]), device=DEV)
    Y = mx.lq_mx_lora_fwd(q, W, A, B, s, T_out=T)
    return (Y,) + tuple(mx.lq_mx_lora_bwd(dY, q, W, A, B, s, T_saved=T))


@pytest.mark.parametrize("M,N,K,r", [(5, 128, 256, 8), (333, 512, 832, 16), (1100, 1024, 512, 64)])
def test_training_step_captured_and_replayed(M, N, K, r):
    """Quantise, forward and backward captured into a graph: every replay on
    new inputs equals the eager step bit for bit, with eager work between."""
    announce(f"mx step graph M={M}")
    X, W, A, B, dY, s = make(M, N, K, r, "fp8", bf16_x=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(X, W, A, B, dY, s, "fp8")
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(X, W, A, B, dY, s, "fp8")
    for k in range(4):
        X.copy_(torch.randn(X.shape, generator=torch.Generator().manual_seed(k)))
        dY.copy_(torch.randn(dY.shape, generator=torch.Generator().manual_seed(50 + k)))
        graph.replay()
        torch.cuda.synchronize()
        eager = step(X, W, A, B, dY, s, "fp8")
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(outs, eager))


def test_two_streams_at_once():
    M, N, K, r = 256, 512, 512, 16
    sets = [make(M, N, K, r, "fp8", seed=i, bf16_x=True) for i in range(2)]
    want = [step(*c[:5], c[5], "fp8") for c in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for c, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append(step(*c[:5], c[5], "fp8"))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(g, w))


def test_decode_follows_training():
    """The trained layer served: one bf16 row through the streaming forward is
    within the rounding of the quantised forward of the same row's values."""
    M, N, K, r = 40, 256, 512, 8
    X, W, A, B, _, s = make(M, N, K, r, "fp8")
    xb = mx.lq_mx_dequantize(X)  # exact in bf16
    Y = mx.lq_mx_lora_fwd(X, W, A, B, s)
    Z = mx.lq_mx_lora_fwd(xb, W, A, B, s)
    _, bY, _, _ = ref_forward(values(X), values(W), A, B, s, scaled=True)
    assert ((Y.double() - Z.double()).abs() <= 2 * bY).all()


def test_binding_refuses_wrong_operands():
    X, W, A, B, dY, s = make(8, 128, 192, 4, "fp8")
    T = torch.empty((8, 4), device=DEV)
    bad = [dict(dY=dY.float()), dict(dY=dY[:, :64].contiguous()), dict(A=A[:, :64].contiguous()),
           dict(T_saved=T[:4]), dict(dA=torch.empty(3, 192, device=DEV)), dict(A=None, B=None),
           dict(dX=torch.empty(8, 128, dtype=torch.bfloat16, device=DEV)), dict(accumulate=True),
           dict(need_grads=False, dA=torch.empty(4, 192, device=DEV)),
           dict(Xq=mx.lq_mx_quantize(torch.zeros(9, 192, device=DEV), "fp8"))]
    for fn, w in ((mx.lq_mx_lora_bwd, W), (mx.lq_lora_bwd_ckpt, mx.lq_mx_dequantize(W))):
        for b in bad:
            kw = dict(dY=dY, Xq=X, W0=w, A=A, B=B, scale=s)
            kw.update(b)
            with pytest.raises(ValueError):
                fn(**kw)


@pytest.mark.parametrize("base", ["mxfp4", "dense", "nf4"])
@pytest.mark.parametrize("M,N,K,r", [(40, 512, 512, 8), (64, 4096, 4096, 16), (130, 192, 1088, 11), (777, 2048, 1024, 8),
                                     (2048, 1024, 4096, 16), (4100, 512, 4096, 64), (300, 1024, 512, 64)])
def test_exact_workspaces(M, N, K, r, base):
    """The backwards in workspaces of just the bytes asked for: the bytes behind
    stay, and with what the fastest path uses the result is that of the size for
    any weight, bit for bit; the least size is within the bounds too."""
    announce(f"bwd workspaces {base} M={M} N={N} K={K} r={r}")
    X, W, A, B, dY, s = make(M, N, K, r, "fp8")
    x, w, fn = values(X), W, mx.lq_mx_lora_bwd
    if base == "mxfp4":
        wd = values(W)
    else:
        fn = mx.lq_lora_bwd_ckpt
        w = wd = (torch.randn((N, K), generator=torch.Generator().manual_seed(9)) * 0.02).to(torch.bfloat16).to(DEV)
        if base == "nf4":
            w = lq.lq_nf4_quantize(wd)
            wd = lq.lq_nf4_dequantize(w).view(N, K)
    T = (x @ A.double().t()).float()
    refs = ref_backward(dY, x, T.double(), wd.double(), A, B, s)

    def run(n, **kw):
        ws = torch.full((n + 4096,), 0x77, dtype=torch.uint8, device=DEV)
        out = fn(dY, X if kw.get("need_grads", True) else None, w, A, B, s, T_saved=T, ws=ws[:n], **kw)
        torch.cuda.synchronize()
        assert (ws[n:] == 0x77).all()
        return out

    size, no = mx.lq_mx_workspace_size, mx.LQ_MX_NO_GRADS
    if base == "mxfp4":
        full, least, dx = (size(mx.LQ_MX_OP_BWD + f, M, N, K, r) for f in (0, 0, no))
        default, grads = full, full
    else:
        default = size(mx.LQ_MX_OP_BWD_CKPT, M, N, K, r)
        kind = int(base == "nf4")
        full = mx.lq_lora_bwd_ckpt_workspace(M, kind, N, K, r)
        grads = least = size(mx.LQ_MX_OP_BWD_CKPT_FUSED, M, N, K, r)
        dx = mx.lq_lora_bwd_ckpt_workspace(M, kind, N, K, r, True, False)
        assert mx.lq_lora_bwd_ckpt_workspace(M, kind, N, K, r, False) == least
        compare(run(size(mx.LQ_MX_OP_BWD_CKPT_FUSED + no, M, N, K, r), need_grads=False)[:1], refs[:1])
    whole = run(default)
    compare(whole, refs)
    assert all(torch.equal(p, q) for p, q in zip(run(full), whole))
    compare(run(least), refs)
    compare(run(dx, need_grads=False)[:1], refs[:1])
    compare(run(grads, need_dx=False)[1:], refs[1:])
    with pytest.raises(mx.LqError):
        run(least - 256)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("K", [64, 128, 192, 512])
def test_rows_of_a_larger_tensor(K, fmt):
    """The backward of a micro-batch whose checkpoint and base are rows of larger
    tensors, T recomputed."""
    M, N, r = 45, 128, 8
    X, W, A, B, dY, s = make(M + 5, N + 64, K, r, fmt)
    x, w = values(X), values(W)
    for m0, n0 in ((1, 1), (5, 64)):
        announce(f"mx bwd rows {m0} / {n0} {fmt} K={K}")
        cut = lambda q, a, n: mx.MxTensor(q.codes[a:a + n], q.scales[a:a + n], n, K, q.format)  # noqa: E731
        b, d = B[n0:n0 + N].contiguous(), dY[m0:m0 + M, :N].contiguous()
        got = mx.lq_mx_lora_bwd(d, cut(X, m0, M), cut(W, n0, N), A, b, s)
        torch.cuda.synchronize()
        xs, ws = x[m0:m0 + M], w[n0:n0 + N]
        Tr = xs @ A.double().t()
        refs = ref_backward(d, xs, Tr, ws, A, b, s)
        _, _, _, bT = ref_forward(xs, ws, A, b, s, False)
        refs = refs[:2] + ((refs[2][0], refs[2][1] + abs(s) * (d.double().abs().t() @ bT)),)
        compare(got, refs)


@pytest.mark.parametrize("N,K", [(32, 64), (63, 128), (96, 100)])
def test_layers_off_the_shape_rules_raise(N, K):
    """Also where no tile fits the layer: an error of the call, from both backwards."""
    announce(f"mx bwd refused shape N={N} K={K}")
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    W, X = mx.lq_mx_quantize(bf(N, K), "fp4"), mx.lq_mx_quantize(bf(8, K), "fp8")
    for fn, w in ((mx.lq_mx_lora_bwd, W), (mx.lq_lora_bwd_ckpt, bf(N, K))):
        with pytest.raises(mx.LqError, match="64"):
            fn(bf(8, N), X, w, bf(4, K), bf(N, 4), 1.0)


@pytest.mark.parametrize("N,K", [(64, 11008), (11008, 64)])
def test_offsets_past_31_bits(N, K):
    """M K (or M N) just below 2^31 elements: dX at both ends and around 2^31
    bytes, dA and dB over all rows."""
    M, r, fmt = 195000, 4, "fp8"
    announce(f"mx bwd long N={N} K={K}")
    g = torch.Generator(device=DEV).manual_seed(0)
    Xq = mx.lq_mx_quantize(torch.randn(M, K, generator=g, device=DEV, dtype=torch.bfloat16), fmt)
    dY = torch.randn(M, N, generator=g, device=DEV, dtype=torch.bfloat16)
    _, W, A, B, _, s = make(1, N, K, r, fmt)
    T = torch.randn(M, r, generator=g, device=DEV)
    dX, dA, dB = mx.lq_mx_lora_bwd(dY, Xq, W, A, B, s, T_saved=T)
    torch.cuda.synchronize()
    w = values(W)
    half = 2**31 // (2 * max(N, K))
    for m0 in (0, half - 50, 2 * half - 50, M - 100):
        m0 = min(m0, M - 100)
        rows = slice(m0, m0 + 100)
        x = values(mx.MxTensor(Xq.codes[rows], Xq.scales[rows], 100, K, fmt))
        want, bound = ref_backward(dY[rows], x, T[rows].double(), w, A, B, s)[0]
        assert_within(dX[rows], want, bound, "dX")
    del dX
    wA, bA, wB, bB = 0, 0, 0, 0
    for m0 in range(0, M, 8192):  # the decoded values (tested above): exact in float32
        n = min(8192, M - m0)
        q = mx.MxTensor(Xq.codes[m0:m0 + n], Xq.scales[m0:m0 + n], n, K, fmt)
        x, d, t = mx.lq_mx_dequantize(q, torch.float32).double(), dY[m0:m0 + n].double(), T[m0:m0 + n].double()
        u, eu = d @ B.double(), gamma(N) * (d.abs() @ B.double().abs())
        wA, bA = wA + s * (u.t() @ x), bA + s * ((gamma(M, parts=3) * u.abs() + eu).t() @ x.abs())
        wB, bB = wB + s * (d.t() @ t), bB + s * gamma(M, parts=3) * (d.abs().t() @ t.abs())
    assert_within(dA, wA, bA + 2.0**-23 * wA.abs(), "dA")
    assert_within(dB, wB, bB + 2.0**-23 * wB.abs(), "dB")


@pytest.mark.parametrize("base", ["dense", "nf4"])
def test_checkpoint_backward_captured_and_replayed(base):
    M, N, K, r = 333, 512, 832, 11
    announce(f"ckpt graph {base}")
    X, _, A, B, dY, s = make(M, N, K, r, "fp8", bf16_x=True)
    W = torch.randn(N, K, generator=torch.Generator().manual_seed(7)) * 0.02
    W = W.to(torch.bfloat16).to(DEV)
    W = W if base == "dense" else lq.lq_nf4_quantize(W)

    def step():
        q = mx.lq_mx_quantize(X, "fp8")
        return mx.lq_lora_bwd_ckpt(dY, q, W, A, B, s)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for k in range(4):
        X.copy_(torch.randn(X.shape, generator=torch.Generator().manual_seed(k)))
        dY.copy_(torch.randn(dY.shape, generator=torch.Generator().manual_seed(50 + k)))
        graph.replay()
        torch.cuda.synchronize()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(outs, eager))
