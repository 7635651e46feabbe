"""Forward of the MXFP4 layer against float64: every input kind, tile variant,
tail and rank form, with bounds derived in mx_helpers."""
import numpy as np
import pytest
import torch

from qlora_parameter_efficient_amd import mx
from tests.gpu_helpers import DEV, announce
from tests.mx_helpers import assert_within, make, ref_forward, values
from tests.mx_helpers import cancelling, expand_bound, gamma

pytestmark = pytest.mark.gpu


def check(M, N, K, r, fmt, seed=0):
    """fmt: "fp8", "fp4" or "bf16" (the activations)."""
    announce(f"mx fwd {fmt} M={M} N={N} K={K} r={r}")
    bf = fmt == "bf16"
    X, W, A, B, _, s = make(M, N, K, r, fmt, seed, bf16_x=bf)
    T = torch.full((M, r), 7.0, dtype=torch.float32, device=DEV) if r else None
    # rows past M and the elements around Y must stay
    out = torch.full((M + 2, N), 5.0, dtype=torch.bfloat16, device=DEV)
    Y = mx.lq_mx_lora_fwd(X, W, A if r else None, B if r else None, s, T_out=T, Y=out[1:M + 1])
    torch.cuda.synchronize()
    x = X.double() if bf else values(X)
    Yr, bY, Tr, bT = ref_forward(x, values(W), A, B, s, scaled=not bf)
    assert_within(Y, Yr, bY, "Y")
    if r:
        assert_within(T, Tr, bT, "T")
    assert (out[0] == 5.0).all() and (out[M + 1] == 5.0).all()


@pytest.mark.parametrize("M", [1, 2, 5, 16, 17, 31, 33, 64])
@pytest.mark.parametrize("N,K,r", [(64, 64, 1), (128, 192, 8), (320, 4096, 16), (64, 11008, 64),
                                   (192, 128, 33), (256, 1088, 0)])
def test_few_bf16_rows(M, N, K, r):
    check(M, N, K, r, "bf16")


@pytest.mark.parametrize("M,N,K,r", [(1, 64, 128, 1), (1, 192, 4096, 16), (2, 64, 8192, 8), (3, 320, 4096, 5),
                                     (4, 128, 4096, 16), (1, 64, 16384, 4), (1, 8256, 4736, 13),
                                     (4, 64, 640, 2), (5, 64, 2048, 16), (1, 128, 4096, 17)])
def test_single_tokens(M, N, K, r):
    """T formed in the stream kernel (M <= 4, r <= 16, r K <= 65536), and just past that."""
    check(M, N, K, r, "bf16")


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("M,N,K,r", [
    (1, 64, 64, 1), (1, 4096, 4096, 16), (7, 128, 320, 8), (33, 64, 256, 0), (64, 192, 576, 11),
    (100, 256, 4160, 24), (70, 512, 8192, 64), (520, 11008, 128, 16), (1030, 11008, 64, 7),
    (65, 320, 128, 64), (100, 256, 512, 32), (129, 448, 1024, 16), (300, 1088, 832, 5),
    (777, 512, 1920, 24), (257, 4096, 448, 16),
])
def test_small_and_ragged(M, N, K, r, fmt):
    check(M, N, K, r, fmt)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("M,N,K,r", [
    (2048, 3200, 512, 16),    # 256 x 128 tiles
    (520, 11008, 320, 9),     # the same with a tail
    (2049, 4160, 320, 11),    # 256 x 256 with a tail and ragged edges
    (4000, 4096, 256, 64),    # 256 x 256 tiles
    (3585, 4160, 576, 9),     # the same with a tail and ragged edges
    (1500, 2048, 384, 16),    # 128 x 128 tiles
    (1500, 2048, 1024, 16),   # the same, scales of several steps per load
    (4000, 4096, 512, 20),    # 256 x 256, the same
    (2048, 3200, 2560, 16),   # 256 x 128, the same
    (100, 512, 4608, 8),      # split K that starts inside such a load
])
def test_tile_variants(M, N, K, r, fmt):
    check(M, N, K, r, fmt)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_one_hot_rows_give_the_weight_columns(fmt):
    """X = rows of the identity: Y is the weight's columns, exactly (each value
    is representable in bf16)."""
    K, N = 320, 192
    _, W, *_ = make(1, N, K, 1, "fp8")
    X = mx.lq_mx_quantize(torch.eye(K, dtype=torch.bfloat16, device=DEV), fmt)
    Y = mx.lq_mx_lora_fwd(X, W)
    assert torch.equal(Y.double(), values(W).t().contiguous())


def test_non_finite_blocks_stay_in_their_rows():
    """A NaN block of X makes its row NaN, one of W its column; nothing else,
    also where the block is the last one before a tail."""
    for fmt in ("fp8", "fp4"):
        for M, N, K in ((70, 128, 320), (40, 128, 256)):
            announce(f"mx fwd NaN {fmt} {M} {N} {K}")
            X, W, A, B, _, s = make(M, N, K, 8, fmt)
            X.scales[3, K // 32 - 1] = 255
            W.scales[5, 0] = 255
            T = torch.empty((M, 8), dtype=torch.float32, device=DEV)
            Y = mx.lq_mx_lora_fwd(X, W, A, B, s, T_out=T)
            nan = torch.isnan(Y).cpu().numpy()
            want = np.zeros((M, N), bool)
            want[3] = True
            want[:, 5] = True
            assert np.array_equal(nan, want)
            assert torch.isnan(T[3]).all() and not torch.isnan(torch.cat([T[:3], T[4:]])).any()


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("M,N,K", [(70, 128, 1024), (40, 512, 4608), (2000, 3200, 512)])
def test_non_finite_blocks_under_wide_scale_loads(M, N, K, fmt):
    """The same where one load brings the scales of several steps (K % 512 == 0),
    whole and split: first, last and middle blocks."""
    announce(f"mx fwd NaN wide {fmt} {M} {N} {K}")
    X, W, A, B, _, s = make(M, N, K, 8, fmt)
    kb = K // 32
    X.scales[3, kb - 1], X.scales[17, 0], X.scales[M - 1, kb // 2 + 1] = 255, 255, 255
    W.scales[5, 7], W.scales[N - 1, kb - 2] = 255, 255
    Y = mx.lq_mx_lora_fwd(X, W, A, B, s)
    nan = torch.isnan(Y).cpu().numpy()
    want = np.zeros((M, N), bool)
    want[[3, 17, M - 1]] = True
    want[:, [5, N - 1]] = True
    assert np.array_equal(nan, want)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("M,N,K,r", [(1, 64, 128, 3), (3, 128, 4096, 16), (3, 64, 192, 8), (13, 320, 4096, 64),
                                     (13, 64, 11008, 33), (17, 128, 512, 16), (64, 192, 320, 5)])
def test_non_finite_values_of_the_adapter_and_the_rows(M, N, K, r, fmt):
    """An infinity or NaN in X makes its row of Y and T non-finite, one in W or B a
    column of Y, one in A everything (its column of T): and nothing else."""
    X, W, A, B, _, s = make(M, N, K, r, fmt, bf16_x=fmt == "bf16")
    inf, nan = float("inf"), float("nan")

    def run(what, X=X, W=W, A=A, B=B):
        announce(f"mx fwd non-finite {what} {fmt} M={M} N={N} K={K} r={r}")
        T = torch.empty((M, r), device=DEV)
        Y = mx.lq_mx_lora_fwd(X, W, A, B, s, T_out=T)
        torch.cuda.synchronize()
        return ~torch.isfinite(Y), ~torch.isfinite(T)

    none_y = torch.zeros((M, N), dtype=torch.bool, device=DEV)
    none_t = torch.zeros((M, r), dtype=torch.bool, device=DEV)

    def cut(t, at, v):
        t = t.clone()
        t[at] = v
        return t

    for m in sorted({0, M // 2, M - 1}):
        for v in (nan, inf, -inf) if fmt == "bf16" else (nan,):
            if fmt == "bf16":
                x = cut(X, (m, K - 1), v)
            else:
                x = mx.MxTensor(X.codes, cut(X.scales, (m, K // 32 - 1), 255), M, K, fmt)
            y, t = none_y.clone(), none_t.clone()
            y[m], t[m] = True, True
            got = run(f"X {v} in row {m}", X=x)
            assert torch.equal(got[0], y) and torch.equal(got[1], t)
    for n in (0, N - 1):
        y = none_y.clone()
        y[:, n] = True
        got = run(f"W NaN in row {n}", W=mx.MxTensor(W.codes, cut(W.scales, (n, K // 64), 255), N, K, "fp4"))
        assert torch.equal(got[0], y) and torch.equal(got[1], none_t)
        for v in (nan, inf):
            got = run(f"B {v} in row {n}", B=cut(B, (n, r - 1), v))
            assert torch.equal(got[0], y) and torch.equal(got[1], none_t)
    for v in (nan, inf):
        t = none_t.clone()
        t[:, r - 1] = True
        got = run(f"A {v}", A=cut(A, (r - 1, K - 1), v))
        assert got[0].all() and torch.equal(got[1], t)


@pytest.mark.parametrize("fmt", ["fp8", "fp4", "bf16"])
@pytest.mark.parametrize("M,N,K,r", [(3, 128, 256, 6), (40, 192, 512, 16), (100, 512, 4608, 8), (520, 11008, 128, 16),
                                     (2048, 3200, 512, 32), (4000, 4096, 256, 64)])
def test_adapter_term_with_cancelling_ranks(M, N, K, r, fmt):
    """On a base of zeros Y is s T B^T alone, and its ranks cancel: T enters with
    more than one bf16's bits in every tile variant."""
    if fmt == "bf16" and M > mx.LQ_MX_ROWS_BF16:
        M = 64
    announce(f"mx fwd cancelling ranks {fmt} M={M} N={N} K={K} r={r}")
    X, *_ = make(M, 64, K, r, fmt, bf16_x=fmt == "bf16")
    A, B = cancelling(r, K, N, 3)
    s = 1.5
    W = mx.lq_mx_quantize(torch.zeros(N, K, device=DEV), "fp4")
    T = torch.empty((M, r), device=DEV)
    Y = mx.lq_mx_lora_fwd(X, W, A, B, s, T_out=T)
    torch.cuda.synchronize()
    x = X.double() if fmt == "bf16" else values(X)
    Tr = x @ A.double().t()
    bT = gamma(K) * (x.abs() @ A.double().abs().t()) + 1e-37
    assert_within(T, Tr, bT, "T")
    Yr = s * (T.double() @ B.double().t())  # of T as it was formed
    assert_within(Y, Yr, expand_bound(Yr, T.double(), 0.0, B.double(), s), "Y")


def moved(q, at):
    """q with its scales ``at`` bytes past a 16-byte boundary."""
    flat = torch.full((q.scales.numel() + 32,), 0x5A, dtype=torch.uint8, device=DEV)
    assert flat.data_ptr() % 16 == 0
    s = flat[at:at + q.scales.numel()].view(q.scales.shape)
    s.copy_(q.scales)
    return mx.MxTensor(q.codes, s, q.rows, q.cols, q.format)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("M,N,K,r,ax,aw", [
    (70, 128, 512, 8, 2, 0), (70, 128, 512, 8, 0, 4), (130, 192, 1024, 16, 8, 2),
    (2000, 3200, 512, 16, 4, 8), (4000, 4096, 256, 5, 2, 6), (100, 512, 4608, 8, 14, 0),
    (100, 256, 4160, 24, 2, 10), (33, 64, 128, 33, 6, 0), (4100, 128, 384, 64, 2, 4)])
def test_scales_at_even_addresses(M, N, K, r, ax, aw, fmt):
    """Scales of X and W off 16 bytes, words or neither; the values beside them
    are not read into the result."""
    announce(f"mx fwd scales at +{ax} / +{aw} {fmt} M={M} N={N} K={K} r={r}")
    X, W, A, B, _, s = make(M, N, K, r, fmt)
    x, w = values(X), values(W)
    T = torch.empty((M, r), device=DEV)
    Y = mx.lq_mx_lora_fwd(moved(X, ax), moved(W, aw), A, B, s, T_out=T)
    torch.cuda.synchronize()
    Yr, bY, Tr, bT = ref_forward(x, w, A, B, s, scaled=True)
    assert_within(Y, Yr, bY, "Y")
    assert_within(T, Tr, bT, "T")


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("K", [64, 128, 192, 256, 512, 832])
def test_rows_of_a_larger_tensor(K, fmt):
    """A micro-batch cut from a checkpoint, and a slice of the layer's outputs:
    consecutive rows of an MX tensor, each wherever its scales begin."""
    M, N, r = 41, 192, 8
    X, W, A, B, _, s = make(M + 7, N + 64, K, r, fmt)
    x, w = values(X), values(W)
    for m0, n0 in ((1, 64), (3, 0), (7, 1), (2, 33)):
        announce(f"mx fwd rows {m0} / {n0} {fmt} K={K}")
        cut = lambda q, a, n: mx.MxTensor(q.codes[a:a + n], q.scales[a:a + n], n, K, q.format)  # noqa: E731
        b = B[n0:n0 + N].contiguous()
        Y = mx.lq_mx_lora_fwd(cut(X, m0, M), cut(W, n0, N), A, b, s)
        torch.cuda.synchronize()
        Yr, bY, _, _ = ref_forward(x[m0:m0 + M], w[n0:n0 + N], A, b, s, scaled=True)
        assert_within(Y, Yr, bY, "Y")


def test_extreme_scales():
    """Scale bytes far from 127 on both sides: products from 2^-200 up to 2^100."""
    M, N, K = 96, 128, 256
    X, W, *_ = make(M, N, K, 1, "fp8")
    X.scales[:48] = 200
    X.scales[48:] = 20
    W.scales[:64] = 150
    W.scales[64:] = 60
    announce("mx fwd extreme scales")
    Y = mx.lq_mx_lora_fwd(X, W).double()
    x, w = values(X), values(W)
    ref = x @ w.t()
    bound = 2.0**-8 * ref.abs() + (2.0**-13 + 2.0**-16) * (x.abs() @ w.abs().t()) + 2.0**-133
    assert ((Y - ref).abs() <= bound).all()


def test_widest_layers():
    """K = 65536 and N = 65536."""
    check(3, 64, 65536, 16, "bf16")
    check(20, 128, 65536, 4, "fp8")
    check(2, 65536, 128, 16, "bf16")
    check(130, 65536, 192, 7, "fp4")


@pytest.mark.parametrize("fmt", ["fp8", "fp4", "bf16"])
@pytest.mark.parametrize("M,N,K,r", [(2, 128, 256, 16), (40, 192, 512, 8), (64, 128, 192, 5), (33, 64, 128, 64)])
def test_t_out_at_any_word(M, N, K, r, fmt):
    """T_out 4 bytes past a 16-byte boundary: the same T and Y, nothing beside it."""
    announce(f"mx fwd T_out at +4 {fmt} M={M} N={N} K={K} r={r}")
    X, W, A, B, _, s = make(M, N, K, r, fmt, bf16_x=fmt == "bf16")
    T = torch.empty((M, r), device=DEV)
    Y = mx.lq_mx_lora_fwd(X, W, A, B, s, T_out=T)
    flat = torch.full((M * r + 8,), 3.0, device=DEV)
    Z = mx.lq_mx_lora_fwd(X, W, A, B, s, T_out=flat[1:1 + M * r].view(M, r))
    torch.cuda.synchronize()
    assert torch.equal(Y, Z) and torch.equal(flat[1:1 + M * r].view(M, r), T)
    assert flat[0] == 3.0 and (flat[1 + M * r:] == 3.0).all()


def test_no_rows():
    _, W, A, B, _, s = make(1, 64, 64, 4, "fp8")
    X = mx.MxTensor(torch.empty((0, 64), dtype=torch.uint8, device=DEV),
                    torch.empty((0, 2), dtype=torch.uint8, device=DEV), 0, 64, "fp8")
    assert mx.lq_mx_lora_fwd(X, W, A, B, s).shape == (0, 64)
    assert mx.lq_mx_lora_fwd(torch.empty((0, 64), dtype=torch.bfloat16, device=DEV), W, A, B, s).shape == (0, 64)


def test_binding_refuses_wrong_operands():
    X, W, A, B, _, s = make(8, 128, 128, 4, "fp8")
    bad = [dict(A=A.float()), dict(A=A[:, :64].contiguous()), dict(B=B[:64]), dict(B=None),
           dict(A=A.t()), dict(X=torch.zeros(8, 64, dtype=torch.bfloat16, device=DEV)),
           dict(X=torch.zeros(8, 128, device=DEV)), dict(T_out=torch.empty(8, 5, device=DEV)),
           dict(Y=torch.empty(8, 64, dtype=torch.bfloat16, device=DEV)), dict(A=A.cpu()),
           dict(W0=mx.MxTensor(W.codes[:64], W.scales, 128, 128, "fp4"))]
    for b in bad:
        kw = dict(X=X, W0=W, A=A, B=B, scale=s)
        kw.update(b)
        with pytest.raises(ValueError):
            mx.lq_mx_lora_fwd(**kw)
    with pytest.raises(mx.LqError):
        mx.lq_mx_lora_fwd(torch.zeros(65, 128, dtype=torch.bfloat16, device=DEV), W, A, B, s)
    with pytest.raises(mx.LqError):  # an 8-bit base is not a weight format
        mx.lq_mx_lora_fwd(X, mx.lq_mx_quantize(torch.zeros(128, 128, device=DEV), "fp8"), A, B, s)


@pytest.mark.parametrize("M,r", [(1, 16), (4, 16), (13, 64), (64, 8), (3, 0)])
def test_decode_captured_and_replayed(M, r):
    """The single-token forward in a graph: every replay on new inputs equals
    the eager call bit for bit, with eager work between the replays."""
    announce(f"mx decode graph M={M} r={r}")
    X, W, A, B, _, s = make(M, 512, 1024, r, "fp8", bf16_x=True)
    call = lambda: mx.lq_mx_lora_fwd(X, W, A if r else None, B if r else None, s)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for k in range(4):
        X.copy_(torch.randn(X.shape, generator=torch.Generator().manual_seed(k)))
        graph.replay()
        torch.cuda.synchronize()
        eager = call()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("N,K", [(64, 11008), (11008, 64)])
def test_offsets_past_31_bits(N, K, fmt):
    """M K (or M N) just below 2^31 elements, 4 GB of bf16: rows at both ends
    and around 2^31 bytes."""
    M, r = 195000, 4
    announce(f"mx long {fmt} N={N} K={K}")
    g = torch.Generator(device=DEV).manual_seed(0)
    X = torch.randn(M, K, generator=g, device=DEV, dtype=torch.bfloat16)
    Xq = mx.lq_mx_quantize(X, fmt)
    del X
    _, W, A, B, _, s = make(1, N, K, r, fmt)
    T = torch.empty(M, r, device=DEV)
    Y = mx.lq_mx_lora_fwd(Xq, W, A, B, s, T_out=T)
    back = mx.lq_mx_dequantize(Xq)
    torch.cuda.synchronize()
    w = values(W)
    half = 2**31 // (2 * max(N, K))  # the row at 2^31 bytes of bf16
    for m0 in (0, half - 50, 2 * half - 50, M - 100):
        m0 = min(m0, M - 100)
        rows = slice(m0, m0 + 100)
        x = values(mx.MxTensor(Xq.codes[rows], Xq.scales[rows], 100, K, fmt))
        assert torch.equal(back[rows].double(), x)
        Yr, bY, Tr, bT = ref_forward(x, w, A, B, s, scaled=True)
        assert_within(T[rows], Tr, bT, "T")
        assert_within(Y[rows], Yr, bY, "Y")
