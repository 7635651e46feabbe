"""Timed cases of the operators around an adapted projection (block.py).

Kinds of case:
  norm      lq_rmsnorm_fwd: residual added, root-mean-square norm, the result in
            the input's type and / or as an MXFP8 / MXFP4 tensor
  norm_bwd  lq_rmsnorm_bwd: gradients of the input and of the gain
  adapt     lq_adapters_fwd: low-rank adapters of many requests, each row its
            own, added beside a shared projection's output
  adapt_bwd lq_adapters_bwd: their dX, dA and dB
  head      lq_head_loss: softmax cross entropy of a large-vocabulary head
            against a label (k = 1) or a teacher's top k entries, its log sum of
            exponentials, and the gradient of the head's input

An adapter pool has `slots` places of rank r: A slots x r x K, B slots x N x r,
the rank in use and the scale of each place; columns past the rank in use are
not part of the adapter.  rows[i] is the place of row i, -1 for none.
"""
import math

import torch

own = False

DEV = "cuda"
LEVELS4 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
EPS = 1e-5


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one token of a decode step on its way into a projection: latency
        dict(name="norm 1x4096", kind="norm", M=1, K=4096, dt="bf16", res=True, y=True, fmt=""),
        # 2048 tokens of training: bf16 for the adapters, 8 bits for an MXFP4 base
        dict(name="norm mx 2048x4096", kind="norm", M=2048, K=4096, dt="bf16", res=True, y=True, fmt="fp8"),
        # float32 activations with odd sides, in float32 and in 4 bits
        dict(name="norm f32 fp4 777x4095", kind="norm", M=777, K=4095, dt="f32", res=False, y=True, fmt="fp4"),
        # the gradients of a long batch
        dict(name="norm bwd 8192x4096", kind="norm_bwd", M=8192, K=4096, dt="bf16", dw=True),
        # one request, one token
        dict(name="adapt 1x4096x4096", kind="adapt", M=1, N=4096, K=4096, r=16, slots=8, requests=1),
        # a decode batch, nearly every row its own adapter, into the gate / up projection
        dict(name="adapt 48x11008x4096", kind="adapt", M=48, N=11008, K=4096, r=32, slots=64, requests=48),
        # prompts of 32 requests
        dict(name="adapt 8192x4096x4096", kind="adapt", M=8192, N=4096, K=4096, r=64, slots=16, requests=32),
        # several users' adapters trained at once, short ragged batch of an odd rank
        dict(name="adapt bwd 777x4096x4096", kind="adapt_bwd", M=777, N=4096, K=4096, r=11, slots=6, requests=9),
        # ... the down projection over a long batch
        dict(name="adapt bwd 4096x4096x11008", kind="adapt_bwd", M=4096, N=4096, K=11008, r=32, slots=8, requests=16),
        # the loss of a short ragged batch
        dict(name="head 130x32000x4096", kind="head", M=130, V=32000, K=4096, k=1),
        # a student against its teacher's top 16 of an odd vocabulary
        dict(name="head top16 1001x50257x2048", kind="head", M=1001, V=50257, K=2048, k=16),
        # the loss of a training batch
        dict(name="head 4096x32000x4096", kind="head", M=4096, V=32000, K=4096, k=1),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def wide(lo, hi):  # layer widths: multiples of 64
        return 64 * max(1, log(lo, hi) // 64)

    kind = rng.choice(["norm", "norm", "norm_bwd", "adapt", "adapt", "adapt", "adapt_bwd", "adapt_bwd", "head", "head"])
    if kind in ("norm", "norm_bwd"):
        c = dict(kind=kind, M=log(1, 8192), K=log(32, 11008), dt=rng.choice(["bf16", "bf16", "f32"]))
        if kind == "norm":
            c["res"], c["fmt"] = rng.random() < 0.7, rng.choice(["", "", "fp8", "fp4"])
            c["y"] = c["fmt"] == "" or not c["res"] or rng.random() < 0.5
        else:
            c["dw"] = rng.random() < 0.6
        return c
    if kind == "head":
        c = dict(kind=kind, M=log(1, 4096), V=log(1000, 64000), K=wide(512, 4096), k=rng.choice([1, 1, 1, 4, 16, 50]))
        c["M"] = max(1, min(c["M"], 4096 * 32000 * 4096 // (c["V"] * c["K"])))
        return c
    M = log(1, 8192) if kind == "adapt" else log(16, 4096)
    c = dict(kind=kind, M=M, N=wide(256, 11008), K=wide(256, 11008), r=rng.choice([4, 8, 11, 16, 32, 64]), slots=log(1, 64 if kind == "adapt" else 12))
    c["requests"] = max(1, min(M, log(1, 64)))
    if kind == "adapt_bwd":
        c["r"] = min(c["r"], 32)
    elif c["M"] > 64:
        c["slots"] = min(c["slots"], 1024 // c["r"])
    if c["N"] * c["K"] > 11008 * 4096:
        c["N"], c["K"] = min(c["N"], 4096), min(c["K"], 11008)
    return c


# ------------------------------------------------------------------ inputs

def _normal(g, shape, sigma, dtype):
    return (torch.randn(shape, generator=g, device=DEV) * sigma).to(dtype)


def _activations(g, M, K, dtype=torch.bfloat16):
    """Unit normal tokens with a few strong channels, as layer inputs have."""
    x = torch.randn((M, K), generator=g, device=DEV)
    gain = torch.rand(K, generator=g, device=DEV)
    x *= torch.where(gain > 0.99, 8.0, 0.5 + gain)
    return x.to(dtype)


def _type(case):
    return torch.float32 if case["dt"] == "f32" else torch.bfloat16


def _prepare_norm(st, g, case):
    M, K, dt = case["M"], case["K"], _type(case)
    st["W"] = (1.0 + 0.1 * torch.randn(K, generator=g, device=DEV)).to(dt)
    st["X"] = _activations(g, M, K, dt)
    if case["kind"] == "norm":
        st["R"] = _activations(g, M, K, dt) if case["res"] else None
    else:
        st["dY"] = _normal(g, (M, K), 1.0, dt)
        st["G"] = _normal(g, (M, K), 1.0, dt)
        st["rstd"] = torch.rsqrt(st["X"].float().square().mean(1) + EPS)


def _prepare_adapters(st, g, case):
    M, N, K, r, n = (case[k] for k in ("M", "N", "K", "r", "slots"))
    st["A"] = _normal(g, (n, r, K), 1.0 / math.sqrt(K), torch.bfloat16)
    st["B"] = _normal(g, (n, N, r), 1.0 / math.sqrt(r), torch.bfloat16)
    few = torch.randint(1, r + 1, (n,), generator=g, device=DEV, dtype=torch.int32)
    full = torch.rand(n, generator=g, device=DEV) < 0.5
    st["rank"] = torch.where(full, torch.full_like(few, r), few)
    st["scale"] = 0.5 + torch.rand(n, generator=g, device=DEV)
    q = case["requests"]
    # requests: runs of consecutive rows, one adapter each (one in 16 has none)
    if q < M:
        cuts = torch.sort(torch.randint(1, M, (q - 1,), generator=g, device=DEV)).values
        request = torch.bucketize(torch.arange(M, device=DEV), cuts, right=True)
    else:
        request = torch.arange(M, device=DEV)
    place = torch.randint(0, n, (q,), generator=g, device=DEV, dtype=torch.int32)
    bare = torch.rand(q, generator=g, device=DEV) < 1 / 16
    bare[0] = False
    st["rows"] = torch.where(bare, torch.full_like(place, -1), place)[request].contiguous()
    st["X"] = _activations(g, M, K)
    if case["kind"] == "adapt":
        st["Y"] = _normal(g, (M, N), 1.3, torch.bfloat16)
        return
    st["dY"] = _normal(g, (M, N), 1.0, torch.bfloat16)
    st["dX"] = _normal(g, (M, K), 1.3, torch.bfloat16)
    live, at = _live(st)
    T = torch.zeros((M, r), device=DEV)
    x = st["X"].float()
    for s in range(n):
        T = torch.where((at == s)[:, None], x @ st["A"][s].float().t(), T)
    st["T"] = torch.where(live, T, torch.zeros_like(T))


def _prepare_head(st, g, case):
    M, V, K, k = (case[n] for n in ("M", "V", "K", "k"))
    st["H"] = _activations(g, M, K)
    st["W"] = _normal(g, (V, K), 0.03, torch.bfloat16)
    # padding rows have no target
    used = torch.rand(M, generator=g, device=DEV) < 0.95
    used[0] = True
    if k == 1:
        t = torch.randint(0, V, (M, 1), generator=g, device=DEV, dtype=torch.int32)
        st["p"], st["scale"] = None, 1.0
    else:
        # k different entries of each row, from a random start with a random stride
        start = torch.randint(0, V, (M, 1), generator=g, device=DEV)
        t = ((start + torch.arange(k, device=DEV) * (V // k)) % V).to(torch.int32)
        st["p"] = torch.softmax(2.0 * torch.randn((M, k), generator=g, device=DEV), 1)
        st["scale"] = 0.5
    st["t"] = torch.where(used[:, None], t, torch.full_like(t, -1))
    st["w"] = torch.full((M,), 1.0 / M, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = dict(case)
    if case["kind"] in ("norm", "norm_bwd"):
        _prepare_norm(st, g, case)
    elif case["kind"] == "head":
        _prepare_head(st, g, case)
    else:
        _prepare_adapters(st, g, case)
    return st


# ------------------------------------------- MX quantisation, elementwise

def _restored(x, fmt):
    """float32 values after quantisation to MXFP8 / MXFP4 (blocks of 32 columns with the smallest power of two that
    leaves every element within the format's largest value; elements to nearest, ties to even)."""
    M, K = x.shape
    kp = -(-K // 32) * 32
    b = torch.nn.functional.pad(x, (0, kp - K)).view(M, kp // 32, 32)
    amax = b.abs().amax(-1)
    frac, ex = torch.frexp(amax)
    top, bits, low, mant = (0.875, 9, -6, 3) if fmt == "fp8" else (0.75, 3, 0, 1)
    e = ex - bits + (frac > top).to(ex.dtype)
    e = torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127)
    a = b * torch.ldexp(torch.ones_like(amax), -e)[..., None]
    _, ex = torch.frexp(a.abs())
    step = torch.ldexp(torch.ones_like(a), (ex - 1).clamp(min=low) - mant)
    q = torch.round(a / step) * step
    return (q * torch.ldexp(torch.ones_like(amax), e)[..., None]).flatten(1)[:, :K]


# --------------------------------------------------------------- one pass

def _live(st):
    """(M x r: the rank columns that row i's adapter has, M: its place or -1)"""
    n, r, rows = st["slots"], st["r"], st["rows"]
    at = torch.where((rows >= 0) & (rows < n), rows, torch.full_like(rows, -1))
    have = st["rank"][at.clamp(min=0).long()]
    return (torch.arange(r, device=DEV) < have[:, None]) & (at >= 0)[:, None], at


def _spread(st, v, live, at):
    """v (M x r, each row's own adapter) as M x (slots r), zero outside the row's adapter."""
    n, r = st["slots"], st["r"]
    mine = torch.arange(n, device=DEV) == at[:, None]
    v = torch.where(live, v, torch.zeros_like(v))
    return torch.where(mine[:, :, None], v[:, None, :], torch.zeros((), device=DEV)).reshape(-1, n * r)


def _adapters_plain(st):
    live, at = _live(st)
    n, r, K, N = (st[k] for k in ("slots", "r", "K", "N"))
    x, place = st["X"].float(), at.clamp(min=0).long()
    s = st["scale"][place][:, None]
    if st["M"] <= 64:
        t = (st["A"][place].float() @ x[:, :, None])[:, :, 0]
        t = torch.where(live, t, torch.zeros_like(t))
        d = (st["B"][place].float() @ (t * s)[:, :, None])[:, :, 0]
    else:
        t = (x @ st["A"].view(n * r, K).float().t()).view(-1, n, r)
        t = t.gather(1, place[:, None, None].expand(-1, 1, r))[:, 0]
        d = _spread(st, t * s, live, at) @ st["B"].transpose(1, 2).reshape(n * r, N).float()
    return (st["Y"].float() + d).to(torch.bfloat16)


def _adapters_bwd_plain(st):
    live, at = _live(st)
    n, r, K, N = (st[k] for k in ("slots", "r", "K", "N"))
    place = at.clamp(min=0).long()
    s = st["scale"][place][:, None]
    d, b = st["dY"].float(), st["B"].transpose(1, 2).reshape(n * r, N).float()
    u = (d @ b.t()).view(-1, n, r).gather(1, place[:, None, None].expand(-1, 1, r))[:, 0]
    u = _spread(st, u * s, live, at)
    t = _spread(st, st["T"] * s, live, at)
    dX = (st["dX"].float() + u @ st["A"].view(n * r, K).float()).to(torch.bfloat16)
    dA = (u.t() @ st["X"].float()).view(n, r, K)
    dB = (t.t() @ d).view(n, r, N).transpose(1, 2).contiguous()
    return dX, dA, dB


def _norm_plain(st):
    dt = st["X"].dtype
    h = st["X"].float() if st["R"] is None else st["X"].float() + st["R"].float()
    h = h.to(dt)
    x = h.float()
    y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * st["W"].float()
    out = [h] if st["res"] else []
    if st["y"]:
        out.append(y.to(dt))
    if st["fmt"]:
        out.append(_restored(y, st["fmt"]).to(torch.bfloat16))
    return out


def _norm_bwd_plain(st):
    h, d, c = st["X"].float(), st["dY"].float(), st["rstd"][:, None]
    g = d * st["W"].float()
    dX = st["G"].float() + c * (g - h * (c * c * (g * h).mean(1, keepdim=True)))
    dX = dX.to(st["X"].dtype)
    return (dX, (d * h * c).sum(0)) if st["dw"] else dX


def _head_plain(st):
    W, t = st["W"].float(), st["t"].long()
    z = (st["H"].float() @ W.t()) * st["scale"]
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    lse = top + torch.log(total)
    ok = t >= 0
    p = ok.float() if st["p"] is None else torch.where(ok, st["p"], torch.zeros_like(st["p"]))
    zt = z.gather(1, t.clamp(min=0))
    loss = (p * (lse - zt)).sum(1)
    d = (e / total) * p.sum(1, keepdim=True)
    d.scatter_add_(1, t.clamp(min=0), -p)
    d *= st["w"][:, None] * st["scale"]
    return loss, lse[:, 0], (d @ W).to(torch.bfloat16)


def _run_plain(st):
    return {"norm": _norm_plain, "norm_bwd": _norm_bwd_plain, "adapt": _adapters_plain, "adapt_bwd": _adapters_bwd_plain,
            "head": _head_plain}[st["kind"]](st)


def _run_own(st):
    from qlora_parameter_efficient_amd import block, mx

    kind = st["kind"]
    if kind == "norm":
        h, y, q = block.lq_rmsnorm_fwd(st["X"], st["W"], EPS, R=st["R"], need_y=st["y"], format=st["fmt"] or None)
        out = [h] if st["res"] else []
        if st["y"]:
            out.append(y)
        if st["fmt"]:
            out.append(mx.lq_mx_dequantize(q, torch.bfloat16))
        return out
    if kind == "norm_bwd":
        dX, dW = block.lq_rmsnorm_bwd(st["dY"], st["X"], st["W"], EPS, rstd=st["rstd"], dH=st["G"], need_dw=st["dw"])
        return (dX, dW) if st["dw"] else dX
    if kind == "head":
        return block.lq_head_loss(st["H"], st["W"], st["t"], st["p"], st["w"], st["scale"])
    pool = block.AdapterPool(st["A"], st["B"], st["scale"], st["rank"])
    if kind == "adapt":
        return block.lq_adapters_fwd(st["X"], pool, st["rows"], st["Y"])
    return block.lq_adapters_bwd(st["dY"], st["X"], pool, st["rows"], st["dX"], T_saved=st["T"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------ floor, exact

def work(case):
    kind, M, K = case["kind"], case["M"], case["K"]
    if kind in ("norm", "norm_bwd"):
        e = 4 if case["dt"] == "f32" else 2
        if kind == "norm_bwd":  # dY, H, G read, dX written
            return dict(bytes=4 * e * M * K + 4 * M + e * K + 4 * K * case["dw"], flops=(10.0 + 3 * case["dw"]) * M * K)
        n = e * (1 + 2 * case["res"] + case["y"])
        if case["fmt"]:  # codes and scales written, read once, and the values written
            n += 2 * ((1.0 if case["fmt"] == "fp8" else 0.5) + 1 / 32) + 2
        return dict(bytes=n * M * K + e * K, flops=6.0 * M * K)
    if kind == "head":
        V, k = case["V"], case["k"]
        return dict(bytes=2 * V * K + 4 * M * K + (4 + 4 * (k > 1)) * M * k + 12 * M, flops=4.0 * M * V * K)
    N, r, n = case["N"], case["r"], case["slots"]
    met = n * (1.0 - (1.0 - 1.0 / n) ** (case["requests"] * 15 / 16)) if n > 1 else 1.0
    rank = 0.5 * r + 0.25 * (r + 1)
    factors, rows = 2.0 * met * rank * (N + K), M * 15 / 16 if case["requests"] > 1 else M
    if kind == "adapt":
        return dict(bytes=factors + 2 * M * K + 4 * M * N + 4 * M, flops=2.0 * rows * rank * (N + K))
    # dY, X, T, dX in and out, dA and dB of every place
    return dict(bytes=factors + 2 * M * N + 6 * M * K + 4 * M * r + 4 * M + 4 * n * r * (N + K), flops=4.0 * rows * rank * (N + K))


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "norm":
        h = st["X"].double()
        if case["res"]:
            h = (h + st["R"].double()).to(_type(case)).double()
        y = h / torch.sqrt((h * h).sum(1, keepdim=True) / case["K"] + EPS) * st["W"].double()
        return ([h] if case["res"] else []) + ([y] if case["y"] else []) + ([None] if case["fmt"] else [])
    if kind == "norm_bwd":
        h, d, c = st["X"].double(), st["dY"].double(), st["rstd"].double().view(-1, 1)
        g = st["W"].double() * d
        inner = (g * h).sum(1, keepdim=True) / case["K"]
        dX = g * c - h * c**3 * inner + st["G"].double()
        return (dX, torch.mv((d * h).t(), c[:, 0])) if case["dw"] else dX
    if kind == "head":
        H, W, t = st["H"].double(), st["W"].double(), st["t"].long()
        z = torch.matmul(H, W.T) * st["scale"]
        lse = torch.logsumexp(z, 1)
        soft = torch.exp(z - lse[:, None])
        loss, hot = torch.zeros_like(lse), torch.zeros_like(z)
        for j in range(case["k"]):
            has = t[:, j] >= 0
            q = has.double() if st["p"] is None else torch.where(has, st["p"][:, j].double(), torch.zeros_like(lse))
            col = t[:, j].clamp(min=0)[:, None]
            loss += q * (lse - torch.take_along_dim(z, col, 1)[:, 0])
            hot.scatter_add_(1, col, q[:, None])
        d = (soft * hot.sum(1, keepdim=True) - hot) * st["w"].double()[:, None] * st["scale"]
        return loss, lse, torch.matmul(d, W)
    # adapters, one place at a time
    N, K, n, r = case["N"], case["K"], case["slots"], case["r"]
    x = st["X"].double()
    rows, ranks, scales = st["rows"].tolist(), st["rank"].tolist(), st["scale"].double().tolist()
    out = (st["Y"] if kind == "adapt" else st["dX"]).double()
    if kind == "adapt_bwd":
        d = st["dY"].double()
        dA, dB = torch.zeros((n, r, K), dtype=torch.float64, device=DEV), torch.zeros((n, N, r), dtype=torch.float64, device=DEV)
    for s in range(n):
        i = [m for m, a in enumerate(rows) if a == s]
        if not i:
            continue
        i, e = torch.tensor(i, device=DEV), ranks[s]
        A, B = st["A"][s, :e].double(), st["B"][s, :, :e].double()
        if kind == "adapt":
            out[i] += scales[s] * (x[i] @ A.T) @ B.T
        else:
            U = d[i] @ B
            out[i] += scales[s] * U @ A
            dA[s, :e] = scales[s] * U.T @ x[i]
            dB[s, :, :e] = scales[s] * d[i].T @ st["T"][i, :e].double()
    return out if kind == "adapt" else (out, dA, dB)
