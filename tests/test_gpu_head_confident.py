"""lq_head_loss on rows whose largest logit is a target: the usual rows of a trained
model, and of a teacher's top entries.

H is h in its first column, zero elsewhere, so that the logits are h W[v, 0]: one
product of two bf16 values, exact in float32.  In the other columns W is zero but for one row
v, so that dH there is D_v W_v: one product, and what is off is D_v's own error
and dH's rounding.

Tolerances, u = 2^-24: an exponential of a difference d is off by (|d| + 4) u of
itself (its argument's product with log2 e, twice), a sum over V of positive terms by its
longest chain, V / 1024 + 32 additions, so every probability and every sum of
probabilities by REL = (V / 1024 + 64 + 4 max |d|) u relative."""
import math

import pytest
import torch

from qlora_parameter_efficient_amd import block

from .block_helpers import HALF_BF16, U32
from .gpu_helpers import DEV, announce

pytestmark = pytest.mark.gpu
K = 64


def rel(V, span):
    return (V / 1024 + 64 + 4 * span) * U32


def case(M, V, h, weights, probe):
    """weights: {v: W[v, 0]}; logits h W[v, 0].  Logits in float64 of one row, H, W"""
    H = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    W = torch.zeros((V, K), dtype=torch.bfloat16, device=DEV)
    H[:, 0] = h
    for v, x in weights.items():
        W[v, 0] = x
    g = torch.Generator(device=DEV).manual_seed(V + probe)
    W[probe, 1:] = torch.randn(K - 1, generator=g, device=DEV).bfloat16()
    return (H[0, 0].double() * W[:, 0].double()).cpu(), H, W


def share_of(V, p):
    """The logit that has probability p beside V - 1 zeros, as bf16."""
    return float(torch.tensor(math.log(p / (1.0 - p) * max(V - 1, 1))).bfloat16())


@pytest.mark.parametrize("p", [0.6, 0.7, 0.9, 0.99, 0.9999])
@pytest.mark.parametrize("M,V", [(1, 256), (300, 300), (3, 2048), (130, 4096), (2, 70001)])
def test_label_that_is_the_largest_logit(M, V, p):
    """D_t = -(1 - p_t), of all other logits' exponentials: its largest entry, which
    is exact in bf16; what float32 keeps of 1 - p must not be lost by subtracting."""
    announce(f"confident label M={M} V={V} p={p}")
    for t in (0, V - 1):
        z, H, W = case(M, V, 1.0, {t: share_of(V, p)}, t)
        w = torch.full((M,), 0.37, device=DEV)
        _, lse, dH = block.lq_head_loss(H, W, torch.full((M,), t, dtype=torch.int32, device=DEV), w=w)
        e = torch.exp(z - z.max())
        rest = float((e.sum() - e[t]) / e.sum()) if p < 0.999 else float(e[torch.arange(V) != t].sum() / e.sum())
        ref = -w[0].double() * rest * W[t, 1:].double()
        r = rel(V, float(z.max()))
        assert bool(((dH[:, 1:].double() - ref).abs() <= (HALF_BF16 + (1 + HALF_BF16) * (r + 8 * U32)) * ref.abs()).all())
        assert abs(float(lse[0]) - float(torch.logsumexp(z, 0))) <= r + U32 * float(lse[0])


TEACHER = {  # targets' probabilities, logits, and an entry to look at beside the largest
    "the argmax, matched too little": ({5: 0.5, 6: 0.25, 7: 0.25}, {5: 12.0, 6: 1.0}, 5),
    "the argmax, matched too much": ({5: 0.5, 6: 0.25, 7: 0.25}, {5: 6.0, 6: 5.5, 7: 5.0, 9: 4.5}, 5),
    "another target": ({5: 0.6, 6: 0.4}, {5: 9.0, 6: 2.0}, 6),
    "no target, beside a matched argmax": ({5: 0.75, 6: 0.25}, {5: 9.0, 9: 8.0, 6: -3.0}, 9),
    "the argmax of equal logits, one a target": ({5: 1.0, 6: 0.5}, {5: 10.0, 9: 10.0}, 9),
    "one index twice": ({5: 0.375, 6: 0.25}, {5: 8.5, 6: 1.0}, 5),
}


@pytest.mark.parametrize("what", TEACHER)
@pytest.mark.parametrize("M,V,shift", [(1, 256, 0), (40, 1000, 0), (5, 70001, 0), (5, 70001, 69980)])
def test_a_teachers_entries_with_the_argmax(M, V, shift, what):
    """Entry D_v = P p_v - q_v, formed in float32 from terms off by REL each, and rounded to
    bf16 over the row's largest: half a step for all but the largest."""
    announce(f"teacher M={M} V={V} shift={shift}: {what}")
    q, weights, probe = TEACHER[what]
    twice = what == "one index twice"
    ids = [v + shift for v in q] + ([5 + shift] if twice else [-1])
    ps = list(q.values()) + ([0.375] if twice else [9.0])
    t = torch.tensor(ids, dtype=torch.int32, device=DEV).expand(M, -1).contiguous()
    p = torch.tensor(ps, device=DEV).expand(M, -1).contiguous()
    at = {v + shift: x for v, x in weights.items()}
    z = case(M, V, 1.0, at, probe + shift)[0]
    soft = torch.softmax(z, 0)
    d = torch.zeros_like(z)
    for i, x in zip(ids, ps):
        if i >= 0:
            d[i] -= x
    total = -float(d.sum())
    d += total * soft
    big = int(d.abs().argmax())
    for v in {probe + shift, big}:
        _, H, W = case(M, V, 1.0, at, v)
        _, _, dH = block.lq_head_loss(H, W, t, p=p)
        ref = d[v] * W[v, 1:].double().cpu()
        r = rel(V, float(z.max() - z.min())) * total * (float(soft[v]) + 1.0)
        own = HALF_BF16 * abs(float(d[v])) if v != big else 0.0
        err = (own + (1 + HALF_BF16) * r) * W[v, 1:].double().cpu().abs()
        assert bool(((dH[:, 1:].double().cpu() - ref).abs() <= HALF_BF16 * ref.abs() + (1 + HALF_BF16) * err).all()), v


def test_a_row_that_is_all_but_certain():
    """1 - p far below 2^-24: the gradient is -(1 - p), not what 1 / sum - 1 leaves."""
    V = 1000
    announce("certain row")
    for h in (24.0, 40.0, 80.0, 200.0):
        z, H, W = case(4, V, h, {5: 1.0}, 5)
        loss, _, dH = block.lq_head_loss(H, W, torch.full((4,), 5, dtype=torch.int32, device=DEV))
        rest = (V - 1) * math.exp(-h)
        ref = -rest / (1.0 + rest) * W[5, 1:].double()
        tiny = 2.0**-126  # float32's and bf16's smallest normal value
        e = HALF_BF16 + (1 + HALF_BF16) * (rel(V, h) + 8 * U32)
        assert bool(((dH[:, 1:].double() - ref).abs() <= e * ref.abs() + 4 * tiny).all()), h


@pytest.mark.parametrize("scale", [1.0, 0.75])
@pytest.mark.parametrize("V", [300, 70001])
def test_loss_of_large_confident_logits(V, scale):
    """Logits in the hundreds, the label's largest by a little or by much: the loss is
    log(1 + the others' sum), as exact as that sum; and (top - z_t) + log(sum) otherwise."""
    announce(f"loss of large logits V={V} scale={scale}")
    for near in (284.0, 288.0, 296.0, 300.0):
        z, H, W = case(7, V, 4.0, {5: 75.0, 9: near / 4.0}, 11)
        z = z * scale
        for t in (5, 9):
            loss, lse, _ = block.lq_head_loss(H, W, torch.full((7,), t, dtype=torch.int32, device=DEV), logit_scale=scale)
            d = z - z.max()
            e = torch.exp(d)
            top = int(z.argmax())
            want = float((z.max() - z[t]) + torch.log1p(e[torch.arange(V) != top].sum()))
            assert bool(((loss.double() - want).abs() <= rel(V, float(z.max() - z[9]) + 1.0) * want).all()), (near, t)
            assert abs(float(lse[0]) - float(torch.logsumexp(z, 0))) <= U32 * float(lse[0]) + rel(V, 0.0)


@pytest.mark.parametrize("V", [1, 60, 1000, 70001])
@pytest.mark.parametrize("h", [40.0, 120.0, 200.0])
def test_heavy_weights_on_a_certain_row(V, h):
    """All of 100 targets are the largest logit, with weights of 50 together: the gradient is
    50 (1 - p), down to nothing, and never 0 times an overflow."""
    announce(f"heavy weights V={V} h={h}")
    t = V // 2
    z, H, W = case(3, V, h, {t: 1.0}, t)
    ids = torch.full((3, 100), t, dtype=torch.int32, device=DEV)
    loss, _, dH = block.lq_head_loss(H, W, ids, p=torch.full((3, 100), 0.5, device=DEV))
    rest = (V - 1) * math.exp(-h)
    ref = -50.0 * rest / (1.0 + rest) * W[t, 1:].double()
    tiny = 2.0**-126
    e = HALF_BF16 + (1 + HALF_BF16) * (rel(V, h) + 108 * U32)
    assert bool(((dH[:, 1:].double() - ref).abs() <= e * ref.abs() + 4 * tiny).all())
    want = 50.0 * math.log1p(rest)
    assert bool(((loss.double() - want).abs() <= (rel(V, h) + 108 * U32) * want + 200 * tiny).all())
