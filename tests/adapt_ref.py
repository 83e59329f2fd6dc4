"""Plain 64-bit forms of the operators that adapt a layer of experts, and the tolerances of the tests.

The router's gradients are those of automatic differentiation of the definitions in fp64, which
test_adapt_ref.py holds against differences.  Tolerances count roundings."""

import math

import torch

TINY = 1e-30
U32 = 2.0 ** -24
U = {torch.float64: 2.0 ** -53, torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
LEAST = {torch.float64: 2.0 ** -1074, torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}      # smallest steps


def inside(got, want, bound, what=""):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((err - bound).max()):.3e}"


def scores(x, there, score):
    """(scores, normalised scores) of fp64 logits x, 0 where not `there`."""
    if score == "softmax":
        top = torch.where(there, x, -math.inf).amax(1, keepdim=True).detach()
        p = torch.where(there, torch.exp(torch.where(there, x - top, 0.0)), 0.0)
        p = p / p.sum(1, keepdim=True).clamp(min=TINY)
        return p, p
    s = torch.where(there, torch.sigmoid(torch.where(there, x, 0.0)), 0.0)
    return s, s / s.sum(1, keepdim=True).clamp(min=TINY)


def spans(offsets, T):
    cuts = [0, T] if offsets is None else [min(max(int(o), 0), T) for o in offsets.tolist()]
    return list(zip(cuts[:-1], cuts[1:]))


def balance(x, ids, score, offsets):
    """(loss as a function of fp64 x, counts, seq_scale)."""
    T, E = x.shape
    k = ids.shape[1]
    there = x.detach() > -math.inf
    _, p = scores(x, there, score)
    rows = spans(offsets, T)
    counts = torch.zeros(len(rows), E, dtype=torch.long, device=x.device)
    n = torch.zeros(len(rows), dtype=torch.float64, device=x.device)
    P = []
    for s, (lo, hi) in enumerate(rows):
        mine = ids[lo:hi].reshape(-1) if hi > lo else ids[:0].reshape(-1)
        mine = mine[(mine >= 0) & (mine < E)].long()
        counts[s] = torch.bincount(mine, minlength=E)
        n[s] = there[lo:hi].any(1).sum() if hi > lo else 0
        P.append(p[lo:hi].sum(0) if hi > lo else p.new_zeros(E))
    full = (n > 0).sum()
    scale = torch.where(n > 0, E / (k * n.clamp(min=1) ** 2 * full.clamp(min=1)), 0.0)
    loss = (scale[:, None] * counts * torch.stack(P)).sum()
    return loss, counts, scale


def weights(x, ids, score, renorm, scale):
    """The router's weights as a function of fp64 x; 0 for ids of -1, of masked and of no experts."""
    E = x.shape[1]
    there = x.detach() > -math.inf
    s, _ = scores(x, there, score)
    at = ids.clamp(0, E - 1).long()
    w = torch.where((ids >= 0) & (ids < E), s.gather(1, at), 0.0)
    if renorm:
        w = w / w.sum(1, keepdim=True).clamp(min=TINY)
    return w * scale


def gate_grad(logits, ids, grad_weights, score, renorm, scale, balance_part=None):
    """(gradient fp64, bound of an fp32 evaluation rounded once).  balance_part: (counts, seq_scale, grad_loss, offsets).

    A score is off by at most (|l - top| + 12) 2^-24 of itself (the exponential's argument and value, the sum of
    positive terms, reciprocal, product); with |l - top| < 40 that is 52 roundings.  A gradient is a sum of
    products of at most four such factors: 256 roundings of the magnitudes cover them."""
    T, E = logits.shape
    x = logits.double()
    there = x > -math.inf
    x = torch.where(there, x, -math.inf).detach()
    leaf = torch.where(there, x, 0.0).requires_grad_()
    full = torch.where(there, leaf, -math.inf)
    total = leaf.sum() * 0.0
    at = ids.clamp(0, E - 1).long()
    ok = (ids >= 0) & (ids < E) & there.gather(1, at)
    s, p = scores(x, there, score)
    mag = torch.zeros(T, E, dtype=torch.float64, device=x.device)
    rest = 1.0 if score == "softmax" else 1.0 - s
    if grad_weights is not None:
        gw = torch.where(ok, grad_weights.double(), 0.0)
        w = weights(full, torch.where(ok, ids, -1), score, renorm, scale)
        total = total + (w * gw).sum()
        chosen = torch.where(ok, s.gather(1, at), 0.0)
        if renorm:
            W = chosen.sum(1, keepdim=True).clamp(min=TINY)
            h = (gw.abs() + (gw.abs() * chosen).sum(1, keepdim=True) / W) / W * abs(scale)
        else:
            h = gw.abs() * abs(scale)
        h = torch.where(ok, h, 0.0)
        H = torch.zeros_like(mag).scatter_add_(1, at, h)
        mag += s * rest * H
        if score == "softmax":
            mag += s * (h * chosen).sum(1, keepdim=True)
    if balance_part is not None:
        counts, seq_scale, grad_loss, offsets = balance_part
        _, pl = scores(full, there, score)
        g = float(grad_loss)
        for i, (lo, hi) in enumerate(spans(offsets, T)):
            if hi > lo:
                a = g * seq_scale[i].double() * counts[i].double()
                total = total + (a * pl[lo:hi]).sum()
                mag[lo:hi] += p[lo:hi] * (a.abs() + (a.abs() * p[lo:hi]).sum(1, keepdim=True))
    grad = torch.autograd.grad(total, leaf)[0]
    grad = torch.where(there, grad, 0.0)
    dt = logits.dtype
    return grad, 256 * U32 * mag + (U[dt] * 1.01 if dt != torch.float32 else 0.0) * grad.abs() + LEAST[dt]
