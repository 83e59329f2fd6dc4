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

    A score is off by at most (1.5 |l - top| + 4) 2^-24 of itself from the exponential (its argument times log2(e) rounded,
    log2(e) itself, two units in the power), and 8 more from the sum of positive terms, the quotient and the
    product; with |l - top| < 32 that is 60 roundings.  A gradient is a sum of products of at most four such
    factors: 256 roundings of the magnitudes cover them."""
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


# ------------------------------------------------------------- low-rank adapters
def chain(n):
    """Roundings of a sum of n products on the tensor cores: a truncating adder (2 U32 a time) for each 8 of them, and 64
    more for the join of parts and the scale."""
    return (n / 8 + 64) * 2 * U32


def split_error(dtype, out_dtype):
    """What the narrow side may lose as a matrix operand: three bf16 parts hold 24 bits, two tf32 parts (beside fp16) 22
    and more.  Beside 16-bit results the bound allows what two bf16 parts lose, 2^-17; test_gpu_adapt_bits.py allows nothing."""
    return 2.0 ** -17 if dtype == torch.bfloat16 and out_dtype != torch.float32 else 2.0 ** -22


def lora(x, a, b, ids, scales, add, out_dtype):
    """(out fp64, bound)."""
    L, N, R = b.shape
    K = x.shape[1]
    lead = tuple(ids.shape)
    flat = ids.reshape(-1)
    S = flat.numel()
    k = S // ids.shape[0] if ids.shape[0] else 1
    rows = x if x.shape[0] == S else x.repeat_interleave(k, 0)
    out = torch.zeros(S, N, dtype=torch.float64, device=x.device)
    bound = torch.zeros_like(out)
    for e in torch.unique(flat[(flat >= 0) & (flat < L)]).tolist():
        s = (flat == e).nonzero()[:, 0]
        c = 1.0 if scales is None else float(scales[e])
        xe, A, B = rows[s].double(), a[e].double(), b[e].double()
        u, eu = xe @ A.t(), (xe.abs() @ A.abs().t()) * chain(K)
        out[s] = c * (u @ B.t())
        bound[s] = abs(c) * ((eu + (u.abs() + eu) * (split_error(x.dtype, out_dtype) + chain(3 * R))) @ B.abs().t())
    if add is not None:
        out = out + add.double().reshape(S, N)
    u = U[out_dtype] * 1.01
    bound = (bound + out.abs() * 2 * U32) * (1 + u) + out.abs() * (u if out_dtype != torch.float32 else 0.0) + LEAST[out_dtype]
    return out.view(*lead, N), bound.view(*lead, N)


def lora_grads(dy, x, a, b, ids, scales, add):
    """((grad_x, bound), (grad_a, bound), (grad_b, bound)) in fp64."""
    L, N, R = b.shape
    K = x.shape[1]
    flat = ids.reshape(-1)
    S = flat.numel()
    k = S // ids.shape[0] if ids.shape[0] else 1
    share = x.shape[0] != S
    rows = x.repeat_interleave(k, 0) if share else x
    dy = dy.reshape(S, N).double()
    zero = lambda *s: torch.zeros(*s, dtype=torch.float64, device=x.device)      # noqa: E731
    dr, er = zero(S, K), zero(S, K)
    da, ea, db, eb = zero(L, R, K), zero(L, R, K), zero(L, N, R), zero(L, N, R)
    for e in torch.unique(flat[(flat >= 0) & (flat < L)]).tolist():
        s = (flat == e).nonzero()[:, 0]
        c = 1.0 if scales is None else float(scales[e])
        xe, A, B, g = rows[s].double(), a[e].double(), b[e].double(), dy[s]
        n = len(s)
        u, eu = c * (xe @ A.t()), abs(c) * (xe.abs() @ A.abs().t()) * chain(K)
        v, ev = c * (g @ B), abs(c) * (g.abs() @ B.abs()) * chain(N)
        split = 2.0 ** -17 if x.dtype == torch.bfloat16 and not share else 2.0 ** -22
        dr[s] = v @ A
        er[s] = (ev + (v.abs() + ev) * (split + chain(3 * R))) @ A.abs()
        da[e] = v.t() @ xe
        ea[e] = (ev + (v.abs() + ev) * (2.0 ** -22 + chain(3 * n))).t() @ xe.abs()
        db[e] = g.t() @ u
        eb[e] = g.abs().t() @ (eu + (u.abs() + eu) * (2.0 ** -22 + chain(3 * n)))
    if share:
        er = (er + dr.abs() * (k + 1) * U32).view(x.shape[0], k, K).sum(1)
        dr = dr.view(x.shape[0], k, K).sum(1)
    if add is not None:
        dr = dr + add.double()
    u = U[x.dtype] * 1.01
    return ((dr, (er + dr.abs() * 2 * U32) * (1 + u) + dr.abs() * u + LEAST[x.dtype]),
            (da, ea + LEAST[torch.float32]), (db, eb + LEAST[torch.float32]))
