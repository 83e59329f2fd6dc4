"""Plain 64-bit forms of the FP8 expert-layer operators, and seeded inputs.

e4m3 values are decoded from their bit fields, sums and products run in fp64,
and every tolerance the tests use is derived here from rounding alone.
"""

import math

import torch

QK = 128
FP8_MAX = 448.0
U32 = 2.0 ** -24        # unit roundoff of fp32
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}   # 24, 11 and 8 significant bits


def blocks(n):
    return (n + QK - 1) // QK


def gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def decode(codes):
    """e4m3 codes -> fp64 values, from the bit fields."""
    b = codes.view(torch.uint8).long()
    sign = 1.0 - 2.0 * (b >> 7).double()
    exp, man = (b >> 3) & 15, (b & 7).double()
    normal = (8.0 + man) * torch.exp2((exp - 10).double())
    v = torch.where(exp == 0, man * 2.0 ** -9, normal)
    return torch.where((b & 127) == 127, math.nan, sign * v)


def nearest_e4m3(v):
    """The nearest e4m3 value (ties to even) of fp64 v with |v| <= 448, and the spacing there."""
    a = v.abs()
    e = torch.frexp(a).exponent.double() - 1
    step = torch.exp2(torch.clamp(e, min=-6.0) - 3.0)
    q = torch.round(a / step) * step
    return torch.sign(v) * q.clamp(max=FP8_MAX), step


def weights(g, E, N, K):
    w = (torch.randn(E, N, K, generator=g, device="cuda") * 110).clamp_(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    s = (torch.rand(E, blocks(N), blocks(K), generator=g, device="cuda") + 0.5) * 2e-4
    return w, s


def rows(g, R, K, dtype=torch.float32):
    x = torch.randn(R, K, generator=g, device="cuda")
    return (x * torch.where(torch.rand(K, generator=g, device="cuda") < 0.02, 20.0, 1.0)).to(dtype)


def codes(g, R, K):
    """Activation codes and scales, random over the whole range."""
    q = (torch.randn(R, K, generator=g, device="cuda") * 60).clamp_(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return q, torch.rand(R, blocks(K), generator=g, device="cuda") * 0.02 + 1e-4


def ids(g, T, E, k, none=0.0, pop=None):
    u = torch.rand(T, E, generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)
    score = -torch.log(-torch.log(u)) + (0 if pop is None else pop)
    out = score.topk(k, 1).indices.to(torch.int32)
    return torch.where(torch.rand(T, k, generator=g, device="cuda") < none, -1, out).to(torch.int32).contiguous()


def expand_rows(s, K):
    return s.double().repeat_interleave(QK, 1)[:, :K]


def expand_matrix(s, N, K):
    return s.double().repeat_interleave(QK, 0)[:N].repeat_interleave(QK, 1)[:, :K]


def product(w, ws, q, s, topk_ids, per_slot, out_dtype):
    """(out [T, k, N] fp64, bound): bound on an fp32 evaluation rounded once to out_dtype.

    Products of e4m3 values have at most 8 significant bits and are exact.  Whatever
    the order of the sums, an element has at most 128 + nb additions, each off by at
    most one unit in the last place of a partial sum (2^-23; a truncating adder
    included), and four roundings from the scales: (132 + nb) 2^-23 of the sum of
    the magnitudes, plus the rounding to out_dtype."""
    T, k = topk_ids.shape
    E, N, K = w.shape
    out = torch.zeros(T * k, N, dtype=torch.float64, device=w.device)
    mag = torch.zeros_like(out)
    flat = topk_ids.reshape(-1)
    for e in torch.unique(flat[(flat >= 0) & (flat < E)]).tolist():
        sel = (flat == e).nonzero()[:, 0]
        src = sel if per_slot else sel // k
        x = decode(q[src]) * expand_rows(s[src], K)
        m = decode(w[e]) * expand_matrix(ws[e], N, K)
        out[sel] = x @ m.t()
        mag[sel] = x.abs() @ m.abs().t()
    u = 0.0 if out_dtype == torch.float32 else U[out_dtype]
    bound = (132 + blocks(K)) * 2 * U32 * mag + out.abs() * u * 1.01
    return out.view(T, k, N), bound.view(T, k, N)


def gate(logits, k, score, bias, n_groups, topk_groups, group_top, renorm, scale):
    """(ids, weights fp64, sure): `sure` marks rows whose order fp32 rounding cannot change
    (every gap that the choice hangs on is 0 or over 2e-6, about 32 roundings, of its size)."""
    x = logits.double()
    T, E = x.shape
    there = x > -math.inf
    if score == "softmax":
        top = torch.where(there, x, -math.inf).max(1, keepdim=True).values
        p = torch.where(there, torch.exp(x - torch.where(top > -math.inf, top, 0.0)), 0.0)
        s = p / p.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        s = torch.where(there, torch.sigmoid(x), 0.0)
    plain = bias is None and n_groups == 1
    key = x if plain else s + (0.0 if bias is None else bias.double())
    key = torch.where(there, key, -math.inf)
    sure = torch.ones(T, dtype=torch.bool, device=x.device)

    def clear(v, n):          # the n best and the first left out
        v = v.sort(1, descending=True).values[:, :n + 1]
        gap = v[:, :-1] - v[:, 1:]
        return ~((gap > 0) & (gap < 2e-6 * v[:, :-1].abs())).any(1)

    if n_groups > 1:
        best = key.view(T, n_groups, -1).sort(2, descending=True).values[:, :, :group_top]
        total = torch.where(best > -math.inf, best, 0.0).sum(2)
        total = torch.where(best[:, :, 0] > -math.inf, total, -math.inf)
        sure &= clear(total, topk_groups)
        pick = torch.argsort(total, dim=1, descending=True, stable=True)[:, :topk_groups]
        inside = torch.zeros_like(total, dtype=torch.bool).scatter_(1, pick, True)
        key = torch.where(inside.repeat_interleave(E // n_groups, 1), key, -math.inf)
    if not plain:
        sure &= clear(key, k)
    order = torch.argsort(key, dim=1, descending=True, stable=True)[:, :k]
    ok = key.gather(1, order) > -math.inf
    w = torch.where(ok, s.gather(1, order), 0.0)
    if renorm:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-30)
    return torch.where(ok, order, -1), w * scale, sure


def act_mul(h, kind):
    g, u = h.double().chunk(2, dim=1)
    if kind == 0:
        return g * torch.sigmoid(g) * u
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))) * u
