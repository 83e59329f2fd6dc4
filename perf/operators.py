"""Measured cases of the FP8 mixture-of-experts operators, each beside its plain form.

Five operators, all of one expert layer in 8-bit floating point (e4m3 codes, one
fp32 scale per 128 values of an activation row and per 128 x 128 block of a
weight matrix):

* gate     router logits -> the chosen experts of each token and their weights
* quant    rows -> e4m3 codes and scales; with `gated`, of act(gate) * up
* product  the routed experts' matrix products (one row per token or per slot, or one dense matrix)
* combine  the weighted sum of a token's expert rows, with an optional row added
* layer    gate, quant, both products with the gated activation between them, and combine, in one call

With `own` false, run() computes them from elementary torch operations in fp32;
with `own` true, by the framework's calls.  exact() computes them in 64 bits.
"""

import math

import torch

own = False

QK = 128              # values per scale along a row, and weight rows per scale
FP8_MAX = 448.0       # largest finite e4m3 value
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # the router of one decoded token: 128 experts, 8 chosen, bf16 logits
        dict(name="gate 1x128", op="gate", tokens=1, experts=128, top_k=8, dtype="bf16", score="softmax", bias=False,
             groups=1, topk_groups=1, group_top=1, renorm=True, scale=1.0, masked=0.0, pitch=128),
        # a mid-sized batch with expert groups and a balancing bias; some experts are
        # masked, the logits are columns of a wider matrix, some rows have no expert left
        dict(name="gate 777x256 grouped", op="gate", tokens=777, experts=256, top_k=8, dtype="fp32", score="sigmoid",
             bias=True, groups=8, topk_groups=4, group_top=2, renorm=True, scale=2.5, masked=0.05, pitch=263),
        # the router of a long prefill
        dict(name="gate 65536x128", op="gate", tokens=65536, experts=128, top_k=8, dtype="bf16", score="softmax",
             bias=False, groups=1, topk_groups=1, group_top=1, renorm=True, scale=1.0, masked=0.0, pitch=128),
        # activations of a small decode batch
        dict(name="quant 64x2048", op="quant", gated=False, rows=64, cols=2048, dtype="bf16", act="silu"),
        # the step between the two expert products of a prefill: 8191 tokens, 8 slots each
        dict(name="quant gated 65528x1408", op="quant", gated=True, rows=65528, cols=1408, dtype="bf16", act="silu"),
        # one decoded token: 8 experts' matrices are read once
        dict(name="product 1 token", op="product", kind="token", tokens=1, experts=128, top_k=8, nrows=768, ncols=2048,
             out="fp32", routing="uniform", unrouted=0.0),
        # ragged: uneven experts, slots with no expert, rows and columns that end inside a scale block
        dict(name="product 509 ragged", op="product", kind="slots", tokens=509, experts=60, top_k=4, nrows=1414,
             ncols=2000, out="fp32", routing="zipf", unrouted=0.02),
        # the prefill batch of the framework's benchmark
        dict(name="product 8191 tokens", op="product", kind="token", tokens=8191, experts=128, top_k=8, nrows=1408,
             ncols=2816, out="bf16", routing="uniform", unrouted=0.0),
        # a small decode batch, with the shared expert's rows added
        dict(name="combine 8x2048", op="combine", tokens=8, top_k=8, cols=2048, dtype="fp32", out="bf16", add=True,
             unrouted=0.0),
        # the prefill batch; some slots have no expert
        dict(name="combine 8191x2816", op="combine", tokens=8191, top_k=8, cols=2816, dtype="bf16", out="bf16",
             add=False, unrouted=0.02),
        # a whole expert layer for one decoded token
        dict(name="layer 1 token", op="layer", tokens=1, experts=128, top_k=8, hidden=2048, inter=768, dtype="bf16",
             act="silu", score="softmax", bias=False, groups=1, topk_groups=1, group_top=1, renorm=True, scale=1.0,
             masked=0.0),
        # a whole expert layer for a long prompt
        dict(name="layer 8192 tokens", op="layer", tokens=8192, experts=128, top_k=8, hidden=2048, inter=768,
             dtype="bf16", act="silu", score="sigmoid", bias=True, groups=1, topk_groups=1, group_top=1, renorm=True,
             scale=1.0, masked=0.0),
    ]


def _log(rng, lo, hi):
    """An odd whole number, spread evenly over the logarithm of [lo, hi]."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = max(lo, min(hi, n | 1))
    return n - 1 + n % 2 if n > lo else n


def _cols(rng, lo, hi, least=16):
    """An odd multiple of `least` or, as often, of 128, up to `hi`."""
    step = rng.choice([least, QK])
    return step * _log(rng, max(1, lo // step), max(1, hi // step))


def _gate_of(rng, tokens, experts):
    groups = rng.choice([g for g in (1, 1, 2, 4, 8) if experts % g == 0 and experts // g >= 2])
    topk_groups = rng.randint(1, groups)
    return dict(top_k=rng.randint(1, min(9, experts // groups * topk_groups)), score=rng.choice(["softmax", "sigmoid"]),
                bias=rng.random() < 0.5, groups=groups, topk_groups=topk_groups, group_top=rng.choice([1, 2]),
                renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]), masked=rng.choice([0.0, 0.1]))


def draw(rng):
    op = rng.choice(["gate", "quant", "product", "product", "product", "combine", "layer", "layer"])
    if op == "gate":
        experts = rng.choice([5, 8, 16, 60, 64, 72, 128, 160, 256, 384, 512])
        tokens = _log(rng, 1, 65535)
        return dict(op=op, tokens=tokens, experts=experts, dtype=rng.choice(sorted(DTYPES)),
                    pitch=experts + rng.choice([0, 0, 3, 64]), **_gate_of(rng, tokens, experts))
    if op == "quant":
        gated, cols = rng.random() < 0.5, _cols(rng, 16, 7184)
        return dict(op=op, gated=gated, rows=_log(rng, 1, max(1, min(65535, 90_000_000 // cols))), cols=cols,
                    dtype=rng.choice(sorted(DTYPES)), act=rng.choice(["silu", "gelu_tanh"]))
    if op == "combine":
        cols, k = _log(rng, 17, 7169), rng.randint(1, 9)
        return dict(op=op, tokens=_log(rng, 1, max(1, min(65535, 150_000_000 // (cols * k)))), top_k=k, cols=cols,
                    dtype=rng.choice(["fp32", "bf16"]), out=rng.choice(sorted(DTYPES)), add=rng.random() < 0.5,
                    unrouted=rng.choice([0.0, 0.05]))
    experts = rng.choice([3, 8, 24, 60, 64, 128])
    tokens = _log(rng, 1, 8191)
    if op == "layer":
        hidden = _cols(rng, 256, 2800)
        inter = _cols(rng, 128, max(144, min(2800, 390_000_000 // (experts * hidden * 3))))
        gate = _gate_of(rng, tokens, experts)
        cap = 250_000_000_000 // (6 * gate["top_k"] * hidden * inter)
        return dict(op=op, tokens=min(tokens, cap | 1), experts=experts, hidden=hidden, inter=inter,
                    dtype=rng.choice(["bf16", "fp16"]), act=rng.choice(["silu", "gelu_tanh"]), **gate)
    kind = rng.choice(["token", "slots", "dense"])
    if kind == "dense":
        experts = 1
    ncols = _cols(rng, 48, 7184)
    nrows = _cols(rng, 17, max(17, min(14337, 400_000_000 // (experts * ncols))), 1)
    k = rng.randint(1, min(experts, 8))
    cap = 250_000_000_000 // (2 * k * nrows * ncols)
    return dict(op=op, kind=kind, tokens=min(tokens, cap | 1), experts=experts, top_k=k, nrows=nrows, ncols=ncols,
                out=rng.choice(["fp32", "bf16"]), routing="uniform" if kind == "dense" else rng.choice(["uniform", "zipf"]),
                unrouted=0.0 if kind == "dense" else rng.choice([0.0, 0.05]))


# ------------------------------------------------------------------ inputs
def _blocks(n):
    return (n + QK - 1) // QK


def _gen(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed((seed * 1_000_003 + 17) % (1 << 62))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _weights(g, experts, nrows, ncols):
    """Expert matrices as a checkpoint stores them: e4m3 codes that fill the range of
    their block, and the blocks' scales (weights of about N(0, 0.02))."""
    w = torch.empty(experts, nrows, ncols, dtype=torch.float8_e4m3fn, device="cuda")
    step = max(1, (1 << 28) // (nrows * ncols))
    for e in range(0, experts, step):
        n = min(experts, e + step) - e
        w[e:e + n] = (_randn(g, n, nrows, ncols) * 110.0).clamp_(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    s = torch.rand(experts, _blocks(nrows), _blocks(ncols), generator=g, device="cuda") + 0.6
    return w, s * (0.02 / 110.0)


def _rows(g, rows, cols, dtype):
    """Activation rows N(0, 1) with one column in a hundred twenty times as large."""
    x = _randn(g, rows, cols)
    big = torch.rand(cols, generator=g, device="cuda") < 0.01
    return (x * torch.where(big, 20.0, 1.0)).to(dtype)


def _logits(g, case):
    """Router logits with uneven experts.  Scores that a 32-bit and a 64-bit
    evaluation could order differently are drawn again; equal ones (which bf16
    logits have often) stay, and go to the lowest expert."""
    T, E = case["tokens"], case["experts"]
    dtype = DTYPES[case["dtype"]]
    popular = _randn(g, E) * 0.5
    # balancing biases of a trained router: small, a few distinct values
    bias = torch.round(_randn(g, E) * 8) / 256 if case["bias"] else None
    masked = torch.rand(T, E, generator=g, device="cuda") < case["masked"]
    if case["masked"] and T > 2:
        masked[T // 2] = True                       # a row that has no expert left
        masked[T // 3, 1:] = True                   # and one that has a single one
    logits = torch.zeros(T, E, device="cuda", dtype=dtype)
    bad = torch.ones(T, dtype=torch.bool, device="cuda")
    for _ in range(12):
        if not bool(bad.any()):
            break
        new = (_randn(g, T, E) * 1.2 + popular).to(dtype)
        new = torch.where(masked, torch.full_like(new, -math.inf), new)
        logits = torch.where(bad[:, None], new, logits)
        bad = _close(logits, bias, case)
    # what is still too close to call: equal logits, ordered by bias and index alone
    logits = torch.where(bad[:, None] & ~masked, torch.zeros_like(logits), logits)
    if case.get("pitch", E) != E:
        wide = torch.zeros(T, case["pitch"], device="cuda", dtype=dtype)
        wide[:, :E] = logits
        logits = wide[:, :E]
    return logits, bias


def _scores64(logits, bias, case):
    """(score, key that orders the choice, available) in 64 bits."""
    x = logits.double()
    there = x > -math.inf
    if case["score"] == "softmax":
        top = x.max(1, keepdim=True).values
        p = torch.where(there, (x - torch.where(top > -math.inf, top, 0.0)).exp(), 0.0)
        s = p / p.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        s = torch.where(there, 1.0 / (1.0 + torch.exp(-x)), 0.0)
    key = x if bias is None and case["groups"] == 1 else s + (0.0 if bias is None else bias.double())
    return s, torch.where(there, key, -math.inf), there


def _groups64(key, case):
    """Each group's sum of its best experts' keys; -inf for a group with none available."""
    T, E = key.shape
    best = key.view(T, case["groups"], -1).sort(2, descending=True).values[:, :, :case["group_top"]]
    total = torch.where(best > -math.inf, best, 0.0).sum(2)
    return torch.where(best[:, :, 0] > -math.inf, total, -math.inf)


def _close(logits, bias, case):
    """Rows whose choice hangs on a difference that 32-bit rounding could turn."""
    _, key, _ = _scores64(logits, bias, case)
    least = 5e-7 if case["score"] == "sigmoid" else 1e-7     # a few roundings of the scores' size

    def near(v):
        v = v.sort(1, descending=True).values
        gap = v[:, :-1] - v[:, 1:]
        return ((gap > 0) & (gap < least)).any(1)

    if case["groups"] == 1:
        if bias is None:
            return torch.zeros(logits.shape[0], dtype=torch.bool, device=logits.device)
        return near(key.topk(min(case["top_k"] + 1, key.shape[1]), 1).values)
    g = _groups64(key, case)
    rank = torch.argsort(g, dim=1, descending=True, stable=True)[:, :case["topk_groups"]]
    inside = torch.zeros_like(g, dtype=torch.bool).scatter_(1, rank, True)
    inside = inside.repeat_interleave(key.shape[1] // case["groups"], 1)
    key = torch.where(inside, key, -math.inf)
    return near(g) | near(key.topk(min(case["top_k"] + 1, key.shape[1]), 1).values)


def _ids(g, case):
    """Distinct experts per token, uniform or with Zipf popularity; unrouted slots are -1."""
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    pop = torch.zeros(E, device="cuda")
    if case["routing"] == "zipf":
        pop = -1.1 * torch.log1p(torch.randperm(E, generator=g, device="cuda").float())
    u = torch.rand(T, E, generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)
    ids = (pop - torch.log(-torch.log(u))).topk(k, 1).indices.to(torch.int32)
    gone = torch.rand(T, k, generator=g, device="cuda") < case["unrouted"]
    return torch.where(gone, -1, ids).to(torch.int32).contiguous()


def prepare(case, seed):
    g = _gen(case, seed)
    op = case["op"]
    st = {"case": case}
    if op == "gate":
        st["logits"], st["bias"] = _logits(g, case)
    elif op == "quant":
        st["x"] = _rows(g, case["rows"], case["cols"] * (2 if case["gated"] else 1), DTYPES[case["dtype"]])
    elif op == "product":
        st["w"], st["ws"] = _weights(g, case["experts"], case["nrows"], case["ncols"])
        rows = case["tokens"] * (case["top_k"] if case["kind"] == "slots" else 1)
        st["a"], st["as"] = _quant_plain(_rows(g, rows, case["ncols"], torch.bfloat16).float())
        if case["kind"] == "dense":
            st["w"], st["ws"] = st["w"][0], st["ws"][0]
        else:
            st["ids"] = _ids(g, case)
    elif op == "combine":
        T, k, N = case["tokens"], case["top_k"], case["cols"]
        st["rows"] = _randn(g, T, k, N).to(DTYPES[case["dtype"]])
        w = torch.rand(T, k, generator=g, device="cuda") + 0.05
        w = w / w.sum(1, keepdim=True)
        st["weights"] = torch.where(torch.rand(T, k, generator=g, device="cuda") < case["unrouted"], 0.0, w)
        st["add"] = _randn(g, T, N).to(DTYPES[case["out"]]) if case["add"] else None
    else:
        st["logits"], st["bias"] = _logits(g, case)
        st["x"] = _rows(g, case["tokens"], case["hidden"], DTYPES[case["dtype"]])
        st["w13"], st["s13"] = _weights(g, case["experts"], 2 * case["inter"], case["hidden"])
        st["w2"], st["s2"] = _weights(g, case["experts"], case["hidden"], case["inter"])
    return st


# -------------------------------------------------------------- plain forms
def _gate_plain(logits, bias, case):
    x = logits.float()
    there = x > -math.inf
    if case["score"] == "softmax":
        top = x.max(1, keepdim=True).values
        p = torch.where(there, torch.exp(x - torch.where(top > -math.inf, top, 0.0)), 0.0)
        s = p / p.sum(1, keepdim=True).clamp(min=1e-30)
    else:
        s = torch.where(there, 1.0 / (1.0 + torch.exp(-x)), 0.0)
    key = x if bias is None and case["groups"] == 1 else (s if bias is None else s + bias)
    key = torch.where(there, key, -math.inf)
    if case["groups"] > 1:
        T, E = key.shape
        best = torch.sort(key.view(T, case["groups"], -1), dim=2, descending=True, stable=True).values
        best = best[:, :, :case["group_top"]]
        total = torch.where(best > -math.inf, best, 0.0).sum(2)
        total = torch.where(best[:, :, 0] > -math.inf, total, -math.inf)
        rank = torch.sort(total, dim=1, descending=True, stable=True).indices[:, :case["topk_groups"]]
        inside = torch.zeros_like(total, dtype=torch.bool).scatter_(1, rank, True)
        key = torch.where(inside.repeat_interleave(E // case["groups"], 1), key, -math.inf)
    order = torch.sort(key, dim=1, descending=True, stable=True)
    chosen, ids = order.values[:, :case["top_k"]], order.indices[:, :case["top_k"]]
    w = torch.where(chosen > -math.inf, s.gather(1, ids), 0.0)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-30)
    ids = torch.where(chosen > -math.inf, ids, -1).to(torch.int32)
    return ids, w * case["scale"]


def _quant_plain(x):
    R, K = x.shape
    nb = _blocks(K)
    b = torch.nn.functional.pad(x, (0, nb * QK - K)).view(R, nb, QK)
    s = b.abs().amax(2)
    s = s / torch.full_like(s, FP8_MAX)      # the rounded quotient (a division by a number multiplies by its reciprocal)
    v = torch.where(s[:, :, None] > 0, b / s[:, :, None], 0.0).clamp(-FP8_MAX, FP8_MAX)
    return v.view(R, nb * QK)[:, :K].to(torch.float8_e4m3fn).contiguous(), s


def _act_plain(h, act):
    g, u = h.chunk(2, dim=-1)
    z = g if act == "silu" else 1.5957691216057308 * (g + 0.044715 * g * g * g)
    return g / (1.0 + torch.exp(-z)) * u


def _dequant_rows(q, s):
    return q.float() * s.repeat_interleave(QK, 1)[:, :q.shape[1]]


def _dequant_weights(w, s):
    s = s.repeat_interleave(QK, -2)[..., :w.shape[-2], :]
    return w.float() * s.repeat_interleave(QK, -1)[..., :w.shape[-1]]


def _product_plain(w, ws, x, ids, per_slot):
    """fp32 [T, k, N] of dequantized rows x; rows of slots without an expert are 0."""
    T, k = ids.shape
    E, N, K = w.shape
    flat = ids.reshape(-1).long()
    there = flat >= 0
    e = flat.clamp(min=0)
    rows = torch.arange(T * k, device=w.device)
    src = rows if per_slot else rows // k
    if T * k <= E:                          # few slots: each with its own copy of its expert's matrix
        mine = _dequant_weights(w.view(torch.uint8)[e].view(torch.float8_e4m3fn), ws[e])
        out = torch.bmm(mine, x[src][:, :, None])[:, :, 0]
    else:                                   # slots sorted by expert into equally long rows of experts
        count = torch.zeros(E, dtype=torch.long, device=w.device).index_add_(0, e, torch.ones_like(e))
        order = torch.argsort(e, stable=True)
        first = torch.cumsum(count, 0) - count
        at = torch.empty_like(rows).index_copy_(0, order, rows) - first[e]
        padded = torch.zeros(E, int(count.max()), K, device=w.device)
        padded[e, at] = x[src]
        out = torch.bmm(padded, _dequant_weights(w, ws).transpose(1, 2))[e, at]
    return torch.where(there[:, None], out, 0.0).view(T, k, N)


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "gate":
        return _gate_plain(st["logits"], st["bias"], case)
    if op == "quant":
        x = st["x"].float()
        return _quant_plain(_act_plain(x, case["act"]) if case["gated"] else x)
    if op == "product":
        x = _dequant_rows(st["a"], st["as"])
        if case["kind"] == "dense":
            out = x @ _dequant_weights(st["w"], st["ws"]).t()
        else:
            out = _product_plain(st["w"], st["ws"], x, st["ids"], case["kind"] == "slots")
        return out.to(DTYPES[case["out"]])
    if op == "combine":
        w = st["weights"][:, :, None]
        y = (torch.where(w != 0, st["rows"].float(), 0.0) * w).sum(1)
        if st["add"] is not None:
            y = y + st["add"].float()
        return y.to(DTYPES[case["out"]])
    ids, weights = _gate_plain(st["logits"], st["bias"], case)
    h = _product_plain(st["w13"], st["s13"], _dequant_rows(*_quant_plain(st["x"].float())), ids, False)
    mid = _quant_plain(_act_plain(h.view(-1, h.shape[-1]), case["act"]))
    rows = _product_plain(st["w2"], st["s2"], _dequant_rows(*mid), ids, True)
    y = (rows * weights[:, :, None]).sum(1)
    return y.to(DTYPES[case["dtype"]]), ids, weights


# ------------------------------------------------------------------- calls
def _gate_args(case, bias):
    return dict(score=case["score"], bias=bias, n_groups=case["groups"], topk_groups=case["topk_groups"],
                group_top=case["group_top"], renormalize=case["renorm"], scale=case["scale"])


def _act_kind(ft, case):
    return ft.ACT_SILU if case["act"] == "silu" else ft.ACT_GELU_TANH


def _calls(st):
    import bit_quantized_moe_quantize_gb300 as ft
    case = st["case"]
    op = case["op"]
    if op == "gate":
        return ft.moe_gate(st["logits"], case["top_k"], **_gate_args(case, st["bias"]))
    if op == "quant":
        if case["gated"]:
            return ft.act_mul_quantize_fp8(st["x"], _act_kind(ft, case))
        return ft.quantize_fp8(st["x"])
    if op == "product":
        dt = DTYPES[case["out"]]
        if case["kind"] == "dense":
            return ft.matmul_fp8_fp8(st["w"], st["ws"], st["a"], st["as"], out_dtype=dt)
        call = ft.moe_fp8_fp8_slots if case["kind"] == "slots" else ft.moe_fp8_fp8
        return call(st["w"], st["ws"], st["a"], st["as"], st["ids"], out_dtype=dt)
    if op == "combine":
        return ft.moe_combine(st["rows"], st["weights"], add=st["add"], out_dtype=DTYPES[case["out"]])
    return ft.moe_layer_fp8(st["x"], st["logits"], st["w13"], st["s13"], st["w2"], st["s2"], case["top_k"],
                            _act_kind(ft, case), **_gate_args(case, st["bias"]))


def run(state):
    return _calls(state) if own else _plain(state)


# -------------------------------------------------------------------- work
def _touched(case):
    """Experts that a batch is expected to touch."""
    E, k, T = case["experts"], case["top_k"], case["tokens"]
    return E * (1.0 - (1.0 - k / E) ** T)


def work(case):
    op = case["op"]
    size = {n: d.itemsize for n, d in DTYPES.items()}
    if op == "gate":
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        return {"bytes": T * E * size[case["dtype"]] + T * k * 8, "flops": T * E * 4}
    if op == "quant":
        n = case["rows"] * case["cols"]
        read = n * size[case["dtype"]] * (2 if case["gated"] else 1)
        return {"bytes": read + n + case["rows"] * _blocks(case["cols"]) * 4, "flops": n * (8 if case["gated"] else 3)}
    if op == "product":
        T, k, N, K = case["tokens"], case["top_k"], case["nrows"], case["ncols"]
        rows = T * k if case["kind"] == "slots" else T
        matrices = _touched(case) * (N * K + _blocks(N) * _blocks(K) * 4)
        return {"bytes": matrices + rows * (K + 4 * _blocks(K)) + T * k * (4 + N * size[case["out"]]),
                "flops": 2 * T * k * N * K}
    if op == "combine":
        T, k, N = case["tokens"], case["top_k"], case["cols"]
        out = T * N * size[case["out"]]
        return {"bytes": T * k * N * size[case["dtype"]] + T * k * 4 + out * (2 if case["add"] else 1),
                "flops": 2 * T * k * N}
    T, k, H, I, E = case["tokens"], case["top_k"], case["hidden"], case["inter"], case["experts"]
    per = 3 * I * H + 4 * _blocks(H) * (_blocks(2 * I) + _blocks(I))
    return {"bytes": _touched(case) * per + T * (E * 2 + k * 8 + 2 * H * size[case["dtype"]]),
            "flops": 6 * T * k * I * H}


# ------------------------------------------------------------------- exact
def _e4m3_64(v):
    """The nearest e4m3 value, ties to even, of 64-bit values."""
    a = v.abs().clamp(max=FP8_MAX)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -40))).clamp(min=-6)
    e = torch.where(a >= 2.0 ** (e + 1), e + 1, torch.where((a < 2.0 ** e) & (e > -6), e - 1, e))
    step = 2.0 ** (e - 3)
    return torch.sign(v) * (torch.round(a / step) * step).clamp(max=FP8_MAX)


def _quant64(x):
    """(codes' values, scales) of 64-bit rows."""
    R, K = x.shape
    nb = _blocks(K)
    b = torch.zeros(R, nb * QK, dtype=torch.float64, device=x.device)
    b[:, :K] = x
    b = b.view(R, nb, QK)
    s = b.abs().amax(2) / FP8_MAX
    q = _e4m3_64(b / torch.where(s > 0, s, 1.0)[:, :, None])
    return q.view(R, nb * QK)[:, :K], s


def _act64(h, act):
    g, u = h[:, :h.shape[1] // 2], h[:, h.shape[1] // 2:]
    if act == "silu":
        return g * torch.sigmoid(g) * u
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3))) * u


def _gate64(logits, bias, case):
    s, key, there = _scores64(logits, bias, case)
    if case["groups"] > 1:
        g = _groups64(key, case)
        rank = torch.argsort(g, dim=1, descending=True, stable=True)[:, :case["topk_groups"]]
        inside = torch.zeros_like(g, dtype=torch.bool).scatter_(1, rank, True)
        key = torch.where(inside.repeat_interleave(key.shape[1] // case["groups"], 1), key, -math.inf)
    ids = torch.argsort(key, dim=1, descending=True, stable=True)[:, :case["top_k"]]
    ok = key.gather(1, ids) > -math.inf
    w = torch.where(ok, s.gather(1, ids), 0.0)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return torch.where(ok, ids, -1), w * case["scale"]


def _product64(w, ws, q, s, ids, per_slot):
    """[slots, N] in 64 bits, expert by expert."""
    T, k = ids.shape
    out = torch.zeros(T * k, w.shape[1], dtype=torch.float64, device=w.device)
    flat = ids.reshape(-1)
    K = w.shape[2]
    for e in torch.unique(flat[flat >= 0]).tolist():
        rows = (flat == e).nonzero()[:, 0]
        src = rows if per_slot else rows // k
        x = q[src].double() * s[src].double().repeat_interleave(QK, 1)[:, :K]
        m = w[e].double() * ws[e].double().repeat_interleave(QK, 0)[:w.shape[1]].repeat_interleave(QK, 1)[:, :K]
        out[rows] = x @ m.t()
    return out


def exact(case, seed):
    if work(case)["flops"] > 2e12:        # a few seconds at this card's rate in 64 bits
        return None
    st = prepare(case, seed)
    op = case["op"]
    if op == "gate":
        return None, _gate64(st["logits"], st["bias"], case)[1]
    if op == "quant":
        x = st["x"].double()
        return _quant64(_act64(x, case["act"]) if case["gated"] else x)
    if op == "product":
        q, s = st["a"].float(), st["as"]
        if case["kind"] == "dense":
            return _product64(st["w"][None], st["ws"][None], q, s,
                              torch.zeros(case["tokens"], 1, dtype=torch.int32, device="cuda"), False)
        out = _product64(st["w"], st["ws"], q, s, st["ids"], case["kind"] == "slots")
        return out.view(case["tokens"], case["top_k"], case["nrows"])
    if op == "combine":
        w = st["weights"].double()[:, :, None]
        y = (torch.where(w != 0, st["rows"].double(), 0.0) * w).sum(1)
        return y if st["add"] is None else y + st["add"].double()
    ids, weights = _gate64(st["logits"], st["bias"], case)
    h = _product64(st["w13"], st["s13"], *_quant64(st["x"].double()), ids, False)
    rows = _product64(st["w2"], st["s2"], *_quant64(_act64(h, case["act"])), ids, True)
    return (rows.view(*ids.shape, -1) * weights[:, :, None]).sum(1), None, weights
