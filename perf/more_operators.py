"""Measured cases of the operators that adapt a layer of quantized experts, each beside its plain form.

The experts' matrices are frozen; what is trained is the router and low-rank adapters beside the
matrices, and the adapters are served.  Five operators:

* balance   router logits and choices -> a load-balance loss over packed sequences, and experts' counts
* gate_bwd  gradients of the router's weights and of that loss -> gradient of the logits
* comb_bwd  gradient of the weighted sum of expert rows -> gradients of the rows and of the weights
* lora      out = add + scale * (x A^T) B^T with an adapter (A, B) per row, or per routed slot
* lora_bwd  its gradients, of x and of every adapter's A and B

With `own` false, run() computes them from elementary torch operations in fp32;
with `own` true, by the framework's calls.  exact() computes them in 64 bits.
"""

import math

import torch

own = False

TINY = 1e-30          # smallest sum that scores are divided by
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # the router of a small training batch: one sequence
        dict(name="balance 512x128", op="balance", tokens=512, experts=128, top_k=8, dtype="bf16", score="softmax",
             seqs=0, masked=0.0, pitch=128),
        # packed sequences of a long batch, fp32 logits, rows of padding
        dict(name="balance 65536x128 packed", op="balance", tokens=65536, experts=128, top_k=8, dtype="fp32",
             score="softmax", seqs=37, masked=0.02, pitch=128),
        # sigmoid scores, renormalised and scaled, masked experts, rows of a wider matrix, several sequences
        dict(name="gate_bwd 777x256", op="gate_bwd", tokens=777, experts=256, top_k=8, dtype="fp32", score="sigmoid",
             renorm=True, scale=2.5, balance=True, seqs=5, masked=0.05, pitch=263),
        # the router of a long batch
        dict(name="gate_bwd 65536x128", op="gate_bwd", tokens=65536, experts=128, top_k=8, dtype="bf16",
             score="softmax", renorm=True, scale=1.0, balance=True, seqs=0, masked=0.0, pitch=128),
        # a few tokens
        dict(name="comb_bwd 8x2048", op="comb_bwd", tokens=8, top_k=8, cols=2048, dtype="fp32", out="bf16",
             unrouted=0.0),
        # the prefill batch of the framework's benchmark; some slots have no expert
        dict(name="comb_bwd 8191x2816", op="comb_bwd", tokens=8191, top_k=8, cols=2816, dtype="bf16", out="bf16",
             unrouted=0.02),
        # one decoded token with its request's adapter
        dict(name="lora 1 token", op="lora", tokens=1, top_k=1, adapters=64, rank=16, ncols=2048, nrows=2048,
             dtype="bf16", out="bf16", add=True, ids="spread", per_slot=False, unrouted=0.0),
        # decoding of 64 requests, most with an adapter of their own, some without any
        dict(name="lora 64 requests", op="lora", tokens=64, top_k=1, adapters=64, rank=16, ncols=4096, nrows=4096,
             dtype="bf16", out="bf16", add=True, ids="spread", per_slot=False, unrouted=0.1),
        # prompts of several requests in one batch
        dict(name="lora 8191 packed", op="lora", tokens=8191, top_k=1, adapters=12, rank=16, ncols=4096, nrows=4096,
             dtype="bf16", out="bf16", add=True, ids="packed", per_slot=False, unrouted=0.05),
        # an adapter for every expert, beside the routed product of a prompt
        dict(name="lora 2048x8 experts", op="lora", tokens=2048, top_k=8, adapters=128, rank=8, ncols=2048, nrows=1536,
             dtype="bf16", out="fp32", add=True, ids="distinct", per_slot=False, unrouted=0.0),
        # a ragged batch of a few requests' adapters, one of them without a token
        dict(name="lora_bwd 509 ragged", op="lora_bwd", tokens=509, top_k=1, adapters=6, rank=24, ncols=1000,
             nrows=1416, dtype="fp16", add=True, ids="packed", per_slot=False, unrouted=0.02),
        # a training batch of one adapter
        dict(name="lora_bwd 8192 tokens", op="lora_bwd", tokens=8192, top_k=1, adapters=1, rank=64, ncols=4096,
             nrows=4096, dtype="bf16", add=False, ids="packed", per_slot=False, unrouted=0.0),
    ]


def _log(rng, lo, hi):
    """An odd whole number, spread evenly over the logarithm of [lo, hi]."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = max(lo, min(hi, n | 1))
    return n - 1 + n % 2 if n > lo else n


def draw(rng):
    op = rng.choice(["balance", "gate_bwd", "comb_bwd", "lora", "lora", "lora", "lora_bwd", "lora_bwd"])
    if op in ("balance", "gate_bwd"):
        experts = rng.choice([5, 8, 16, 60, 64, 72, 128, 160, 256, 384, 512])
        tokens = _log(rng, 1, 65535 if experts <= 128 else 16383)
        case = dict(op=op, tokens=tokens, experts=experts, top_k=rng.randint(1, min(9, experts)),
                    dtype=rng.choice(sorted(DTYPES)), score=rng.choice(["softmax", "sigmoid"]),
                    seqs=rng.choice([0, 1, _log(rng, 2, 300)]), masked=rng.choice([0.0, 0.1]),
                    pitch=experts + rng.choice([0, 0, 3, 64]))
        if op == "gate_bwd":
            case.update(renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]), balance=rng.random() < 0.6)
        return case
    if op == "comb_bwd":
        cols, k = _log(rng, 17, 7169), rng.randint(1, 9)
        cols += rng.choice([0, 8 - cols % 8])
        return dict(op=op, tokens=_log(rng, 1, max(1, min(65535, 150_000_000 // (cols * k)))), top_k=k, cols=cols,
                    dtype=rng.choice(["fp32", "bf16"]), out=rng.choice(sorted(DTYPES)),
                    unrouted=rng.choice([0.0, 0.05]))
    kind = rng.choice(["packed", "spread", "distinct"])
    adapters = rng.choice([1, 3, 12, 64]) if kind != "distinct" else rng.choice([16, 60, 128])
    rank = 8 * _log(rng, 1, 16) if rng.random() < 0.3 else rng.choice([8, 16, 32, 64])
    ncols, nrows = 8 * _log(rng, 4, 896), 8 * _log(rng, 4, 896)
    k = rng.randint(2, 8) if kind == "distinct" else rng.choice([1, 1, 1, 4])
    slots = 40_000_000 // (ncols + nrows) if op == "lora" else 25_000_000 // (ncols + nrows)
    tokens = _log(rng, 1, max(1, min(8191, slots // k)))
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    case = dict(op=op, tokens=tokens, top_k=k, adapters=adapters, rank=rank, ncols=ncols, nrows=nrows, dtype=dtype,
                add=rng.random() < 0.7, ids=kind, per_slot=k > 1 and rng.random() < 0.5,
                unrouted=rng.choice([0.0, 0.1]))
    if op == "lora":
        case["out"] = rng.choice(["fp32", dtype])
    return case


# ------------------------------------------------------------------ inputs
def _gen(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed((seed * 1_000_003 + 29) % (1 << 62))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _router(g, case):
    """Logits with uneven experts (columns of a wider matrix where the pitch says so), the
    experts chosen for each row, and the offsets of the packed sequences (some empty)."""
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    dtype = DTYPES[case["dtype"]]
    x = _randn(g, T, E) * 1.2 + _randn(g, E) * 0.5
    masked = torch.rand(T, E, generator=g, device="cuda") < case["masked"]
    if case["masked"] and T > 2:
        masked[T // 2] = True                       # a row of padding
        masked[T // 3, 1:] = True                   # and one with a single expert
    x = torch.where(masked, -math.inf, x).to(dtype)
    wide = torch.zeros(T, case["pitch"], device="cuda", dtype=dtype)
    wide[:, :E] = x
    top = x.float().topk(k, 1)
    ids = torch.where(top.values > -math.inf, top.indices, -1).to(torch.int32).contiguous()
    offsets = None
    if case["seqs"]:
        cut = torch.randint(0, T + 1, (case["seqs"] - 1,), generator=g, device="cuda")
        ends = torch.tensor([0, T], device="cuda")
        offsets = torch.cat([ends, cut]).sort().values.to(torch.int32)
    return wide[:, :E], ids, offsets


def _adapter_ids(g, case):
    """The adapter of each slot: runs of neighbouring tokens (packed prompts), any (a decoding
    batch), or distinct ones per token (experts); -1: none.  Of several packed adapters the last has no token."""
    T, k, L = case["tokens"], case["top_k"], case["adapters"]
    if case["ids"] == "packed":
        n = max(1, min(T, 2 * L))
        start = torch.randint(0, T, (n,), generator=g, device="cuda")
        new = torch.zeros(T, dtype=torch.long, device="cuda").index_fill_(0, start, 1)
        which = torch.randint(0, max(1, L - 1), (T + 1,), generator=g, device="cuda")
        gone = torch.rand(T + 1, generator=g, device="cuda") < case["unrouted"]
        run_of = new.cumsum(0)
        ids = torch.where(gone[run_of], -1, which[run_of])[:, None].expand(T, k)
    elif case["ids"] == "distinct":
        ids = torch.rand(T, L, generator=g, device="cuda").topk(k, 1).indices
    else:
        ids = torch.randint(0, L, (T, k), generator=g, device="cuda")
    if case["ids"] != "packed":
        ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < case["unrouted"], -1, ids)
    return ids.to(torch.int32).contiguous()


def prepare(case, seed):
    g = _gen(case, seed)
    op = case["op"]
    st = {"case": case}
    if op in ("balance", "gate_bwd"):
        st["logits"], st["ids"], st["offsets"] = _router(g, case)
        if op == "gate_bwd":
            T, k = case["tokens"], case["top_k"]
            st["grad_weights"] = _randn(g, T, k)
            if case["balance"]:      # what the loss' forward call gave, and the gradient that arrives at it
                _, st["counts"], st["seq_scale"] = _balance_plain(st["logits"], st["ids"], st["offsets"], case)
                st["grad_loss"] = torch.rand((), generator=g, device="cuda") * T
    elif op == "comb_bwd":
        T, k, N = case["tokens"], case["top_k"], case["cols"]
        st["grad_out"] = _randn(g, T, N).to(DTYPES[case["out"]])
        st["rows"] = _randn(g, T, k, N).to(DTYPES[case["dtype"]])
        w = torch.rand(T, k, generator=g, device="cuda") + 0.05
        w = w / w.sum(1, keepdim=True)
        st["weights"] = torch.where(torch.rand(T, k, generator=g, device="cuda") < case["unrouted"], 0.0, w)
    else:
        T, k, L, R, K, N = (case[n] for n in ("tokens", "top_k", "adapters", "rank", "ncols", "nrows"))
        dt = DTYPES[case["dtype"]]
        ids = _adapter_ids(g, case)
        st["ids"] = ids[:, 0].contiguous() if k == 1 else ids
        lead = (T,) if k == 1 else (T, k)
        rows = T * k if case["per_slot"] else T
        st["x"] = _randn(g, rows, K).to(dt)
        st["a"] = (_randn(g, L, R, K) / math.sqrt(K)).to(dt)
        st["b"] = (_randn(g, L, N, R) * 0.3 / math.sqrt(R)).to(dt)
        st["scales"] = torch.rand(L, generator=g, device="cuda") + 0.5
        st["add"] = None
        if op == "lora":
            if case["add"]:
                st["add"] = _randn(g, *lead, N).to(DTYPES[case["out"]])
        else:
            st["grad_out"] = _randn(g, *lead, N).to(dt)
            if case["add"]:
                st["add"] = _randn(g, rows, K).to(dt)
    return st


# -------------------------------------------------------------- plain forms
def _scores_plain(logits, score):
    """(scores, their normalised form, 1 - score, rows that count) in fp32."""
    x = logits.float()
    there = x > -math.inf
    if score == "softmax":
        top = torch.where(there, x, -math.inf).amax(1, keepdim=True)
        p = torch.where(there, torch.exp(x - torch.where(top > -math.inf, top, 0.0)), 0.0)
        p = p / p.sum(1, keepdim=True).clamp(min=TINY)
        return p, p, None, there.any(1)
    s = torch.where(there, 1.0 / (1.0 + torch.exp(-x)), 0.0)
    rest = torch.where(there, 1.0 / (1.0 + torch.exp(x)), 0.0)
    return s, s / s.sum(1, keepdim=True).clamp(min=TINY), rest, there.any(1)


def _seq_of(offsets, T):
    """(sequence of each row, number of sequences)."""
    if offsets is None:
        return torch.zeros(T, dtype=torch.long, device="cuda"), 1
    row = torch.arange(T, device="cuda")
    return torch.searchsorted(offsets.long(), row, right=True) - 1, offsets.numel() - 1


def _balance_plain(logits, ids, offsets, case):
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    _, p, _, counted = _scores_plain(logits, case["score"])
    seq, S = _seq_of(offsets, T)
    n = torch.zeros(S, device="cuda").index_add_(0, seq, counted.float())
    P = torch.zeros(S, E, dtype=torch.float64, device="cuda").index_add_(0, seq, p.double())
    flat = (seq[:, None] * E + ids.long()).reshape(-1)
    hit = (ids.reshape(-1) >= 0)
    counts = torch.zeros(S * E, dtype=torch.int32, device="cuda")
    counts.index_add_(0, torch.where(hit, flat, 0), hit.to(torch.int32))
    counts = counts.view(S, E)
    scale = torch.where(n > 0, E / (k * n.clamp(min=1) ** 2 * (n > 0).sum().clamp(min=1)), 0.0)
    loss = (scale.double()[:, None] * counts * P).sum().float()
    return loss, counts, scale


def _gate_bwd_plain(st, case):
    logits, ids = st["logits"], st["ids"]
    s, p, rest, _ = _scores_plain(logits, case["score"])
    ok = ids >= 0
    at = ids.clamp(min=0).long()
    chosen = torch.where(ok, s.gather(1, at), 0.0)
    gw = torch.where(ok, st["grad_weights"], 0.0)
    if case["renorm"]:
        total = chosen.sum(1, keepdim=True).clamp(min=TINY)
        h = (gw - (gw * chosen).sum(1, keepdim=True) / total) / total * case["scale"]
    else:
        h = gw * case["scale"]
    h = torch.where(ok, h, 0.0)
    H = torch.zeros_like(s).scatter_add_(1, at, h)
    if case["score"] == "softmax":
        out = s * (H if case["renorm"] else H - (h * chosen).sum(1, keepdim=True))
    else:
        out = s * rest * H
    if case["balance"]:
        seq, _ = _seq_of(st["offsets"], case["tokens"])
        a = st["grad_loss"] * st["seq_scale"][seq][:, None] * st["counts"][seq].float()
        d = p * (a - (a * p).sum(1, keepdim=True))
        out = out + (d if rest is None else d * rest)
    return out.to(logits.dtype)


def _by_adapter(ids, L):
    """Slots sorted by adapter into equally long rows of adapters: (slots that have one, their
    adapters, their places in the rows, length of a row)."""
    flat = ids.reshape(-1).long()
    slots = (flat >= 0).nonzero()[:, 0]
    e = flat[slots]
    order = torch.argsort(e, stable=True)
    slots, e = slots[order], e[order]
    count = torch.zeros(L, dtype=torch.long, device="cuda").index_add_(0, e, torch.ones_like(e))
    first = torch.cumsum(count, 0) - count
    return slots, e, torch.arange(e.numel(), device="cuda") - first[e], int(count.max())


def _padded(rows, e, at, L, n):
    out = torch.zeros(L, max(n, 1), rows.shape[1], device="cuda")
    out[e, at] = rows
    return out


def _lora_plain(st, case):
    L, k, N = case["adapters"], case["top_k"], case["nrows"]
    S = st["ids"].numel()
    slots, e, at, n = _by_adapter(st["ids"], L)
    src = slots if case["per_slot"] else slots // k
    u = torch.bmm(_padded(st["x"][src].float(), e, at, L, n), st["a"].float().transpose(1, 2))
    d = torch.bmm(u, st["b"].float().transpose(1, 2))[e, at] * st["scales"][e][:, None]
    out = torch.zeros(S, N, device="cuda") if st["add"] is None else st["add"].float().reshape(S, N)
    return out.index_add(0, slots, d).to(DTYPES[case["out"]]).view(*st["ids"].shape, N)


def _lora_bwd_plain(st, case):
    L, k, K, N = case["adapters"], case["top_k"], case["ncols"], case["nrows"]
    slots, e, at, n = _by_adapter(st["ids"], L)
    src = slots if case["per_slot"] else slots // k
    a, b, scale = st["a"].float(), st["b"].float(), st["scales"][:, None, None]
    x = _padded(st["x"][src].float(), e, at, L, n)
    dy = _padded(st["grad_out"].reshape(-1, N)[slots].float(), e, at, L, n)
    u = torch.bmm(x, a.transpose(1, 2))
    v = torch.bmm(dy, b) * scale
    dx = torch.zeros(st["x"].shape, device="cuda") if st["add"] is None else st["add"].float()
    dx = dx.index_add(0, src, torch.bmm(v, a)[e, at]).to(st["x"].dtype)
    return dx, torch.bmm(v.transpose(1, 2), x), torch.bmm(dy.transpose(1, 2), u) * scale


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "balance":
        return _balance_plain(st["logits"], st["ids"], st["offsets"], case)
    if op == "gate_bwd":
        return _gate_bwd_plain(st, case)
    if op == "comb_bwd":
        w, dy = st["weights"], st["grad_out"].float()[:, None, :]
        dw = torch.where(w != 0, (st["rows"].float() * dy).sum(2), 0.0)
        return (w[:, :, None] * dy).to(st["rows"].dtype), dw
    return _lora_plain(st, case) if op == "lora" else _lora_bwd_plain(st, case)


# ------------------------------------------------------------------- calls
def _calls(st):
    import bit_quantized_moe_quantize_gb300 as ft
    case = st["case"]
    op = case["op"]
    if op == "balance":
        return ft.moe_balance_loss(st["logits"], st["ids"], score=case["score"], seq_offsets=st["offsets"])
    if op == "gate_bwd":
        loss = {n: st[n] for n in ("counts", "seq_scale", "grad_loss")} if case["balance"] else {}
        return ft.moe_gate_backward(st["logits"], st["ids"], st["grad_weights"], score=case["score"],
                                    renormalize=case["renorm"], scale=case["scale"],
                                    seq_offsets=st["offsets"] if case["balance"] else None, **loss)
    if op == "comb_bwd":
        return ft.moe_combine_backward(st["grad_out"], st["rows"], st["weights"])
    if op == "lora":
        return ft.lora_add(st["x"], st["a"], st["b"], st["ids"], scales=st["scales"], add=st["add"],
                           out_dtype=DTYPES[case["out"]])
    return ft.lora_backward(st["grad_out"], st["x"], st["a"], st["b"], st["ids"], scales=st["scales"], add=st["add"])


def run(state):
    return _calls(state) if own else _plain(state)


# -------------------------------------------------------------------- work
def _touched(case):
    """Adapters that a batch is expected to touch."""
    L, slots = case["adapters"], case["tokens"] * case["top_k"]
    return L * (1.0 - (1.0 - 1.0 / L) ** slots) if case["ids"] != "packed" else max(1, min(L - 1, slots))


def work(case):
    op = case["op"]
    size = {n: d.itemsize for n, d in DTYPES.items()}
    T, k = case["tokens"], case["top_k"]
    if op == "balance":
        E, S = case["experts"], max(1, case["seqs"])
        return {"bytes": T * E * size[case["dtype"]] + T * k * 4 + S * E * 4 + S * 8, "flops": 4 * T * E}
    if op == "gate_bwd":
        E, S = case["experts"], max(1, case["seqs"])
        sparse = not case["balance"] and (case["renorm"] or case["score"] == "sigmoid")
        read = T * (k if sparse else E) * size[case["dtype"]]
        return {"bytes": read + T * E * size[case["dtype"]] + T * k * 8 + (S * E * 4 if case["balance"] else 0),
                "flops": 8 * T * E}
    if op == "comb_bwd":
        N = case["cols"]
        return {"bytes": 2 * T * k * N * size[case["dtype"]] + T * N * size[case["out"]] + T * k * 8,
                "flops": 3 * T * k * N}
    L, R, K, N = (case[n] for n in ("adapters", "rank", "ncols", "nrows"))
    slots, rows = T * k, T * k if case["per_slot"] else T
    used = _touched(case) * R * (K + N) * 2
    if op == "lora":
        return {"bytes": rows * K * 2 + slots * (4 + N * size[case["out"]] * (2 if case["add"] else 1)) + used,
                "flops": 2 * slots * R * (K + N)}
    return {"bytes": rows * K * 2 * (3 if case["add"] else 2) + slots * (4 + N * 2) + used + L * R * (K + N) * 4,
            "flops": 2 * slots * R * (3 * K + 2 * N)}


# ------------------------------------------------------------------- exact
def _scores64(logits, score):
    x = logits.double()
    there = x > -math.inf
    if score == "softmax":
        p = torch.softmax(torch.where(there, x, -math.inf), 1)
        p = torch.where(there, p, 0.0)          # a row of padding is NaN in a softmax
        return p, p, 1.0, there
    s = torch.where(there, torch.sigmoid(x), 0.0)
    return s, s / s.sum(1, keepdim=True).clamp(min=TINY), torch.sigmoid(-x), there


def _rows64(offsets, T):
    cuts = [0, T] if offsets is None else offsets.tolist()
    return list(zip(cuts[:-1], cuts[1:]))


def _balance64(st, case):
    E, k = case["experts"], case["top_k"]
    _, p, _, there = _scores64(st["logits"], case["score"])
    spans = _rows64(st["offsets"], case["tokens"])
    scale = torch.zeros(len(spans), dtype=torch.float64, device="cuda")
    full = 0
    loss = 0.0
    for i, (lo, hi) in enumerate(spans):
        n = int(there[lo:hi].any(1).sum()) if hi > lo else 0
        if n:
            mine = st["ids"][lo:hi]
            f = torch.bincount(mine[mine >= 0].long(), minlength=E).double() * E / (k * n)
            loss += float((f * p[lo:hi].sum(0) / n).sum())
            scale[i] = E / (k * n * n)
            full += 1
    return torch.tensor(loss / max(1, full), dtype=torch.float64, device="cuda"), None, scale / max(1, full)


def _gate_bwd64(st, case):
    """By differentiation: the weights and the loss as functions of the logits, in 64 bits."""
    ids, E = st["ids"], case["experts"]
    x = st["logits"].double()
    there = x > -math.inf
    x = torch.where(there, x, 0.0).requires_grad_()
    if case["score"] == "softmax":
        lift = torch.where(there, x, -1e4)
        s = torch.softmax(lift, 1) * there
        p = s
    else:
        s = torch.sigmoid(x) * there
        p = s / s.sum(1, keepdim=True).clamp(min=TINY)
    ok = ids >= 0
    w = s.gather(1, ids.clamp(min=0).long()) * ok
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=TINY)
    total = (w * case["scale"] * torch.where(ok, st["grad_weights"], 0.0)).sum()
    if case["balance"]:
        for i, (lo, hi) in enumerate(_rows64(st["offsets"], case["tokens"])):
            P = p[lo:hi].sum(0)
            total = total + st["grad_loss"].double() * st["seq_scale"][i].double() * (st["counts"][i] * P).sum()
    return torch.autograd.grad(total, x)[0] * there


def _lora64(st, case, grad):
    L, k = case["adapters"], case["top_k"]
    flat = st["ids"].reshape(-1)
    x = st["x"].double()
    rows = x if case["per_slot"] else x.repeat_interleave(k, 0)
    if not grad:
        N = case["nrows"]
        out = torch.zeros(flat.numel(), N, dtype=torch.float64, device="cuda")
        if st["add"] is not None:
            out += st["add"].double().view_as(out)
        for e in range(L):
            mine = (flat == e).nonzero()[:, 0]
            out[mine] += (rows[mine] @ st["a"][e].double().t()) @ st["b"][e].double().t() * st["scales"][e].double()
        return out.view(*st["ids"].shape, N)
    dy = st["grad_out"].double().reshape(flat.numel(), -1)
    da, db = torch.zeros(st["a"].shape, dtype=torch.float64, device="cuda"), torch.zeros(
        st["b"].shape, dtype=torch.float64, device="cuda")
    dr = torch.zeros_like(rows)
    for e in range(L):
        mine = (flat == e).nonzero()[:, 0]
        a, b, c = st["a"][e].double(), st["b"][e].double(), st["scales"][e].double()
        v = dy[mine] @ b * c
        dr[mine] = v @ a
        da[e] = v.t() @ rows[mine]
        db[e] = dy[mine].t() @ (rows[mine] @ a.t()) * c
    dx = dr if case["per_slot"] else dr.view(x.shape[0], k, -1).sum(1)
    return dx if st["add"] is None else dx + st["add"].double(), da, db


def exact(case, seed):
    if work(case)["flops"] > 2e12:
        return None
    st = prepare(case, seed)
    op = case["op"]
    if op == "balance":
        return _balance64(st, case)
    if op == "gate_bwd":
        return _gate_bwd64(st, case)
    if op == "comb_bwd":
        w, dy = st["weights"].double(), st["grad_out"].double()
        dw = torch.einsum("tn,tkn->tk", dy, st["rows"].double())
        return w[:, :, None] * dy[:, None, :], torch.where(w != 0, dw, 0.0)
    return _lora64(st, case, op == "lora_bwd")
