"""The FP8 expert-layer operators against plain 64-bit forms (fp8_ref.py)."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import fp8_ref as R  # noqa: E402


@pytest.fixture(scope="module")
def ft():
    import bit_quantized_moe_quantize_gb300 as ft
    from bit_quantized_moe_quantize_gb300 import build
    build.build()
    ft.load()
    ft.read_device_error()
    yield ft
    assert ft.read_device_error() == 0


def inside(got, want, bound, what=""):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((err - bound).max()):.3e}"


# ------------------------------------------------------------------- gate
GATES = [
    dict(T=1, E=8, k=2), dict(T=3, E=1, k=1), dict(T=257, E=5, k=5), dict(T=64, E=128, k=8),
    dict(T=100, E=60, k=4, score="sigmoid"), dict(T=33, E=160, k=6, score="softmax", bias=True),
    dict(T=129, E=256, k=8, score="sigmoid", bias=True, G=8, TG=4, GT=2, scale=2.5),
    dict(T=50, E=72, k=3, G=8, TG=2, GT=1), dict(T=17, E=64, k=6, score="sigmoid", G=32, TG=5, GT=2),
    dict(T=9, E=4096, k=40, score="softmax", bias=True), dict(T=5, E=4096, k=1, G=64, TG=64, GT=2),
    dict(T=1000, E=512, k=9, renorm=False), dict(T=40, E=33, k=33, score="sigmoid", scale=0.5, renorm=False),
    dict(T=6, E=48, k=48), dict(T=31, E=1024, k=8), dict(T=31, E=1025, k=8, score="sigmoid", bias=True),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("c", GATES)
@pytest.mark.parametrize("mask", [0.0, 0.3])
def test_gate(ft, c, dtype, mask):
    T, E, k = c["T"], c["E"], c["k"]
    score, scale, renorm = c.get("score", "softmax"), c.get("scale", 1.0), c.get("renorm", True)
    G, TG, GT = c.get("G", 1), c.get("TG", 1), c.get("GT", 1)
    g = R.gen(T * 7919 + E)
    wide = torch.randn(T, E + 5, generator=g, device="cuda").to(dtype)
    logits = wide[:, :E]
    if mask:
        gone = torch.rand(T, E, generator=g, device="cuda") < mask
        gone[T // 2] = True
        kind = torch.where(torch.rand(T, E, generator=g, device="cuda") < 0.5, -math.inf, math.nan).to(dtype)
        logits.copy_(torch.where(gone, kind, logits))
    bias = torch.round(torch.randn(E, generator=g, device="cuda") * 8) / 64 if c.get("bias") else None
    ids, w = ft.moe_gate(logits, k, score=score, bias=bias, n_groups=G, topk_groups=TG, group_top=GT,
                         renormalize=renorm, scale=scale)
    want, ww, sure = R.gate(logits, k, score, bias, G, TG, GT, renorm, scale)
    assert sure.float().mean() > 0.5
    assert torch.equal(ids[sure].long(), want[sure])
    # s: exp within 2 ulp of an argument off by half an ulp (|l| < 8: 2^-21 of it), its sum, a
    # quotient; the weights: their sum of k, a quotient, a product: 64 roundings cover them
    inside(w[sure], ww[sure], 64 * R.U32 * ww[sure].abs() + 1e-30, "weights")
    assert ((ids >= 0) | (w == 0)).all()
    if mask:
        assert (ids[T // 2] == -1).all() and (w[T // 2] == 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gate_ties_and_limits(ft, dtype):
    """Equal keys go to the lowest index; lowest values, infinities and zeros of both signs order as numbers."""
    low = torch.finfo(dtype).min
    inf = math.inf
    rows = [[1, 1, 1, 1, 1, 1, 1, 1], [0.0, -0.0, 0.0, -0.0, 1, -1, 1, -1], [low] * 8,
            [low, -inf, low, -inf, low, 0, -inf, low], [inf, 1, inf, 2, 0, 0, 0, 0], [-inf] * 7 + [low],
            [math.nan, 3, math.nan, 3, 1, 2, math.nan, math.nan], [-inf] * 8]
    want = [[0, 1, 2, 3], [4, 6, 0, 1], [0, 1, 2, 3], [5, 0, 2, 4], [0, 2, 3, 1], [7, -1, -1, -1], [1, 3, 5, 4],
            [-1, -1, -1, -1]]
    logits = torch.tensor(rows, dtype=torch.float32).to(dtype).cuda()
    for score in ("softmax", "sigmoid"):
        ids, w = ft.moe_gate(logits, 4, score=score, renormalize=False)
        assert ids.tolist() == want, score
        assert torch.isfinite(w).all()
    ids, w = ft.moe_gate(logits, 4)
    assert torch.allclose(w[0].cpu(), torch.full((4,), 0.25))
    assert w[4].tolist() == [0.5, 0.5, 0.0, 0.0]
    assert w[5].tolist() == [1.0, 0.0, 0.0, 0.0]


def test_gate_masked_groups(ft):
    """A group with no expert left is not chosen before one that has some; one left counts alone."""
    inf = math.inf
    logits = torch.tensor([[-inf, -inf, 0.0, -inf, 1.0, 1.0], [-inf, -inf, -inf, -inf, -inf, 2.0]], device="cuda")
    ids, _ = ft.moe_gate(logits, 3, score="sigmoid", n_groups=3, topk_groups=2, group_top=2)
    assert ids.tolist() == [[4, 5, 2], [5, -1, -1]]


# -------------------------------------------------------------- quantizer
SHAPES = [(1, 16), (3, 128), (5, 144), (2, 2048), (7, 2000), (130, 1408), (1, 65536)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize(ft, shape, dtype):
    """Codes and scales are those of the formula in IEEE fp32, bit for bit."""
    rows, K = shape
    x = R.rows(R.gen(rows * 31 + K), rows, K, dtype)
    x[rows // 2, : min(K, 128)] = 0
    q, s = ft.quantize_fp8(x)
    xc = x.float().cpu()
    nb = R.blocks(K)
    b = torch.nn.functional.pad(xc, (0, nb * 128 - K)).view(rows, nb, 128)
    want_s = b.abs().amax(2) / torch.tensor(448.0)          # fp32 on the host: IEEE
    assert torch.equal(s.cpu(), want_s)
    d = torch.where(want_s[:, :, None] > 0, b / want_s[:, :, None], 0.0)
    want, _ = R.nearest_e4m3(d.double())
    assert torch.equal(R.decode(q).cpu(), want.view(rows, -1)[:, :K])


def test_quantize_limits(ft):
    """Tiny, largest and non-finite values."""
    x = torch.zeros(6, 128, device="cuda")
    x[0, :] = 2.0 ** -149          # amax / 448 underflows to 0: codes 0
    x[1, 3] = 2.0 ** -126
    x[2, :2] = torch.tensor([torch.finfo(torch.float32).max, -torch.finfo(torch.float32).max])
    x[3, 5] = math.inf
    x[4, 7] = math.nan
    q, s = ft.quantize_fp8(x)
    v = R.decode(q)
    assert float(s[0, 0]) == 0 and (v[0] == 0).all()
    assert float(v[1, 3]) == 448 and int((v[1] != 0).sum()) == 1
    assert v[2, :2].tolist() == [448, -448]
    assert math.isinf(float(s[3, 0])) and math.isnan(float(s[4, 0]))
    assert torch.isnan((v[3, 5] * s[3, 0].double())) and torch.isnan(v[4] * s[4, 0].double()).all()
    assert float(s[5, 0]) == 0 and (v[5] == 0).all()


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", SHAPES)
def test_act_mul_quantize(ft, shape, dtype, kind):
    rows, I = shape
    h = (torch.randn(rows, 2 * I, generator=R.gen(rows + I), device="cuda") * 3).to(dtype)
    q, s = ft.act_mul_quantize_fp8(h, kind)
    a = R.act_mul(h, kind)
    nb = R.blocks(I)
    amax = torch.nn.functional.pad(a.abs(), (0, nb * 128 - I)).view(rows, nb, 128).amax(2)
    # the activation in fp32: |z| < 2^8 off by four roundings moves exp(-z) by 2^-14, six more beside it
    rel = 2.0 ** -13
    inside(s, amax / 448, amax / 448 * rel, "scales")
    scale = s.double().repeat_interleave(128, 1)[:, :I]
    t = torch.where(scale > 0, a / scale, 0.0)
    _, step = R.nearest_e4m3(t.abs().clamp(max=448))
    inside(R.decode(q), t, step * 0.5 * (1 + rel) + t.abs() * rel, "codes")


# ---------------------------------------------------------------- product
PRODUCTS = [
    # E, k, N, K, T, out, unrouted
    (1, 1, 1, 16, 1, torch.float32, 0.0), (4, 2, 128, 128, 3, torch.float32, 0.0),
    (8, 2, 130, 144, 5, torch.bfloat16, 0.2), (3, 3, 257, 272, 40, torch.float32, 0.1),
    (128, 8, 96, 256, 1, torch.float32, 0.0), (60, 4, 333, 400, 77, torch.bfloat16, 0.05),
    (5, 2, 511, 1040, 301, torch.float32, 0.0), (2, 1, 384, 2000, 1031, torch.float32, 0.01),
    (16, 4, 768, 512, 700, torch.bfloat16, 0.0), (4, 1, 1408, 2816, 900, torch.bfloat16, 0.0),
    (7, 2, 129, 128, 2048, torch.float32, 0.3), (3, 2, 255, 48, 513, torch.bfloat16, 0.0),
    (64, 6, 64, 1152, 33, torch.float32, 1.0),
]


@pytest.mark.parametrize("per_slot", [False, True])
@pytest.mark.parametrize("c", PRODUCTS)
def test_product(ft, c, per_slot):
    E, k, N, K, T, dt, none = c
    g = R.gen(E * 101 + N + K)
    w, ws = R.weights(g, E, N, K)
    q, s = R.codes(g, T * k if per_slot else T, K)
    ids = R.ids(g, T, E, k, none, pop=torch.linspace(0, 2, E, device="cuda"))
    fn = ft.moe_fp8_fp8_slots if per_slot else ft.moe_fp8_fp8
    guard = 1031
    buf = torch.full((T * k * N + 2 * guard,), 12345.0, dtype=dt, device="cuda")
    out = buf[guard:-guard].view(T, k, N)
    fn(w, ws, q, s, ids, out=out)
    want, bound = R.product(w, ws, q, s, ids, per_slot, dt)
    inside(out, want, bound)
    assert (out[ids < 0] == 0).all()
    assert (buf[:guard] == buf[0]).all() and (buf[-guard:] == buf[0]).all() and float(buf[0]) > 12000


@pytest.mark.parametrize("c", [(1, 17, 48), (3, 128, 128), (37, 1000, 2000), (300, 257, 512), (1025, 640, 1152)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_dense(ft, c, dt):
    M, N, K = c
    g = R.gen(M + N + K)
    w, ws = R.weights(g, 1, N, K)
    q, s = R.codes(g, M, K)
    out = ft.matmul_fp8_fp8(w[0], ws[0], q, s, out_dtype=dt)
    want, bound = R.product(w, ws, q, s, torch.zeros(M, 1, dtype=torch.int32, device="cuda"), False, dt)
    inside(out, want[:, 0], bound[:, 0])


@pytest.mark.parametrize("T", [1, 2, 17, 64, 300, 1300])
def test_product_one_expert_takes_all(ft, T):
    """Every slot on one expert of many, the last one."""
    E, N, K = 9, 300, 640
    g = R.gen(T)
    w, ws = R.weights(g, E, N, K)
    q, s = R.codes(g, T, K)
    ids = torch.full((T, 1), E - 1, dtype=torch.int32, device="cuda")
    out = ft.moe_fp8_fp8(w, ws, q, s, ids)
    want, bound = R.product(w, ws, q, s, ids, False, torch.float32)
    inside(out, want, bound)


def test_product_nan_stays_in_its_row(ft):
    """A NaN code or an infinite scale spoils its own slot (or weight row) only."""
    E, N, K, T = 4, 200, 384, 50
    g = R.gen(5)
    w, ws = R.weights(g, E, N, K)
    q, s = R.codes(g, T, K)
    ids = R.ids(g, T, E, 2)
    clean = ft.moe_fp8_fp8(w, ws, q, s, ids)
    qb = q.clone()
    qb.view(torch.uint8)[7, 100] = 0x7F
    out = ft.moe_fp8_fp8(w, ws, qb, s, ids)
    assert torch.isnan(out[7]).all()
    keep = torch.arange(T, device="cuda") != 7
    assert torch.equal(out[keep], clean[keep])
    wb = w.clone()
    wb.view(torch.uint8)[2, 11, 30] = 0xFF
    out = ft.moe_fp8_fp8(wb, ws, q, s, ids)
    hit = (ids == 2)
    assert torch.isnan(out[hit][:, 11]).all()
    out[:, :, 11], clean[:, :, 11] = 0, 0
    assert torch.equal(out, clean)


def test_product_bad_ids(ft):
    E, N, K, T = 4, 96, 128, 6
    g = R.gen(6)
    w, ws = R.weights(g, E, N, K)
    q, s = R.codes(g, T, K)
    ids = R.ids(g, T, E, 2)
    ids[2, 1], ids[4, 0], ids[5] = E, -2, -1
    out = ft.moe_fp8_fp8(w, ws, q, s, ids)
    want, bound = R.product(w, ws, q, s, ids, False, torch.float32)
    inside(out, want, bound)
    assert (out[2, 1] == 0).all() and (out[4, 0] == 0).all() and (out[5] == 0).all()
    assert ft.read_device_error() == ft.FT_DEVERR_BAD_EXPERT_ID
    ids[2, 1], ids[4, 0] = -1, -1
    ft.moe_fp8_fp8(w, ws, q, s, ids)
    assert ft.read_device_error() == 0


def test_product_past_32_bit_offsets(ft):
    """Weights of more than 2^32 bytes, and more than 2^32 activation bytes."""
    E, N, K = 18, 14336, 17408
    g = R.gen(8)
    w = torch.randint(0, 120, (E, N, K), dtype=torch.uint8, generator=g, device="cuda")
    ws = torch.rand(E, R.blocks(N), R.blocks(K), generator=g, device="cuda") * 1e-4
    q, s = R.codes(g, 2, K)
    ids = torch.tensor([[E - 1], [0]], dtype=torch.int32, device="cuda")
    out = ft.moe_fp8_fp8(w, ws, q, s, ids)
    for t, e in ((0, E - 1), (1, 0)):
        sel = slice(N - 200, N)
        x = R.decode(q[t:t + 1]) * R.expand_rows(s[t:t + 1], K)
        m = R.decode(w[e, sel].contiguous()) * R.expand_matrix(ws[e], N, K)[sel]
        inside(out[t, :, sel], x @ m.t(), (132 + R.blocks(K)) * 2 * R.U32 * (x.abs() @ m.abs().t()))
    del w, out
    M, N, K = 70001, 24, 65536
    w, ws = R.weights(g, 1, N, K)
    q = torch.randint(0, 120, (M, K), dtype=torch.uint8, generator=g, device="cuda")
    s = torch.rand(M, R.blocks(K), generator=g, device="cuda") * 1e-3
    out = ft.matmul_fp8_fp8(w[0], ws[0], q, s)
    pick = torch.tensor([0, 1, 40000, M - 2, M - 1], device="cuda")
    want, bound = R.product(w, ws, q[pick], s[pick], torch.zeros(5, 1, dtype=torch.int32, device="cuda"), False,
                            torch.float32)
    inside(out[pick], want[:, 0], bound[:, 0])


# ---------------------------------------------------------------- combine
@pytest.mark.parametrize("c", [(1, 1, 1), (3, 8, 2048), (7, 2, 129), (300, 6, 2816), (65, 9, 100), (2, 33, 17)])
@pytest.mark.parametrize("ri", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ro", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("add", [False, True])
def test_combine(ft, c, ri, ro, add):
    T, k, N = c
    g = R.gen(T + k + N)
    rows = torch.randn(T, k, N, generator=g, device="cuda").to(ri)
    w = torch.rand(T, k, generator=g, device="cuda")
    w = torch.where(torch.rand(T, k, generator=g, device="cuda") < 0.3, 0.0, w)
    rows[w == 0] = math.nan                      # rows that no expert wrote are not read
    a = torch.randn(T, N, generator=g, device="cuda").to(ro) if add else None
    y = ft.moe_combine(rows, w, add=a, out_dtype=ro)
    terms = torch.where(w[:, :, None] > 0, rows.double() * w.double()[:, :, None], 0.0)
    want, mag = terms.sum(1), terms.abs().sum(1)
    if add:
        want, mag = want + a.double(), mag + a.double().abs()
    u = R.U[ro]
    inside(y, want, (k + 2) * R.U32 * mag + want.abs() * u * 1.01 + (2.0 ** -25 if ro == torch.float16 else 0))


def test_combine_unaligned(ft):
    """Rows and outputs that start at any element."""
    T, k, N = 5, 3, 64
    g = R.gen(2)
    for off in (1, 2, 4):
        rows = torch.randn(T * k * N + off, generator=g, device="cuda").to(torch.bfloat16)[off:].view(T, k, N)
        w = torch.rand(T, k, generator=g, device="cuda")
        out = torch.empty(T * N + off, dtype=torch.bfloat16, device="cuda")[off:].view(T, N)
        y = ft.moe_combine(rows, w, out=out)
        assert torch.equal(y, ft.moe_combine(rows.clone(), w))


# ------------------------------------------------------------------ layer
LAYERS = [
    dict(T=1, E=8, k=2, H=256, I=128, dt=torch.bfloat16), dict(T=5, E=16, k=4, H=272, I=144, dt=torch.float16, kind=1),
    dict(T=1, E=128, k=8, H=512, I=256, dt=torch.bfloat16, score="sigmoid", bias=True),
    dict(T=70, E=32, k=6, H=400, I=208, dt=torch.bfloat16, score="sigmoid", bias=True, G=4, TG=2, GT=2, mask=0.2),
    dict(T=600, E=8, k=2, H=640, I=400, dt=torch.bfloat16), dict(T=1100, E=4, k=2, H=1024, I=512, dt=torch.float16),
    dict(T=300, E=64, k=8, H=2048, I=768, dt=torch.bfloat16, scale=2.5),
    dict(T=33, E=4, k=4, H=1040, I=16, dt=torch.bfloat16, renorm=False),
]


def layer_inputs(c):
    g = R.gen(c["T"] * 13 + c["E"])
    E, H, I, T = c["E"], c["H"], c["I"], c["T"]
    x = R.rows(g, T, H, c["dt"])
    logits = torch.randn(T, E, generator=g, device="cuda")
    if c.get("mask"):
        logits = torch.where(torch.rand(T, E, generator=g, device="cuda") < c["mask"], -math.inf, logits)
        logits[0] = -math.inf
    bias = torch.round(torch.randn(E, generator=g, device="cuda") * 8) / 64 if c.get("bias") else None
    w13, s13 = R.weights(g, E, 2 * I, H)
    w2, s2 = R.weights(g, E, H, I)
    opt = dict(score=c.get("score", "softmax"), bias=bias, n_groups=c.get("G", 1), topk_groups=c.get("TG", 1),
               group_top=c.get("GT", 1), renormalize=c.get("renorm", True), scale=c.get("scale", 1.0))
    return x, logits, w13, s13, w2, s2, opt


@pytest.mark.parametrize("c", LAYERS)
def test_layer(ft, c):
    """Against the 64-bit form on the quantizer's own codes (which test_quantize pins).

    Off by the bf16 rounding of each expert row and of y (at most 2^-8 each, 2^-9.2 rms, independent), and by the
    codes that fp32 rounding turns (one in some thousand, by at most an eighth): 2^-7 of the
    norm covers them."""
    x, logits, w13, s13, w2, s2, opt = layer_inputs(c)
    k, kind = c["k"], c.get("kind", 0)
    y, ids, w = ft.moe_layer_fp8(x, logits, w13, s13, w2, s2, k, kind, **opt)
    gi, gw = ft.moe_gate(logits, k, **opt)
    assert torch.equal(ids, gi) and torch.equal(w, gw)
    q, s = ft.quantize_fp8(x)
    h, _ = R.product(w13, s13, q, s, ids, False, torch.float32)
    a = R.act_mul(h.view(-1, h.shape[2]), kind)
    nb = R.blocks(c["I"])
    sc = torch.nn.functional.pad(a.abs(), (0, nb * 128 - c["I"])).view(a.shape[0], nb, 128).amax(2) / 448
    t = a / torch.where(sc > 0, sc, 1.0).repeat_interleave(128, 1)[:, :c["I"]]
    m = R.nearest_e4m3(t)[0] * sc.repeat_interleave(128, 1)[:, :c["I"]]
    flat = ids.reshape(-1)
    rows = torch.zeros(flat.numel(), c["H"], dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        sel = (flat == e).nonzero()[:, 0]
        rows[sel] = m[sel] @ (R.decode(w2[e]) * R.expand_matrix(s2[e], c["H"], c["I"])).t()
    want = (rows.view(*ids.shape, -1) * w.double()[:, :, None]).sum(1)
    assert y.dtype == c["dt"] and torch.isfinite(y).all()
    rel = float((y.double() - want).norm() / want.norm())
    assert rel < 2.0 ** -7, rel
    if c.get("mask"):
        assert (y[0] == 0).all() and (ids[0] == -1).all()


def test_layer_on_other_streams_and_in_a_graph(ft):
    """Calls on two streams at once, each with its own workspace, and a captured call replayed."""
    c = dict(T=40, E=16, k=4, H=512, I=256, dt=torch.bfloat16)
    x, logits, w13, s13, w2, s2, opt = layer_inputs(c)
    x2 = (x.float() * 0.5).to(x.dtype).flip(0).contiguous()
    want = ft.moe_layer_fp8(x, logits, w13, s13, w2, s2, 4, **opt)[0].clone()
    want2 = ft.moe_layer_fp8(x2, logits, w13, s13, w2, s2, 4, **opt)[0].clone()
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(10):
        with torch.cuda.stream(sa):
            got.append((ft.moe_layer_fp8(x, logits, w13, s13, w2, s2, 4, **opt)[0], want))
        with torch.cuda.stream(sb):
            got.append((ft.moe_layer_fp8(x2, logits, w13, s13, w2, s2, 4, **opt)[0], want2))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in got)
    static = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ft.moe_layer_fp8(static, logits, w13, s13, w2, s2, 4, **opt)[0]
    for src, ref in ((x, want), (x2, want2), (x, want)):
        static.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)


def test_same_bits_every_time(ft):
    c = dict(T=333, E=8, k=2, H=640, I=384, dt=torch.bfloat16)
    x, logits, w13, s13, w2, s2, opt = layer_inputs(c)
    first = ft.moe_layer_fp8(x, logits, w13, s13, w2, s2, 2, **opt)[0].clone()
    for _ in range(5):
        assert torch.equal(ft.moe_layer_fp8(x, logits, w13, s13, w2, s2, 2, **opt)[0], first)


def test_empty(ft):
    z = torch.zeros(0, 256, device="cuda", dtype=torch.bfloat16)
    q, s = ft.quantize_fp8(z)
    assert q.shape == (0, 256) and s.shape == (0, 2)
    w, ws = R.weights(R.gen(1), 4, 64, 256)
    ids, wt = ft.moe_gate(torch.zeros(0, 4, device="cuda"), 2)
    assert ft.moe_fp8_fp8(w, ws, q, s, ids).shape == (0, 2, 64)
    assert ft.moe_combine(torch.zeros(0, 2, 64, device="cuda"), wt).shape == (0, 64)


def test_binding_refuses(ft):
    g = R.gen(3)
    w, ws = R.weights(g, 4, 64, 256)
    q, s = R.codes(g, 6, 256)
    ids = R.ids(g, 6, 4, 2)
    with pytest.raises(ValueError):
        ft.moe_fp8_fp8(w, ws[:, :, :1].contiguous(), q, s, ids)          # scales of another shape
    with pytest.raises(ValueError):
        ft.moe_fp8_fp8(w.transpose(1, 2), ws, q, s, ids)                 # not contiguous
    with pytest.raises(TypeError):
        ft.moe_fp8_fp8(w, ws, q, s, ids.long())
    with pytest.raises(TypeError):
        ft.moe_fp8_fp8(w.float(), ws, q, s, ids)
    with pytest.raises(TypeError):
        ft.moe_fp8_fp8(w, ws, q, s, ids, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        ft.moe_fp8_fp8_slots(w, ws, q, s, ids)                           # rows per token, not per slot
    with pytest.raises(ft.FtError):
        ft.quantize_fp8(torch.zeros(2, 40, device="cuda"))               # not a multiple of 16 columns
    with pytest.raises(TypeError):
        ft.quantize_fp8(torch.zeros(2, 64, device="cuda", dtype=torch.float64))
    with pytest.raises(TypeError):
        ft.quantize_fp8(torch.zeros(2, 64))
    with pytest.raises(ValueError):
        ft.moe_gate(torch.zeros(2, 8, device="cuda"), 2, score="linear")
    with pytest.raises(ValueError):
        ft.moe_gate(torch.zeros(8, 2, device="cuda").t(), 2)
    with pytest.raises(ft.FtError):
        ft.moe_gate(torch.zeros(2, 8, device="cuda"), 3, n_groups=4, topk_groups=1)
    with pytest.raises(ValueError):
        ft.moe_combine(torch.zeros(2, 3, 8, device="cuda"), torch.zeros(2, 2, device="cuda"))


# ------------------------------------------------------- between the variants
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("E", [7, 16, 17, 32, 33, 128, 129, 256, 257, 511, 512, 513])
@pytest.mark.parametrize("k", [1, 7, 8, 9])
def test_gate_many_ties(ft, E, k, dtype):
    """Logits of a few values, masked ones among them: the choice and its order are exact."""
    if k > E:
        return
    T = 211
    g = R.gen(E * 16 + k)
    logits = torch.randint(-3, 4, (T, E), generator=g, device="cuda").to(dtype) / 2
    logits = torch.where(torch.rand(T, E, generator=g, device="cuda") < 0.1, -math.inf, logits)
    logits[3, 1:] = -math.inf
    for score in ("softmax", "sigmoid"):
        ids, w = ft.moe_gate(logits, k, score=score)
        want, ww, _ = R.gate(logits, k, score, None, 1, 1, 1, True, 1.0)
        assert torch.equal(ids.long(), want)
        inside(w, ww, 64 * R.U32 * ww + 1e-30, "weights")


@pytest.mark.parametrize("off", [8, 16, 24])
def test_quantize_unaligned(ft, off):
    """Codes at any 8 bytes, scales at any 4, rows at any 16."""
    x = R.rows(R.gen(off), 9, 272, torch.bfloat16)
    q, s = ft.quantize_fp8(x)
    xs = torch.empty(9 * 272 + 8, dtype=torch.bfloat16, device="cuda")[8:].view(9, 272).copy_(x)
    qo = torch.empty(9 * 272 + off, dtype=torch.uint8, device="cuda")[off:].view(torch.float8_e4m3fn).view(9, 272)
    so = torch.empty(9 * 3 + 1, device="cuda")[1:].view(9, 3)
    ft.quantize_fp8(xs, qo, so)
    assert torch.equal(qo.view(torch.uint8), q.view(torch.uint8)) and torch.equal(so, s)


def routed(ft, E, k, N, K, T, dt, none=0.0, pop=None, per_slot=False):
    g = R.gen(E + 3 * N + 5 * K + 7 * T)
    w, ws = R.weights(g, E, N, K)
    q, s = R.codes(g, T * k if per_slot else T, K)
    ids = R.ids(g, T, E, k, none, pop)
    out = (ft.moe_fp8_fp8_slots if per_slot else ft.moe_fp8_fp8)(w, ws, q, s, ids, out_dtype=dt)
    want, bound = R.product(w, ws, q, s, ids, per_slot, dt)
    inside(out, want, bound)
    assert (out[ids < 0] == 0).all()


@pytest.mark.parametrize("per_slot", [False, True])
@pytest.mark.parametrize("T", [5, 6, 120, 121, 520, 521])
def test_product_around_the_tile_widths(ft, T, per_slot):
    """40 experts, 4 slots a token: 0.5, 12 and 52 slots per expert, and one token more."""
    routed(ft, 40, 4, 144, 272, T, torch.float32, 0.0, per_slot=per_slot)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("c", [
    # E, k, N, K, T, unrouted, popularity of the last expert over the first
    (128, 8, 130, 144, 150, 0.1, 0.0),      # over 1024 slots, tiles of 16
    (128, 8, 65, 400, 129, 0.0, 9.0),       # the same, most slots on some experts
    (60, 4, 130, 2000, 509, 0.02, 4.0),     # tiles of 32, short last block
    (100, 5, 32, 16, 205, 0.3, 2.0), (1024, 8, 48, 128, 100, 0.1, 1.0), (1023, 3, 33, 144, 900, 0.0, 3.0),
    (1100, 2, 40, 144, 12, 0.0, 0.0),       # more experts than the fast order takes: slots by themselves,
    (1100, 8, 40, 144, 700, 0.1, 2.0),      # tiles of 16
    (1100, 8, 40, 48, 8300, 0.05, 1.0),     # and of 256
    (5, 4, 32, 16, 66000, 0.1, 1.0),        # more slots than it takes
    (3, 3, 33, 32, 20000, 0.0, 0.0),
])
def test_product_orders(ft, c, dt):
    E, k, N, K, T, none, pop = c
    routed(ft, E, k, N, K, T, dt, none, torch.linspace(0, pop, E, device="cuda"))


@pytest.mark.parametrize("T", [3, 60, 700, 2500])
def test_bad_ids_in_every_tile_width(ft, T):
    """Ids that are no expert raise the flag and give zero rows; -1 gives zero rows only."""
    E, k, N, K = 24, 4, 72, 144
    g = R.gen(T)
    w, ws = R.weights(g, E, N, K)
    q, s = R.codes(g, T, K)
    ids = R.ids(g, T, E, k, 0.1)
    ft.moe_fp8_fp8(w, ws, q, s, ids)
    assert ft.read_device_error() == 0
    ids[0, 1], ids[T // 2, 0], ids[T - 1, 3] = E, -2 ** 31, 2 ** 31 - 1
    out = ft.moe_fp8_fp8(w, ws, q, s, ids)
    assert ft.read_device_error() == ft.FT_DEVERR_BAD_EXPERT_ID
    want, bound = R.product(w, ws, q, s, ids, False, torch.float32)
    inside(out, want, bound)
    assert (out[(ids < 0) | (ids >= E)] == 0).all()


@pytest.mark.parametrize("M", [1, 2, 12, 13, 52, 53, 128, 257])
def test_dense_unaligned(ft, M):
    """Scales and outputs that start at any element, around the tile widths."""
    N, K = 130, 400
    g = R.gen(M)
    w, ws = R.weights(g, 1, N, K)
    q, s = R.codes(g, M, K)
    ws1 = torch.empty(ws.numel() + 1, device="cuda")[1:].view(ws.shape[1:]).copy_(ws[0])
    s1 = torch.empty(s.numel() + 3, device="cuda")[3:].view(s.shape).copy_(s)
    for dt in (torch.float32, torch.bfloat16):
        out = torch.empty(M * N + 1, dtype=dt, device="cuda")[1:].view(M, N)
        ft.matmul_fp8_fp8(w[0], ws1, q, s1, out=out)
        want, bound = R.product(w, ws, q, s, torch.zeros(M, 1, dtype=torch.int32, device="cuda"), False, dt)
        inside(out, want[:, 0], bound[:, 0])


MORE_LAYERS = [
    # few tokens: all in three launches; 9 slots a token for 8 warps; short last blocks; masked experts
    dict(T=2, E=64, k=9, H=272, I=144, dt=torch.bfloat16), dict(T=8, E=128, k=8, H=272, I=400, dt=torch.float16, kind=1),
    dict(T=3, E=40, k=4, H=1040, I=16, dt=torch.bfloat16, score="sigmoid", mask=0.9, renorm=False),
    dict(T=1, E=1, k=1, H=16, I=16, dt=torch.bfloat16), dict(T=700, E=2048, k=1, H=48, I=32, dt=torch.bfloat16),
    # the same with larger matrices: separate launches
    dict(T=2, E=8, k=2, H=4096, I=2048, dt=torch.bfloat16),
    # tiles of 16 and 32, over and under 1024 slots
    dict(T=150, E=128, k=8, H=272, I=144, dt=torch.bfloat16, mask=0.3), dict(T=100, E=20, k=4, H=400, I=272, dt=torch.float16, kind=1),
    # tiles of 256: the activation with the first product, and after it
    dict(T=300, E=6, k=3, H=272, I=384, dt=torch.bfloat16, kind=1, mask=0.3),
    dict(T=300, E=6, k=3, H=272, I=208, dt=torch.float16, kind=1, mask=0.3),
    dict(T=8300, E=1100, k=8, H=48, I=128, dt=torch.bfloat16),
]


@pytest.mark.parametrize("c", MORE_LAYERS)
def test_layer_variants(ft, c):
    test_layer(ft, c)


@pytest.mark.parametrize("c", [dict(T=1, E=128, k=8, H=512, I=256, dt=torch.bfloat16),
                               dict(T=600, E=8, k=2, H=640, I=384, dt=torch.bfloat16),
                               dict(T=150, E=128, k=8, H=272, I=144, dt=torch.bfloat16)])
def test_layer_streams_and_graph_of_every_width(ft, c):
    """The same bits from two streams at once, behind other work, and from a captured call."""
    x, logits, w13, s13, w2, s2, opt = layer_inputs(c)
    k = c["k"]
    x2 = (x.float() * 0.5).to(x.dtype)
    lg2 = logits.flip(1).contiguous()
    want = [ft.moe_layer_fp8(a, l, w13, s13, w2, s2, k, **opt)[0].clone() for a, l in ((x, logits), (x2, lg2))]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(20):
        for i, (a, l) in enumerate(((x, logits), (x2, lg2))):
            with torch.cuda.stream(streams[i]):
                y = ft.moe_layer_fp8(a * 1, l + 0, w13, s13, w2, s2, k, **opt)[0]
                got.append((y * 1, want[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in got)
    sx, sl = x.clone(), logits.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ft.moe_layer_fp8(sx, sl, w13, s13, w2, s2, k, **opt)[0] * 1
    for i, (a, l) in enumerate(((x2, lg2), (x, logits))):
        sx.copy_(a)
        sl.copy_(l)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[1 - i])


def test_layer_of_no_tokens(ft):
    c = dict(T=0, E=4, k=2, H=256, I=128, dt=torch.bfloat16)
    x, logits, w13, s13, w2, s2, opt = layer_inputs(c)
    y, ids, w = ft.moe_layer_fp8(x, logits, w13, s13, w2, s2, 2, **opt)
    assert y.shape == (0, 256) and ids.shape == (0, 2) and w.shape == (0, 2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("c", [(64, 4, 2, 1, 8), (64, 2, 1, 2, 9), (128, 8, 3, 2, 8), (256, 8, 4, 2, 8), (256, 16, 5, 1, 6), (256, 2, 2, 2, 12),
                               (512, 4, 2, 2, 8), (512, 32, 7, 2, 8), (32, 2, 1, 1, 4), (160, 2, 1, 2, 6), (384, 8, 3, 2, 8), (1024, 16, 4, 2, 8)])
@pytest.mark.parametrize("bias", [False, True])
def test_gate_groups(ft, c, dtype, bias):
    """Groups of whole lanes and others; masked experts, groups and rows; ties between groups by the lowest."""
    E, G, TG, GT, k = c
    T = 97
    g = R.gen(E + 31 * G + k)
    logits = torch.randint(-4, 5, (T, E), generator=g, device="cuda").to(dtype) / 2
    logits = torch.where(torch.rand(T, E, generator=g, device="cuda") < 0.2, -math.inf, logits)
    logits.view(T, G, -1)[torch.rand(T, G, generator=g, device="cuda") < 0.3] = -math.inf
    logits[5] = -math.inf
    b = torch.randint(0, 3, (E,), generator=g, device="cuda").float() / 4 if bias else None
    ids, w = ft.moe_gate(logits, k, score="sigmoid", bias=b, n_groups=G, topk_groups=TG, group_top=GT, scale=2.5)
    want, ww, sure = R.gate(logits, k, "sigmoid", b, G, TG, GT, True, 2.5)
    assert sure.float().mean() > 0.5
    assert torch.equal(ids[sure].long(), want[sure])
    inside(w[sure], ww[sure], 64 * R.U32 * ww[sure].abs() + 1e-30, "weights")
    assert (ids[5] == -1).all()
