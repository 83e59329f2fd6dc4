"""The FP8 layer's codes between its products are the quantizer's, whatever the batch and n_inter."""

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


def inputs(T, E, k, H, I, dt=torch.bfloat16):
    g = R.gen(T + E + H + I)
    x = R.rows(g, T, H, dt)
    logits = torch.randn(T, E, generator=g, device="cuda")
    return x, logits, *R.weights(g, E, 2 * I, H), *R.weights(g, E, H, I)


# one slot each, tiles of 16, 32 and 256 with and without whole blocks of n_inter; a few tokens
BATCHES = [(1, 16, 2, 272, 144), (3, 40, 4, 1040, 528), (20, 8, 2, 272, 128), (100, 8, 2, 272, 256), (300, 6, 3, 272, 208),
           (300, 6, 3, 272, 256), (700, 4, 2, 400, 384)]


def norm_apart(ft, c, kind, x, logits, w13, s13, w2, s2):
    """The layer's distance from the 64-bit form on the quantizer's own codes of x, over the form's norm."""
    T, E, k, H, I = c
    y, ids, w = ft.moe_layer_fp8(x, logits, w13, s13, w2, s2, k, kind)
    q, s = ft.quantize_fp8(x)
    h, _ = R.product(w13, s13, q, s, ids, False, torch.float32)
    a = R.act_mul(h.view(-1, 2 * I), kind)
    nb = R.blocks(I)
    sc = torch.nn.functional.pad(a.abs(), (0, nb * 128 - I)).view(-1, nb, 128).amax(2) / 448
    sc = sc.repeat_interleave(128, 1)[:, :I]
    m = R.nearest_e4m3(a / torch.where(sc > 0, sc, 1.0))[0] * sc
    flat = ids.reshape(-1)
    rows = torch.zeros(flat.numel(), H, dtype=torch.float64, device="cuda")
    for e in range(E):
        sel = (flat == e).nonzero()[:, 0]
        rows[sel] = m[sel] @ (R.decode(w2[e]) * R.expand_matrix(s2[e], H, I)).t()
    want = (rows.view(T, k, H) * w.double()[:, :, None]).sum(1)
    assert torch.isfinite(y).all()
    return float((y.double() - want).norm() / want.norm())


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("down", [-46, -55])
@pytest.mark.parametrize("c", BATCHES)
def test_layer_of_tiny_values(ft, c, down, kind):
    """Gate and up 2^down of their usual size, so that act(gate) * up is about 2^(2 down - 1) of its
    own (1e-28, 1e-34), which the second matrix's scales undo.  A block's scale is then still a normal
    fp32 number, so the layer is as near to the 64-bit form as it is at the usual size (2^-7 of the norm: two
    bf16 roundings, and the codes that fp32 rounding turns)."""
    x, logits, w13, s13, w2, s2 = inputs(*c)
    assert norm_apart(ft, c, kind, x, logits, w13, s13 * 2.0 ** down, w2, s2 * 2.0 ** (-2 * down)) < 2.0 ** -7


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("down", [-60, -90, -102])
@pytest.mark.parametrize("c", [c for c in BATCHES if c[4] % 128 == 0])
def test_layer_is_the_same_at_every_size(ft, c, down, kind):
    """Up rows 2^down as large and the second matrix 2^-down: products by powers of 2 are exact while all that a
    code depends on stays normal in fp32 (the largest values are about 1, what rounds to the smallest code
    2^-19 of them, 2^-121 here at the least), so y is the same bit for bit."""
    T, E, k, H, I = c
    x, logits, w13, s13, w2, s2 = inputs(*c)
    want = ft.moe_layer_fp8(x, logits, w13, s13, w2, s2, k, kind)[0]
    low = s13.clone()
    low[:, I // 128:] *= 2.0 ** down
    assert torch.equal(ft.moe_layer_fp8(x, logits, w13, low, w2, s2 * 2.0 ** -down, k, kind)[0], want)
    assert float(want.abs().max()) > 0


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("c", BATCHES)
def test_layer_nan_stays_in_its_token(ft, c, bad):
    """A value of x that is no number spoils its own token's row and no other, in every form of the layer."""
    T, E, k, H, I = c
    x, logits, w13, s13, w2, s2 = inputs(*c)
    clean = ft.moe_layer_fp8(x, logits, w13, s13, w2, s2, k)[0]
    xb = x.clone()
    xb[T // 2, H - 3] = bad
    y = ft.moe_layer_fp8(xb, logits, w13, s13, w2, s2, k)[0]
    assert torch.isnan(y[T // 2]).all()
    keep = torch.arange(T, device="cuda") != T // 2
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("T", [2, 20, 100, 400])
def test_product_nan_stays_in_its_row(ft, T):
    """A NaN code spoils its own slots, or its own weight row, at every tile width."""
    E, k, N, K = 8, 2, 200, 384
    g = R.gen(T)
    w, ws = R.weights(g, E, N, K)
    q, s = R.codes(g, T, K)
    ids = R.ids(g, T, E, k)
    clean = ft.moe_fp8_fp8(w, ws, q, s, ids)
    qb = q.clone()
    qb.view(torch.uint8)[T // 2, 300] = 0x7F
    out = ft.moe_fp8_fp8(w, ws, qb, s, ids)
    assert torch.isnan(out[T // 2]).all()
    keep = torch.arange(T, device="cuda") != T // 2
    assert torch.equal(out[keep], clean[keep])
    wb = w.clone()
    wb.view(torch.uint8)[2, 131, 30] = 0xFF
    out = ft.moe_fp8_fp8(wb, ws, q, s, ids)
    hit = ids == 2
    assert torch.isnan(out[hit][:, 131]).all()
    assert torch.equal(out[~hit], clean[~hit])
    out[:, :, 131], clean[:, :, 131] = 0, 0
    assert torch.equal(out, clean)


def with_operators(ft, c, dt, kind, rows_dtype):
    """y of the layer, and of the operators called one by one."""
    T, E, k, H, I = c
    x, logits, w13, s13, w2, s2 = inputs(*c, dt)
    y, ids, w = ft.moe_layer_fp8(x, logits, w13, s13, w2, s2, k, kind)
    gi, gw = ft.moe_gate(logits, k)
    assert torch.equal(ids, gi) and torch.equal(w, gw)
    h = ft.moe_fp8_fp8(w13, s13, *ft.quantize_fp8(x), ids)
    mid = ft.act_mul_quantize_fp8(h.view(-1, 2 * I), kind)
    rows = ft.moe_fp8_fp8_slots(w2, s2, *mid, ids, out_dtype=rows_dtype)
    return y, ft.moe_combine(rows, w, out_dtype=dt)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("c", BATCHES)
def test_layer_is_its_operators(ft, c, dt, kind):
    """The same bits as the operators called one by one, with the second product's rows in fp32, or (bf16 layers with
    more than 52 slots per expert) in bf16.

    With more than 52 slots per expert and n_inter % 128 == 0 the first product quantizes act(gate) * up itself, off by
    up to 10 * 2^-24: of values and scales together at most 2 * 10 * 2^-24 * 16 = 2e-5 lie so near a tie (16 to a
    factor of 2) that their code turns, one value in 66 tokens of 768, which moves a row by an eighth of one of its
    768 terms, some 0.004 of it: sqrt(1 / 66) * 0.004 = 5e-4 of the norm; scales that are one bit off turn roundings of
    rows and y, far less.  2^-10 covers both."""
    many = c[0] * c[2] > 52 * c[1]
    y, want = with_operators(ft, c, dt, kind, torch.bfloat16 if many and dt == torch.bfloat16 else torch.float32)
    if not (many and c[4] % 128 == 0):
        assert torch.equal(y, want)
        return
    off = (y.double() - want.double()).abs()
    assert float(off.norm() / want.double().norm()) < 2.0 ** -10
    assert (off.amax(1) <= 2.0 ** -5 * want.double().abs().amax(1)).all()


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("up", [6, 21, 60, 100])
@pytest.mark.parametrize("c", BATCHES)
def test_layer_of_far_gates(ft, c, up, kind):
    """Gates 2^up of their usual size: act(g) is g or 0, also where g^3 or g log2(e) leaves fp32; the second matrix
    undoes the size.  As near to the operators as test_layer_is_its_operators says."""
    T, E, k, H, I = c
    x, logits, w13, s13, w2, s2 = inputs(*c)
    far = s13.clone()
    far[:, :I // 128] *= 2.0 ** up              # (rows of a block that gate and up share stay as they are)
    s2 = s2 * 2.0 ** -up
    y, ids, w = ft.moe_layer_fp8(x, logits, w13, far, w2, s2, k, kind)
    h = ft.moe_fp8_fp8(w13, far, *ft.quantize_fp8(x), ids)
    mid = ft.act_mul_quantize_fp8(h.view(-1, 2 * I), kind)
    many = T * k > 52 * E
    rows = ft.moe_fp8_fp8_slots(w2, s2, *mid, ids, out_dtype=torch.bfloat16 if many else torch.float32)
    want = ft.moe_combine(rows, w, out_dtype=x.dtype)
    assert torch.isfinite(y).all() and float(want.abs().max()) > 0
    if not (many and I % 128 == 0):
        assert torch.equal(y, want)
        return
    off = (y.double() - want.double()).abs()
    assert float(off.norm() / want.double().norm()) < 2.0 ** -10
    assert (off.amax(1) <= 2.0 ** -5 * want.double().abs().amax(1)).all()
