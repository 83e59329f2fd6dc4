"""The gated activation of the FP8 operators is the formula's in fp32, also far from zero."""

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
    return ft


def z_of(g, kind):
    return g if kind == 0 else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)


def act_bound(z, kind):
    """How far an fp32 evaluation of act(g) * up / 448 may be off, over its size, in units of 2^-24: exp 4 (2 ulp)
    and 1 for a correction of its argument, the sum 1, the reciprocal 2, two products and the quotient by
    448 1 each, and 1 to spare.  For GELU z itself is off by two constants, three products, a sum and a product,
    7 of its size, of which act(g) sees the part exp(-z) / (1 + exp(-z))."""
    return (12 + (7 * z.abs() * torch.sigmoid(-z) if kind else 0)) * R.U32


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", [0, 1])
def test_act_far_from_zero(ft, kind, dtype):
    """One value in every block, so that the block's scale is that value's: g / (1 + exp(-z)) * up / 448.

    z ends at -88: past it exp overflows fp32."""
    n = 4096
    g = torch.linspace(-87.9, 20, n) if kind == 0 else torch.linspace(-10.0, 6, n)
    g = g.to(dtype).float()
    up = torch.full((n,), 1e6)
    up[z_of(g.double(), kind) < -60] = 1e30          # keeps the product inside fp32's normal range
    h = torch.zeros(n, 2 * 128)
    at = torch.arange(n) % 128
    h[torch.arange(n), at] = g
    h[torch.arange(n), 128 + at] = up
    h = h.to(dtype).cuda()
    q, s = ft.act_mul_quantize_fp8(h, kind)
    gd, ud = h[:, :128].double().gather(1, at[:, None].cuda())[:, 0], h[:, 128:].double().gather(1, at[:, None].cuda())[:, 0]
    z = z_of(gd, kind)
    assert float(z.min()) >= -88
    want = gd / (1 + torch.exp(-z)) * ud
    rel = act_bound(z, kind)
    err = (s[:, 0].double() - want.abs() / 448).abs()
    bad = ~(err <= rel * want.abs() / 448)
    assert not bad.any(), f"{int(bad.sum())} of {n} outside, the first at g = {float(gd[bad][0])}"
    live = R.decode(q).gather(1, at[:, None].cuda())[:, 0]
    assert torch.equal(live, torch.where(want == 0, 0.0, 448.0 * torch.sign(want)))


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("size", [3.0, 30.0])
def test_act_quantize(ft, kind, dtype, size):
    """Scales within the bound of their block's values; codes the nearest to their quotients, or next to a tie."""
    rows, I = 700, 400
    h = (torch.randn(rows, 2 * I, generator=R.gen(rows + kind), device="cuda") * size).to(dtype)
    q, s = ft.act_mul_quantize_fp8(h, kind)
    g, u = h.double().chunk(2, 1)
    z = z_of(g, kind)
    a = torch.where(z > -88, g / (1 + torch.exp(-z)) * u, 0.0)
    off = a.abs() * act_bound(z, kind) + (z <= -88) * g.abs() * u.abs() * 2.0 ** -126
    nb = R.blocks(I)

    def block_max(v):
        return torch.nn.functional.pad(v, (0, nb * 128 - I)).view(rows, nb, 128).amax(2)

    amax, worst = block_max(a.abs()), block_max(off)
    assert ((s.double() - amax / 448).abs() <= worst / 448).all()
    scale = s.double().repeat_interleave(128, 1)[:, :I]
    t = a / scale
    step = R.nearest_e4m3(t.abs().clamp(max=448))[1]
    assert ((R.decode(q) - t).abs() <= step / 2 * (1 + 2.0 ** -20) + off / scale + t.abs() * R.U32).all()


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("size", [3.0, 30.0])
def test_act_quantize_is_the_formula_in_fp32(ft, kind, dtype, size):
    """Codes and scales are those that elementary fp32 operations give, bit for bit."""
    rows, I = 700, 400
    h = (torch.randn(rows, 2 * I, generator=R.gen(rows + kind), device="cuda") * size).to(dtype)
    q, s = ft.act_mul_quantize_fp8(h, kind)
    g, u = h.float().chunk(2, 1)
    z = g if kind == 0 else 1.5957691216057308 * (g + 0.044715 * g * g * g)
    a = g / (1.0 + torch.exp(-z)) * u
    nb = R.blocks(I)
    b = torch.nn.functional.pad(a, (0, nb * 128 - I)).view(rows, nb, 128)
    amax = b.abs().amax(2)
    want = amax / torch.full_like(amax, 448.0)
    assert torch.equal(s, want)
    t = torch.where(want[:, :, None] > 0, b / want[:, :, None], 0.0)
    assert torch.equal(R.decode(q), R.nearest_e4m3(t.double())[0].view(rows, -1)[:, :I])


@pytest.mark.parametrize("kind", [0, 1])
def test_act_limits(ft, kind):
    """Gates whose exponential or cube leaves fp32: act(g) is g or 0, and only what is not finite spoils its block."""
    big = 3e38
    gates = [big, -big, 1e13, -1e13, 1e6, -1e6, 2.0 ** 20, -2.0 ** 20, 200.0, -200.0, -89.0, 0.0, math.inf, -math.inf, math.nan]
    h = torch.zeros(len(gates), 256)
    h[:, 7] = torch.tensor(gates)
    h[:, 128 + 7] = 0.5
    h[:, 9], h[:, 128 + 9] = 64.0, 2.0 ** -10
    q, s = ft.act_mul_quantize_fp8(h.cuda(), kind)
    v = (R.decode(q) * s.double()).cpu()
    for i, g in enumerate(gates):
        if not math.isfinite(g):
            assert not math.isfinite(float(s[i, 0])), g
            continue
        want = max(g, 0.0) * 0.5
        assert abs(float(v[i, 7]) - want) <= want * 2.0 ** -20, (g, float(v[i, 7]))
        assert float(s[i, 0]) > 0 and torch.isfinite(v[i]).all()
