"""The FP8 layer on inputs whose every sum is exact: each element of y has one right value.

x holds whole numbers with 448 in every block of 128, so its scales are 1 and its codes itself.
Gate rows give a token (and block) one large g, where act(g) = g in fp32 (exp(-16.7) rounds off beside 1);
an up row picks one column of x, so that a block of g * up has the scale g * 2^n and codes that
are whole numbers times a power of 2.  The second matrix holds small whole numbers and the chosen
experts' weights are 1.  Every partial sum then has at most 24 bits (asserted below), whatever its
order, and y is rounded once to its type; bf16 layers of more than 52 slots per expert round each
expert's row to bf16 before that.
"""

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


def to_codes(v):
    q = v.to(torch.float8_e4m3fn)
    assert torch.equal(R.decode(q), v.double())
    return q


def inputs(T, E, k, H, I, dt, none):
    g = R.gen(T * 31 + E * 7 + H + I)

    def whole(*shape, n=3):
        return torch.randint(-n, n + 1, shape, generator=g, device="cuda").float()

    x = whole(T, H)
    x[:, 5::128] = 448
    # columns that a block of up rows has to pick for its largest value to be 448 * 2^n
    w13 = torch.zeros(E, 2 * I, H, device="cuda")
    w13[:, :I, 5] = 1
    w13[:, :I, 6 % H] += 1
    w13[:, :I, 9 % H] += 2
    pick = torch.randint(0, H, (E, I), generator=g, device="cuda")
    pick[:, ::128] = 5
    sign = torch.randint(0, 2, (E, I), generator=g, device="cuda").float() * 2 - 1
    w13[:, I:].scatter_(2, pick[:, :, None], sign[:, :, None])
    rb, cb = R.blocks(2 * I), R.blocks(H)
    odd = torch.arange(E, device="cuda")[:, None, None] + torch.arange(rb, device="cuda")[None, :, None] + \
        torch.arange(cb, device="cuda")[None, None, :]
    s13 = torch.where(odd % 2 == 0, 0.125, 0.25)
    w2 = whole(E, H, I, n=1)
    s2 = torch.where((torch.arange(E, device="cuda")[:, None, None] + torch.arange(cb, device="cuda")[None, :, None] +
                      torch.arange(R.blocks(I), device="cuda")[None, None, :]) % 2 == 0, -1.0, 1.0) / 1024
    # k experts at +100 (sigmoid 1 in fp32), the others at -100; some tokens have fewer, one none
    order = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :k]
    logits = torch.full((T, E), -float("inf"), device="cuda")
    logits.scatter_(1, order, 100.0)
    logits[torch.rand(T, E, generator=g, device="cuda") < none] = -float("inf")
    if none:
        logits[T // 2] = -float("inf")
    return x.to(dt), logits, to_codes(w13), s13, to_codes(w2), s2


def rows64(x, ids, w13, s13, w2, s2):
    """The expert rows in 64 bits, and the most bits that a partial sum of one can need."""
    T, k = ids.shape
    E, H, I = w2.shape
    out = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
    flat, bits = ids.reshape(-1), 0.0
    for e in torch.unique(flat[flat >= 0]).tolist():
        sel = (flat == e).nonzero()[:, 0]
        h = x[sel // k].double() @ (R.decode(w13[e]) * R.expand_matrix(s13[e], 2 * I, H)).t()
        g, a = h[:, :I], h[:, :I] * h[:, I:]
        assert float(g.min()) > 17.4 and float(g.max()) < 2 ** 9
        nb = R.blocks(I)
        amax = torch.nn.functional.pad(a.abs(), (0, nb * 128 - I)).view(-1, nb, 128).amax(2)
        scale = (amax / 448).repeat_interleave(128, 1)[:, :I]
        t = a / scale
        assert torch.equal(R.nearest_e4m3(t)[0], t)
        m = R.decode(w2[e]) * R.expand_matrix(s2[e], H, I)
        out[sel] = a @ m.t()
        # in units of the finest term: h is a multiple of 2^-3, a of 2^-6, m of 2^-10
        bits = max(bits, float((a.abs() @ m.abs().t()).max()) * 2.0 ** 16)
    return out.view(T, k, H), bits


CASES = [
    # T, E, k, H, I, masked
    # a few tokens
    (1, 8, 2, 272, 144, 0.0), (3, 64, 4, 400, 272, 0.1), (8, 128, 8, 144, 128, 0.2),
    (20, 40, 1, 1040, 816, 0.1),                  # few slots, larger matrices: separate launches
    (2, 3, 2, 48, 16, 0.0),                       # tiles of 16
    (40, 16, 4, 272, 256, 0.1), (150, 128, 8, 272, 144, 0.1), (100, 20, 4, 400, 272, 0.2),
    (1000, 100, 3, 144, 128, 0.1),                # tiles of 32, over 1024 slots
    # tiles of 256: the activation in the first product, and after it; tails of slots, rows and columns
    (300, 6, 3, 272, 256, 0.1), (300, 6, 3, 272, 208, 0.1), (777, 4, 2, 400, 384, 0.05),
    (531, 5, 4, 1040, 128, 0.3), (65, 1, 1, 144, 128, 0.0), (257, 1, 1, 528, 384, 0.0),
    (8300, 12, 2, 48, 128, 0.1), (9000, 40, 6, 80, 144, 0.2),
]


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("c", CASES)
def test_layer_exact(ft, c, dt, kind):
    T, E, k, H, I, none = c
    x, logits, w13, s13, w2, s2 = inputs(T, E, k, H, I, dt, none)
    buf = torch.full((T * H + 2 * 1031,), 1234.0, dtype=dt, device="cuda")
    y = buf[1031:-1031].view(T, H)                       # starts at an odd element
    out, ids, w = ft.moe_layer_fp8(x, logits, w13, s13, w2, s2, k, kind, score="sigmoid", renormalize=False, out=y)
    assert out.data_ptr() == y.data_ptr()
    assert ((ids >= 0) == (w == 1)).all() and ((ids >= 0) | (w == 0)).all()
    assert torch.equal((ids >= 0).sum(1), (logits > 0).sum(1))
    rows, bits = rows64(x, ids, w13, s13, w2, s2)
    assert bits < 2.0 ** 24 and float(rows.abs().sum(1).max()) * 2.0 ** 16 < 2.0 ** 24
    if dt == torch.bfloat16 and T * k > 52 * E:
        rows = rows.float().to(dt).double()
    want = rows.sum(1).to(dt)
    assert torch.isfinite(want).all()
    wrong = y != want
    assert not wrong.any(), f"{int(wrong.sum())} of {wrong.numel()} differ, the first at {wrong.nonzero()[0].tolist()}"
    assert (buf[:1031] == buf[0]).all() and (buf[-1031:] == buf[0]).all()


@pytest.mark.parametrize("ldt", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [1, 40, 500])
def test_layer_logits(ft, T, ldt):
    """Logits of every type whose rows lie apart give the same layer, and the router's own outputs."""
    E, k, H, I = 8, 2, 272, 144
    x, _, w13, s13, w2, s2 = inputs(T, E, k, H, I, torch.bfloat16, 0.0)
    wide = torch.randn(T, E + 3, generator=R.gen(T), device="cuda").to(ldt)
    logits = wide[:, 2:2 + E]
    y, ids, w = ft.moe_layer_fp8(x, logits, w13, s13, w2, s2, k)
    i1 = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w1 = torch.zeros(T, k, device="cuda")
    got = ft.moe_gate(logits, k, topk_ids=i1, topk_weights=w1)
    assert got[0].data_ptr() == i1.data_ptr() and got[1].data_ptr() == w1.data_ptr()
    assert torch.equal(ids, i1) and torch.equal(w, w1)
    assert torch.equal(y, ft.moe_layer_fp8(x, logits.contiguous(), w13, s13, w2, s2, k)[0])
