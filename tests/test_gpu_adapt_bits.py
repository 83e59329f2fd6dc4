"""How many bits A x and B^T dy keep on their way through an adapter, and what long sums lose (adapt_bits.py)."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import adapt_bits as D  # noqa: E402

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
N = K = 72


@pytest.fixture(scope="module")
def ft():
    import bit_quantized_moe_quantize_gb300 as ft
    from bit_quantized_moe_quantize_gb300 import build
    build.build()
    ft.load()
    ft.read_device_error()
    yield ft
    assert ft.read_device_error() == 0


# tokens, slots of each, adapters, rank: one launch, tiles of 16, 64 and 128 slots, both sides of the ranks where parts change places
SIZES = [(2, 1, 1, 8), (64, 1, 5, 40), (100, 2, 3, 128), (400, 1, 64, 16), (300, 2, 40, 72), (600, 2, 3, 40), (1200, 1, 4, 64),
         (3000, 1, 2, 64), (1400, 2, 1, 16), (700, 2, 2, 128)]


def ranks(e, R):
    """Two ranks of adapter e."""
    return e % R, (e + R // 2) % R


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def setup(T, k, L):
    """(generator, adapters of the tokens' pairs as ids, scales: powers of two)."""
    e = torch.arange(T, device="cuda") // 2 % L
    ids = e.to(torch.int32) if k == 1 else e[:, None].repeat(1, k).to(torch.int32)
    return gen(T + L), e, ids, torch.exp2(torch.arange(L, device="cuda").float() % 2)


def digits(L, R, n, cols_first, dtype):
    """Matrices [L, R, n] or [L, n, R] with the digits at the first three rows' values of one rank and the next three of another."""
    m = torch.zeros(L, R, n, device="cuda")
    for e in range(L):
        r0, r1 = ranks(e, R)
        m[e, r0, 0:3] = torch.tensor(D.DIGITS, device="cuda")
        m[e, r1, 3:6] = torch.tensor(D.DIGITS, device="cuda")
    return (m.transpose(1, 2) if cols_first else m).contiguous().to(dtype)


def opposed(L, R, n, cols_first, dtype):
    """Matrices that take the difference of the two ranks, times 1, 2 or 4 by column."""
    m = torch.zeros(L, R, n, device="cuda")
    p = torch.exp2(torch.arange(n, device="cuda").float() % 3)
    for e in range(L):
        r0, r1 = ranks(e, R)
        m[e, r0], m[e, r1] = p, -p
    return (m.transpose(1, 2) if cols_first else m).contiguous().to(dtype), p.double()


def rows_of(d, n, dtype):
    """[rows, n] with both numbers' values at the first six columns."""
    x = torch.zeros(d.shape[1], n, device="cuda")
    x[:, 0:3], x[:, 3:6] = D.wide(d[0]), D.wide(d[1])
    return x.to(dtype)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype,out", [(BF, F32), (BF, BF), (HF, F32), (HF, HF)])
def test_product_is_exact(ft, size, dtype, out):
    T, k, L, R = size
    g, e, ids, scales = setup(T, k, L)
    d, diff = D.numbers(g, T, "cuda")
    b, p = opposed(L, R, N, True, dtype)
    got = ft.lora_add(rows_of(d, K, dtype), digits(L, R, K, False, dtype), b, ids, scales=scales, out_dtype=out)
    want = (diff * scales[e])[:, None] * p
    assert torch.equal(got.double(), want if k == 1 else want[:, None, :].expand(T, k, N))


def paired(d, n, dtype):
    """Rows 2 i and 2 i + 1 whose numbers differ by as much at both ranks, up to the sign."""
    first = rows_of(d, n, dtype)
    x = torch.zeros(2 * len(first), n, device="cuda", dtype=dtype)
    x[0::2] = first
    x[1::2] = -rows_of(d.flip(0), n, dtype)
    return x


def one_each(pairs, rows, n, dtype):
    """One 1 in each row, rows of a pair in the same column; sums over pairs by column."""
    at = pairs % n
    x = torch.zeros(rows, n, device="cuda", dtype=dtype)
    x[torch.arange(rows, device="cuda"), at] = 1
    return x, at


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_gradients_of_x_and_a_are_exact(ft, size, dtype):
    T, k, L, R = size
    g, e, ids, scales = setup(T, k, L)
    S, pairs = T * k, torch.arange(T * k, device="cuda") // 2
    d, diff = D.numbers(g, S // 2, "cuda")
    dy = paired(d, N, dtype)                                    # by slot
    x, at = one_each(pairs if k == 1 else torch.arange(T, device="cuda"), T, K, dtype)
    a, p = opposed(L, R, K, False, dtype)
    slot_e = e if k == 1 else e.repeat_interleave(2)
    gx, ga, _ = ft.lora_backward(dy if k == 1 else dy.view(T, k, N), x, a, digits(L, R, N, True, dtype), ids, scales=scales, need_b=False)
    each = (diff[pairs] * scales[slot_e].double())[:, None] * p
    assert torch.equal(gx.double(), each if k == 1 else each.view(T, k, K).sum(1))
    want = torch.zeros(L, R, K, dtype=torch.float64, device="cuda")
    pe, col = slot_e[::2], at[::2] if k == 1 else at
    r0 = pe % R
    r1 = (pe + R // 2) % R
    want.index_put_((pe, r0, col), diff * scales[pe].double(), accumulate=True)
    want.index_put_((pe, r1, col), -diff * scales[pe].double(), accumulate=True)
    assert torch.equal(ga.double(), want)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_gradient_of_b_is_exact(ft, size, dtype):
    T, k, L, R = size
    g, e, ids, scales = setup(T, k, L)
    d, diff = D.numbers(g, T // 2, "cuda")
    x = paired(d, K, dtype)                                     # by token: a token's slots have the same
    dy, at = one_each(torch.arange(T, device="cuda") // 2, T, N, dtype)
    dy = dy if k == 1 else dy[:, None, :].repeat(1, k, 1)
    b, _ = opposed(L, R, N, True, dtype)
    _, _, gb = ft.lora_backward(dy, x, digits(L, R, K, False, dtype), b, ids, scales=scales, need_x=False, need_a=False)
    want = torch.zeros(L, N, R, dtype=torch.float64, device="cuda")
    pe, col = e[::2], at[::2]
    want.index_put_((pe, col, pe % R), k * diff * scales[pe].double(), accumulate=True)
    want.index_put_((pe, col, (pe + R // 2) % R), -k * diff * scales[pe].double(), accumulate=True)
    assert torch.equal(gb.double(), want)


def ones_and_more(g, *s, dtype):
    """Values in [1, 2): sums of their products only rise."""
    return (1.0 + torch.randint(0, 128, s, generator=g, device="cuda").float() / 128.0).to(dtype)


@pytest.mark.parametrize("T", [16, 300])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_long_sums_of_the_first_product(ft, T, dtype):
    """65536 products.  A stage's 64 are 8 truncations of at most 2^-23 of its sum; the stages of a CTA, 128, and the parts of the
    eight CTAs and four warps are added by rounding to nearest: 2^-20 + 142 2^-24.  An accumulator that went on through
    a CTA's stages would lose some 512 2^-25."""
    g = gen(T)
    x, a = ones_and_more(g, T, 65536, dtype=dtype), ones_and_more(g, 1, 8, 65536, dtype=dtype)
    b = torch.zeros(1, 64, 8, device="cuda", dtype=dtype)
    b[0, torch.arange(64), torch.arange(64) % 8] = 1
    got = ft.lora_add(x, a, b, torch.zeros(T, dtype=torch.int32, device="cuda"), out_dtype=F32)
    want = (x.double() @ a[0].double().t()).repeat(1, 8)
    assert float(((got.double() - want) / want).abs().max()) < 2.0 ** -20 + 142 * 2.0 ** -24


@pytest.mark.parametrize("dtype", [BF, HF])
def test_long_sums_of_the_gradients(ft, dtype):
    """65536 slots of one adapter in four chunks of 16384.  bf16: the 16 truncations (2^-23 each) of 128 slots, then 128 such sums,
    four chunks and three parts by rounding to nearest; fp16: the 8 of 32 slots, then 512 sums and four chunks.  An
    accumulator that went on through a chunk would lose some 1024 (2048) 2^-25.4 of the sum."""
    T, W, R = 65536, 4096, 16
    g = gen(5)
    x, dy = ones_and_more(g, T, W, dtype=dtype), torch.zeros(T, W, device="cuda", dtype=dtype)
    dy[:, 0] = ones_and_more(g, T, dtype=dtype)
    b = torch.zeros(1, W, R, device="cuda", dtype=dtype)
    b[0, 0] = 1 + torch.arange(R, device="cuda") / 16
    a = torch.zeros(1, R, W, device="cuda", dtype=dtype)
    _, ga, _ = ft.lora_backward(dy, x, a, b, torch.zeros(T, dtype=torch.int32, device="cuda"), need_x=False, need_b=False)
    v = dy[:, :1].double() * b[0, :1].double()
    bound = 2.0 ** -19 + 135 * 2.0 ** -24 if dtype == BF else 2.0 ** -20 + 516 * 2.0 ** -24
    want = v.t() @ x[:, ::61].double()
    assert float(((ga[0, :, ::61].double() - want) / want).abs().max()) < bound
