"""Load-balance loss and the router's and the weighted sum's gradients against plain 64-bit forms (adapt_ref.py)."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import adapt_ref as A  # noqa: E402
from adapt_ref import U, U32, inside  # noqa: E402

TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def ft():
    import bit_quantized_moe_quantize_gb300 as ft
    from bit_quantized_moe_quantize_gb300 import build
    build.build()
    ft.load()
    ft.read_device_error()
    yield ft
    assert ft.read_device_error() == 0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def router(seed, T, E, k, dtype, mask=0.0, pitch=0):
    """Logits of size 1 to 6 (rows E + pitch apart) and distinct ids, -1 for masked experts."""
    g = gen(seed)
    wide = (torch.randn(T, E + pitch, generator=g, device="cuda") * 1.5).to(dtype)
    x = wide[:, :E]
    if mask:
        gone = torch.rand(T, E, generator=g, device="cuda") < mask
        gone[T // 2] = True
        kind = torch.where(torch.rand(T, E, generator=g, device="cuda") < 0.5, -math.inf, math.nan).to(dtype)
        x.copy_(torch.where(gone, kind, x))
    ids = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32)
    ids = torch.where(x.gather(1, ids.long()) > -math.inf, ids, -1).to(torch.int32).contiguous()
    return g, x, ids


def cuts(g, T, S):
    if S == 0:
        return None
    c = torch.randint(0, T + 1, (S + 1,), generator=g, device="cuda").sort().values.to(torch.int32)
    return c


# ---------------------------------------------------------------- balance
SIZES = [dict(T=1, E=1, k=1), dict(T=1, E=8, k=2, S=1), dict(T=3, E=5, k=5, S=2), dict(T=64, E=128, k=8),
         dict(T=65, E=128, k=8), dict(T=257, E=60, k=4, S=7), dict(T=1000, E=33, k=3, S=1000),
         dict(T=2000, E=256, k=8, S=3), dict(T=777, E=257, k=9, S=40), dict(T=130, E=512, k=8),
         dict(T=67, E=4096, k=6, S=5), dict(T=20000, E=64, k=6, S=12), dict(T=20000, E=160, k=2), dict(T=3, E=513, k=1)]


def check_balance(ft, x, ids, score, off):
    loss, counts, scale = ft.moe_balance_loss(x, ids, score=score, seq_offsets=off)
    want, wc, ws = A.balance(torch.where(x > -math.inf, x, -math.inf).double(), ids, score, off)
    assert torch.equal(counts.long(), wc)
    inside(scale, ws, 2 * U32 * ws, "seq_scale")
    # p: 60 roundings (gate_grad's); its sum over at most 128 rows of a lane, 64 lanes' and 608 CTAs' parts by
    # groups, all positive: under 190 roundings; counts and scales are exact but for one
    inside(loss, want, 256 * U32 * want, "loss")
    return loss, counts, scale


@pytest.mark.parametrize("c", SIZES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", TYPES)
def test_balance(ft, c, score, dtype):
    T, E, k = c["T"], c["E"], c["k"]
    for mask, pitch in ((0.0, 0), (0.3, 5)):
        g, x, ids = router(T + E, T, E, k, dtype, mask, pitch)
        check_balance(ft, x, ids, score, cuts(g, T, c.get("S", 0)))


def test_balance_edges(ft):
    """No token, rows outside the sequences, only padding, an even load, ids that repeat, offsets out of range."""
    x = torch.zeros(0, 8, device="cuda")
    loss, counts, scale = ft.moe_balance_loss(x, torch.zeros(0, 2, dtype=torch.int32, device="cuda"))
    assert float(loss) == 0 and not counts.any() and float(scale) == 0
    off = torch.zeros(20, dtype=torch.int32, device="cuda")
    loss, counts, scale = ft.moe_balance_loss(x, torch.zeros(0, 2, dtype=torch.int32, device="cuda"), seq_offsets=off)
    assert float(loss) == 0 and counts.shape == (19, 8) and not counts.any() and not scale.any()
    x = torch.full((70, 8), -math.inf, device="cuda")
    none = torch.full((70, 2), -1, dtype=torch.int32, device="cuda")
    loss, counts, scale = ft.moe_balance_loss(x, none)
    assert float(loss) == 0 and not counts.any() and float(scale) == 0
    x = torch.zeros(512, 8, device="cuda")
    ids = torch.arange(1024, device="cuda").remainder(8).view(512, 2).to(torch.int32)
    loss, counts, _ = ft.moe_balance_loss(x, ids)
    assert abs(float(loss) - 1) < 64 * U32 and (counts == 128).all()
    ids[:] = 3
    loss, counts, _ = ft.moe_balance_loss(x, ids)
    assert abs(float(loss) - 1) < 64 * U32 and int(counts[0, 3]) == 1024
    g, x, ids = router(9, 300, 16, 2, torch.float32)
    off = torch.tensor([-5, 40, 40, 900, 901], dtype=torch.int32, device="cuda")
    loss, counts, scale = check_balance(ft, x, ids, "softmax", off)
    assert int(counts.sum()) == 600 and float(scale[1]) == 0 and float(scale[3]) == 0


def test_balance_bad_ids(ft):
    g, x, ids = router(4, 100, 16, 2, torch.bfloat16)
    ids[7, 1] = 16
    ids[50, 0] = -2
    check_balance(ft, x, ids, "softmax", None)
    assert ft.read_device_error() == ft.FT_DEVERR_BAD_EXPERT_ID


# --------------------------------------------------------- gate's gradient
@pytest.mark.parametrize("c", SIZES)
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("dtype", TYPES)
def test_gate_backward(ft, c, score, renorm, dtype):
    T, E, k = c["T"], c["E"], c["k"]
    for mask, pitch in ((0.0, 0), (0.3, 5)):
        g, x, ids = router(T * 3 + E, T, E, k, dtype, mask, pitch)
        off = cuts(g, T, c.get("S", 0))
        gw = torch.randn(T, k, generator=g, device="cuda")
        gw[ids < 0] = math.nan                          # takes no part
        if T > 2 and k > 1:
            ids[T // 3, 1] = ids[T // 3, 0]             # one that repeats
        _, counts, scale = ft.moe_balance_loss(x, ids, score=score, seq_offsets=off)
        gl = torch.rand((), generator=g, device="cuda") * T
        loss = dict(counts=counts, seq_scale=scale, grad_loss=gl, seq_offsets=off)
        part = (counts, scale, gl, off)
        for w, b in ((gw, None), (None, part), (gw, part)):
            got = ft.moe_gate_backward(x, ids, w, score=score, renormalize=renorm, scale=1.5, **(loss if b else {}))
            want, bound = A.gate_grad(x, ids, w, score, renorm, 1.5, b)
            inside(got, want, bound, f"{'weights ' if w is not None else ''}{'loss' if b else ''}")


@pytest.mark.parametrize("E,k", [(24, 3), (64, 12), (128, 8), (200, 4), (512, 40), (600, 6)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_backward_rows_in_turn(ft, E, k, score):
    """More rows than the lanes have room for at once, the last ones a set that is not full; ids that repeat and leave in between."""
    T = {24: 60_001, 64: 60_001, 128: 60_001, 200: 29_999, 512: 9_001, 600: 2_003}[E]
    g, x, ids = router(E, T, E, k, torch.bfloat16, 0.1, 8)
    ids[::7, 1] = ids[::7, 0]
    ids[5::11, 2] = -1
    gw = torch.randn(T, k, generator=g, device="cuda")
    got = ft.moe_gate_backward(x, ids, gw, score=score)
    want, bound = A.gate_grad(x, ids, gw, score, True, 1.0, None)
    inside(got, want, bound)
    assert torch.equal(got, ft.moe_gate_backward(x, ids, gw, score=score))


def test_gate_backward_repeats(ft):
    """One expert in all of a row's 40 slots: added in the slots' order, the same bits every time."""
    g, x, _ = router(2, 33, 64, 40, torch.float32)
    ids = torch.randint(0, 3, (33, 40), generator=g, device="cuda", dtype=torch.int32)
    gw = torch.randn(33, 40, generator=g, device="cuda")
    first = ft.moe_gate_backward(x, ids, gw, score="sigmoid")
    want, bound = A.gate_grad(x, ids, gw, "sigmoid", True, 1.0)
    inside(first, want, 2 * bound)      # sums of up to 40 slots: as many roundings more
    for _ in range(5):
        assert torch.equal(first, ft.moe_gate_backward(x, ids, gw, score="sigmoid"))


def test_gate_backward_limits(ft):
    """Lowest values, infinities, rows of padding, sums below the smallest divisor."""
    inf, low = math.inf, torch.finfo(torch.float32).min
    x = torch.tensor([[inf, 1, inf, 2], [low, low, low, low], [-inf] * 4, [low, 0, -inf, math.nan], [-200, -200, 0, 0],
                      [-100, -100, -100, -100], [100, 100, 100, 0]], device="cuda")
    ids = torch.tensor([[0, 2], [0, 1], [0, 1], [1, 2], [0, 1], [0, 1], [0, 1]], dtype=torch.int32, device="cuda")
    gw = torch.tensor([[1.0, -2.0]] * 7, device="cuda")
    counts = torch.tensor([[3, 4, 5, 2]], dtype=torch.int32, device="cuda")
    loss = dict(counts=counts, seq_scale=torch.ones(1, device="cuda"), grad_loss=torch.ones(1, device="cuda"))
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            for b in ({}, loss):
                got = ft.moe_gate_backward(x, ids, gw, score=score, renormalize=renorm, **b)
                assert torch.isfinite(got).all(), (score, renorm, got)
                assert not got[2].any() and not got[3, 2:].any()
    got = ft.moe_gate_backward(x, ids, gw)
    assert torch.allclose(got[0].cpu(), torch.tensor([0.75, 0, -0.75, 0]))      # two at infinity: 1/2 each
    assert torch.allclose(got[1].cpu(), torch.tensor([0.75, -0.75, 0, 0]))
    # e^-200 / 2 each: under the smallest divisor, where weights are s / 1e-30 and shrink with the others' scores
    assert got[4].abs().max() < 1e-30


def test_gate_backward_bad_ids(ft):
    g, x, ids = router(4, 100, 16, 2, torch.bfloat16)
    gw = torch.randn(100, 2, generator=g, device="cuda")
    ids[7, 1] = 16
    ids[50, 0] = -2
    got = ft.moe_gate_backward(x, ids, gw)
    want, bound = A.gate_grad(x, ids, gw, "softmax", True, 1.0)
    inside(got, want, bound)
    assert ft.read_device_error() == ft.FT_DEVERR_BAD_EXPERT_ID


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradients_against_differences(ft, score):
    """The whole router: differences of weights and loss along a direction, in fp64, against the gradient."""
    g, x, _ = router(11, 200, 24, 3, torch.float32)
    ids, _ = ft.moe_gate(x, 3, score=score)
    gw = torch.randn(200, 3, generator=g, device="cuda")
    off = torch.tensor([0, 50, 200], dtype=torch.int32, device="cuda")
    _, counts, scale = ft.moe_balance_loss(x, ids, score=score, seq_offsets=off)
    gl = torch.tensor(30.0, device="cuda")
    got = ft.moe_gate_backward(x, ids, gw, score=score, counts=counts, seq_scale=scale, grad_loss=gl, seq_offsets=off)
    d = torch.randn(200, 24, generator=g, device="cuda").double()

    def f(v):
        return float((A.weights(v, ids, score, True, 1.0) * gw.double()).sum() + 30.0 * A.balance(v, ids, score, off)[0])

    e = 1e-5
    diff = (f(x.double() + e * d) - f(x.double() - e * d)) / (2 * e)
    _, bound = A.gate_grad(x, ids, gw, score, True, 1.0, (counts, scale, gl, off))
    # rounding of sums of some 1e3 terms of size 1, and e^2 times a third derivative of as many terms
    assert abs(float((got.double() * d).sum()) - diff) < float((bound * d.abs()).sum()) + 1e3 * 2.0 ** -52 / e + 1e3 * e * e


# ------------------------------------------------------ combine's gradient
COMBINES = [(1, 1, 1), (1, 8, 2048), (3, 2, 17), (5, 3, 2813), (130, 8, 256), (40, 9, 1416), (700, 4, 40), (2, 1, 7168),
            (3000, 2, 64), (1, 3, 5)]


def check_combine(ft, dy, rows, w, **need):
    gr, gw = ft.moe_combine_backward(dy, rows, w, **need)
    T, k, N = rows.shape
    want = torch.where(w[:, :, None] != 0, w.double()[:, :, None] * dy.double()[:, None, :], 0.0)
    if gr is not None:
        dt = rows.dtype
        inside(gr, want, (U32 + (U[dt] if dt != torch.float32 else 0.0)) * 1.01 * want.abs() + A.LEAST[dt], "rows")
    if gw is not None:
        prod = torch.where(w[:, :, None] != 0, rows.double(), 0.0) * dy.double()[:, None, :]
        # a lane's share of the columns in turn, then 5 + 3 additions
        inside(gw, prod.sum(2), (N / 32 + 16) * U32 * prod.abs().sum(2), "weights")
    return gr, gw


@pytest.mark.parametrize("size", COMBINES)
@pytest.mark.parametrize("rt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("yt", TYPES)
def test_combine_backward(ft, size, rt, yt):
    T, k, N = size
    g = gen(T * 31 + N)
    dy = torch.randn(T, N, generator=g, device="cuda").to(yt)
    rows = torch.randn(T, k, N, generator=g, device="cuda").to(rt)
    w = torch.rand(T, k, generator=g, device="cuda")
    w[torch.rand(T, k, generator=g, device="cuda") < 0.2] = 0
    rows[w == 0] = math.nan                   # not read
    check_combine(ft, dy, rows, w)


def test_combine_backward_parts(ft):
    """Either gradient alone, operands that are aligned to their elements only, no token."""
    g = gen(3)
    flat = torch.randn(4 * 3 * 64 + 1, generator=g, device="cuda")[1:]
    rows, w = flat.view(4, 3, 64), torch.rand(4, 3, generator=g, device="cuda")
    dy = torch.randn(4 * 64 + 1, generator=g, device="cuda").to(torch.bfloat16)[1:].view(4, 64)
    assert check_combine(ft, dy, rows, w, need_rows=False)[0] is None
    assert check_combine(ft, dy, rows, w, need_weights=False)[1] is None
    out = torch.full((4 * 3 * 64 + 3,), 7.0, device="cuda")
    check_combine(ft, dy, rows, w, grad_rows=out[2:-1].view(4, 3, 64))
    assert out[:2].tolist() == [7, 7] and float(out[-1]) == 7
    gr, gw = ft.moe_combine_backward(dy[:0], rows[:0], w[:0])
    assert gr.shape == (0, 3, 64) and gw.shape == (0, 3)


def test_combine_backward_against_differences(ft):
    g = gen(8)
    T, k, N = 20, 3, 96
    dy = torch.randn(T, N, generator=g, device="cuda")
    rows, w = torch.randn(T, k, N, generator=g, device="cuda"), torch.rand(T, k, generator=g, device="cuda") + 0.1
    gr, gw = ft.moe_combine_backward(dy, rows, w)
    dr, dw = torch.randn(T, k, N, generator=g, device="cuda").double(), torch.randn(T, k, generator=g, device="cuda").double()

    def f(e):
        return float((((w.double() + e * dw)[:, :, None] * (rows.double() + e * dr)).sum(1) * dy.double()).sum())

    diff = (f(1e-4) - f(-1e-4)) / 2e-4
    got = float((gr.double() * dr).sum() + (gw.double() * dw).sum())
    size = float((gr.double() * dr).abs().sum() + (gw.double() * dw).abs().sum())
    assert abs(got - diff) < 32 * U32 * size


# ------------------------------------------------- streams, graphs, sizes
def test_streams_and_graphs(ft):
    """On another stream, and replayed from a graph with new inputs: the eager call's bits."""
    g, x, ids = router(21, 3000, 128, 8, torch.bfloat16)
    off = cuts(g, 3000, 6)
    gw = torch.randn(3000, 8, generator=g, device="cuda")
    rows = torch.randn(500, 8, 64, generator=g, device="cuda")
    dy, w = torch.randn(500, 64, generator=g, device="cuda"), torch.rand(500, 8, generator=g, device="cuda")
    gl = torch.ones((), device="cuda")

    def step():
        loss, counts, scale = ft.moe_balance_loss(x, ids, seq_offsets=off)
        out = ft.moe_gate_backward(x, ids, gw, counts=counts, seq_scale=scale, grad_loss=gl, seq_offsets=off)
        return (loss, counts, scale, out) + ft.moe_combine_backward(dy, rows, w)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    x.copy_(x.flip(0))
    off.copy_((off.flip(0) * -1 + 3000).to(torch.int32))
    gw.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(step(), got))


def test_far_offsets(ft):
    """Elements past the 32-bit range."""
    T, E = 540_000, 4096
    x = torch.zeros(T, E, device="cuda", dtype=torch.float16)
    x[-1, 7] = 3
    ids = torch.zeros(T, 1, device="cuda", dtype=torch.int32)
    ids[-1] = 7
    gw = torch.ones(T, 1, device="cuda")
    out = ft.moe_gate_backward(x, ids, gw, renormalize=False)
    want, bound = A.gate_grad(x[-3:], ids[-3:], gw[-3:], "softmax", False, 1.0)
    inside(out[-3:], want, bound)
    loss, counts, _ = ft.moe_balance_loss(x, ids)
    assert int(counts[0, 0]) == T - 1 and int(counts[0, 7]) == 1
    assert abs(float(loss) - 1) < 1e-4            # all but one row are even
    del x, out
    T, k, N = 66_000, 4, 8200
    rows = torch.zeros(T, k, N, device="cuda", dtype=torch.bfloat16)
    rows[-1] = 2
    dy = torch.ones(T, N, device="cuda", dtype=torch.bfloat16)
    w = torch.full((T, k), 0.5, device="cuda")
    gr, gw = ft.moe_combine_backward(dy, rows, w)
    assert (gr[-1] == 0.5).all() and (gw[-1] == 2 * N).all() and not gw[:-1].any()


def test_refusals(ft):
    g, x, ids = router(1, 10, 16, 2, torch.float32)
    gw = torch.zeros(10, 2, device="cuda")
    with pytest.raises(ValueError):
        ft.moe_gate_backward(x, ids, gw, counts=torch.zeros(1, 16, dtype=torch.int32, device="cuda"))
    with pytest.raises(ft.FtError):
        ft.moe_gate_backward(x, ids)
    with pytest.raises(ValueError):
        ft.moe_gate_backward(x, ids, gw, score="tanh")
    with pytest.raises(ValueError):
        ft.moe_gate_backward(x, ids[:5].contiguous(), gw)
    with pytest.raises(TypeError):
        ft.moe_balance_loss(x, ids.long())
    with pytest.raises(ValueError):
        ft.moe_balance_loss(x, ids, seq_offsets=torch.zeros(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        ft.moe_balance_loss(x, ids, seq_offsets=torch.zeros(3, device="cuda"))
    with pytest.raises(TypeError):
        ft.moe_balance_loss(x.cpu(), ids)
    rows, w = torch.zeros(4, 2, 8, device="cuda"), torch.zeros(4, 2, device="cuda")
    with pytest.raises(ValueError):
        ft.moe_combine_backward(torch.zeros(4, 9, device="cuda"), rows, w)
    with pytest.raises(TypeError):
        ft.moe_combine_backward(torch.zeros(4, 8, device="cuda"), rows.half(), w)
    with pytest.raises(ft.FtError):
        ft.moe_combine_backward(torch.zeros(4, 8, device="cuda"), rows, w, need_rows=False, need_weights=False)
