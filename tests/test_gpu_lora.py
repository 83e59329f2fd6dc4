"""Low-rank adapters and their gradients against plain 64-bit forms (adapt_ref.py)."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import adapt_ref as A  # noqa: E402
from adapt_ref import inside  # noqa: E402

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


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


def randn(g, *s):
    return torch.randn(*s, generator=g, device="cuda")


def make(c, dtype, out=None):
    """Inputs of a case: T tokens of k slots, L adapters of rank R, K columns, N rows; ids "any", "runs", "one" or "none"."""
    T, k, L, R, K, N = (c[n] for n in ("T", "k", "L", "R", "K", "N"))
    g = gen(T * 7 + R + K)
    kind = c.get("ids", "any")
    if kind == "runs":
        ids = torch.randint(0, L, (T // 50 + 1,), generator=g, device="cuda").repeat_interleave(50)[:T, None].repeat(1, k)
    elif kind == "one":
        ids = torch.full((T, k), L - 1, device="cuda")
    elif kind == "none":
        ids = torch.full((T, k), -1, device="cuda")
    else:
        ids = torch.randint(0, L, (T, k), generator=g, device="cuda")
    if c.get("gap"):
        ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < c["gap"], -1, ids)
    ids = ids.to(torch.int32).contiguous()
    if c.get("flat"):
        ids = ids[:, 0].contiguous()
    rows = T * k if c.get("slots") else T
    x = randn(g, rows, K).to(dtype)
    a, b = (randn(g, L, R, K) / math.sqrt(K)).to(dtype), (randn(g, L, N, R) / math.sqrt(R)).to(dtype)
    scales = None if c.get("plain") else torch.rand(L, generator=g, device="cuda") + 0.5
    return g, x, a, b, ids, scales


CASES = [
    dict(T=1, k=1, L=1, R=8, K=8, N=8, flat=True, plain=True), dict(T=1, k=1, L=64, R=16, K=2048, N=2048, flat=True),
    dict(T=7, k=8, L=60, R=16, K=256, N=520, gap=0.2), dict(T=64, k=1, L=64, R=16, K=1024, N=1032, gap=0.1, flat=True),
    dict(T=32, k=8, L=3, R=24, K=200, N=72, slots=True), dict(T=256, k=1, L=1, R=40, K=72, N=1416, ids="one", flat=True),
    dict(T=257, k=1, L=1, R=40, K=72, N=1416, ids="one", flat=True), dict(T=257, k=1, L=600, R=8, K=1000, N=64, flat=True),
    dict(T=300, k=4, L=5, R=128, K=136, N=264, gap=0.5), dict(T=1000, k=1, L=4, R=64, K=512, N=776, ids="runs", gap=0.02),
    dict(T=500, k=3, L=9, R=32, K=2000, N=96, slots=True, gap=0.1), dict(T=90, k=8, L=128, R=72, K=64, N=8),
    dict(T=300, k=1, L=2, R=16, K=64, N=128, ids="none", flat=True), dict(T=2049, k=2, L=1, R=8, K=72, N=136, ids="one"),
    dict(T=1100, k=1, L=16, R=48, K=328, N=4104, flat=True), dict(T=5, k=1, L=2, R=16, K=7168, N=64, ids="none"),
    dict(T=700, k=1, L=1, R=64, K=8, N=64, ids="one", flat=True), dict(T=1500, k=1, L=2, R=64, K=320, N=328, ids="runs", flat=True),
    dict(T=1300, k=1, L=1, R=128, K=128, N=192, ids="one", flat=True), dict(T=1290, k=1, L=2, R=16, K=4096, N=64, ids="runs", gap=0.01),
    dict(T=40000, k=1, L=7, R=8, K=64, N=64, gap=0.1, flat=True), dict(T=3000, k=6, L=300, R=8, K=72, N=64, gap=0.1),
    dict(T=271, k=1, L=1030, R=8, K=64, N=64, gap=0.1), dict(T=200, k=1, L=3, R=104, K=4096, N=200, gap=0.1),
]


@pytest.mark.parametrize("c", CASES)
@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, F32), (HF, HF), (HF, F32)])
@pytest.mark.parametrize("with_add", [True, False])
def test_lora_add(ft, c, dtype, out, with_add):
    g, x, a, b, ids, scales = make(c, dtype)
    add = randn(g, *ids.shape, c["N"]).to(out) if with_add else None
    got = ft.lora_add(x, a, b, ids, scales=scales, add=add, out_dtype=out)
    want, bound = A.lora(x, a, b, ids, scales, add, out)
    inside(got, want, bound)
    if with_add:
        none = ids < 0
        assert torch.equal(got[none], add[none])
        mine = add.clone()
        assert ft.lora_add(x, a, b, ids, scales=scales, add=mine, out=mine) is mine
        assert torch.equal(mine, got)


@pytest.mark.parametrize("c", CASES)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("with_add", [True, False])
def test_lora_backward(ft, c, dtype, with_add):
    g, x, a, b, ids, scales = make(c, dtype)
    dy = randn(g, *ids.shape, c["N"]).to(dtype)
    add = randn(g, *x.shape).to(dtype) if with_add else None
    got = ft.lora_backward(dy, x, a, b, ids, scales=scales, add=add)
    for name, p, (want, bound) in zip(("x", "a", "b"), got, A.lora_grads(dy, x, a, b, ids, scales, add)):
        inside(p, want, bound, name)
    if with_add:      # in place, and each alone: the same bits
        mine = add.clone()
        part = ft.lora_backward(dy, x, a, b, ids, scales=scales, add=mine, grad_x=mine, need_a=False, need_b=False)
        assert part[1] is None and part[2] is None and torch.equal(part[0], got[0])
        part = ft.lora_backward(dy, x, a, b, ids, scales=scales, need_x=False, need_b=False)
        assert part[0] is None and torch.equal(part[1], got[1])
        part = ft.lora_backward(dy, x, a, b, ids, scales=scales, need_x=False, need_a=False)
        assert torch.equal(part[2], got[2])


@pytest.mark.parametrize("dtype", [BF, HF])
def test_values_far_apart(ft, dtype):
    """Rows, ranks and adapters of very different sizes: each as exact as its own size allows."""
    c = dict(T=700, k=1, L=3, R=32, K=256, N=128, flat=True)
    g, x, a, b, ids, scales = make(c, dtype)
    x *= torch.exp2(torch.randint(-12, 5, (700, 1), generator=g, device="cuda").float()).to(dtype)
    a *= torch.exp2(torch.randint(-6, 3, (3, 32, 1), generator=g, device="cuda").float()).to(dtype)
    scales = torch.tensor([1e-3, 1.0, 300.0], device="cuda")
    got = ft.lora_add(x, a, b, ids, scales=scales, out_dtype=F32)
    inside(got, *A.lora(x, a, b, ids, scales, None, F32))
    dy = (randn(g, 700, 128) * torch.exp2(torch.randint(-9, 3, (700, 1), generator=g, device="cuda").float())).to(dtype)
    for name, p, (want, bound) in zip("xab", ft.lora_backward(dy, x, a, b, ids, scales=scales),
                                      A.lora_grads(dy, x, a, b, ids, scales, None)):
        inside(p, want, bound, name)


@pytest.mark.parametrize("T", [30, 400])
def test_rows_apart(ft, T):
    """A NaN in a row, an adapter or a row without an adapter stays where it belongs."""
    c = dict(T=T, k=1, L=3, R=16, K=128, N=96, flat=True)
    g, x, a, b, ids, scales = make(c, BF)
    ids[5], ids[6] = -1, 0
    x[5] = math.nan
    x[6, 3] = math.nan
    add = randn(g, T, 96).to(BF)
    b[2] = math.inf
    got = ft.lora_add(x, a, b, ids, scales=scales, add=add)
    assert torch.equal(got[5], add[5]) and torch.isnan(got[6]).all()
    ok = (ids < 2)
    ok[6] = False
    want, bound = A.lora(x, a, b[:2].contiguous(), ids, scales, add, BF)
    inside(got[ok], want[ok], bound[ok])
    dy = randn(g, T, 96).to(BF)
    gx, ga, gb = ft.lora_backward(dy, x, a, b, ids, scales=scales)
    assert torch.isfinite(ga[:2][1]).all() and torch.isfinite(gb[1]).all() and (gx[5] == 0).all()
    assert torch.isfinite(gx[ok]).all()


def test_adapters_apart(ft):
    """An adapter that is no number leaves its neighbours' results alone, at ranks and sizes whose last stage is not full."""
    for R, N in ((64, 136), (64, 128), (16, 72)):
        g, x, a, b, ids, scales = make(dict(T=900, k=1, L=3, R=R, K=136, N=N, ids="runs", flat=True), BF)
        ids.copy_((torch.arange(900, device="cuda") // 300).to(torch.int32))
        want = ft.lora_add(x, a, b, ids, scales=scales)
        dy = randn(g, 900, N).to(BF)
        grads = ft.lora_backward(dy, x, a, b, ids, scales=scales)
        a[1], b[1], dy[300:600], x[300:600] = math.nan, math.inf, math.nan, math.inf
        got = ft.lora_add(x, a, b, ids, scales=scales)
        keep = ids != 1
        assert torch.equal(got[keep], want[keep])
        gx, ga, gb = ft.lora_backward(dy, x, a, b, ids, scales=scales)
        assert torch.equal(gx[keep], grads[0][keep])
        assert torch.equal(ga[::2], grads[1][::2]) and torch.equal(gb[::2], grads[2][::2])


def test_bad_ids(ft):
    for T in (40, 400):
        g, x, a, b, ids, scales = make(dict(T=T, k=2, L=3, R=16, K=64, N=64), BF)
        ids[3, 1], ids[T - 1, 0] = 3, -7
        add = randn(g, T, 2, 64).to(BF)
        got = ft.lora_add(x, a, b, ids, scales=scales, add=add)
        assert torch.equal(got[3, 1], add[3, 1]) and torch.equal(got[T - 1, 0], add[T - 1, 0])
        inside(got, *A.lora(x, a, b, ids, scales, add, BF))
        assert ft.read_device_error() == ft.FT_DEVERR_BAD_EXPERT_ID
        dy = randn(g, T, 2, 64).to(BF)
        for need in (dict(), dict(need_x=False, need_a=False)):
            got = ft.lora_backward(dy, x, a, b, ids, scales=scales, **need)
            for p, (want, bound) in zip(got, A.lora_grads(dy, x, a, b, ids, scales, None)):
                if p is not None:
                    inside(p, want, bound)
            assert ft.read_device_error() == ft.FT_DEVERR_BAD_EXPERT_ID


def test_no_tokens(ft):
    x, a, b = torch.zeros(0, 64, device="cuda", dtype=BF), torch.ones(2, 8, 64, device="cuda", dtype=BF), torch.ones(2, 72, 8, device="cuda", dtype=BF)
    ids = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert ft.lora_add(x, a, b, ids).shape == (0, 72)
    gx, ga, gb = ft.lora_backward(torch.zeros(0, 72, device="cuda", dtype=BF), x, a, b, ids)
    assert gx.shape == (0, 64) and not ga.any() and not gb.any()


def test_only_its_elements(ft):
    """Nothing around the outputs is written."""
    for T in (33, 300):
        g, x, a, b, ids, scales = make(dict(T=T, k=1, L=3, R=24, K=72, N=40, flat=True, gap=0.2), BF)
        buf = torch.full((T * 40 + 64,), 7.0, device="cuda", dtype=BF)
        ft.lora_add(x, a, b, ids, scales=scales, out=buf[32:-32].view(T, 40))
        assert (buf[:32] == 7).all() and (buf[-32:] == 7).all()
        big = [torch.full((n + 64,), 7.0, device="cuda", dtype=d) for n, d in ((T * 72, BF), (3 * 24 * 72, F32), (3 * 40 * 24, F32))]
        ft.lora_backward(randn(g, T, 40).to(BF), x, a, b, ids, scales=scales, grad_x=big[0][32:-32].view(T, 72),
                         grad_a=big[1][32:-32].view(3, 24, 72), grad_b=big[2][32:-32].view(3, 40, 24))
        for t in big:
            assert (t[:32] == 7).all() and (t[-32:] == 7).all()


@pytest.mark.parametrize("T", [48, 900])
def test_streams_graphs_repeats(ft, T):
    """The same bits on another stream, again, and replayed from a graph with new inputs."""
    g, x, a, b, ids, scales = make(dict(T=T, k=2, L=4, R=16, K=512, N=256, gap=0.1), BF)
    dy, add = randn(g, T, 2, 256).to(BF), randn(g, T, 2, 256).to(BF)

    def step():
        return (ft.lora_add(x, a, b, ids, scales=scales, add=add),) + ft.lora_backward(dy, x, a, b, ids, scales=scales)

    want = step()
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(want, step()))
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
    ids.copy_((ids + 2).remainder(5) - 1)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(step(), got))


def test_two_streams_at_once(ft):
    jobs = []
    for seed in range(2):
        g, x, a, b, ids, scales = make(dict(T=2000 + seed, k=1, L=5, R=32, K=1024, N=1024, flat=True), BF)
        jobs.append((x, a, b, ids, scales, ft.lora_add(x, a, b, ids, scales=scales)))
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in jobs], [[], []]
    for _ in range(10):
        for i, (st, (x, a, b, ids, scales, _)) in enumerate(zip(streams, jobs)):
            with torch.cuda.stream(st):
                got[i].append(ft.lora_add(x, a, b, ids, scales=scales))
    torch.cuda.synchronize()
    assert all(torch.equal(p, jobs[i][5]) for i in range(2) for p in got[i])


@pytest.mark.parametrize("R", [16, 72])
def test_gradients_on_two_streams_at_once(ft, R):
    """Both calls' kernels want tensor memory and most of an SM's shared memory."""
    jobs = []
    for seed in range(2):
        g, x, a, b, ids, scales = make(dict(T=1600 + seed, k=2, L=3, R=R, K=512, N=768, gap=0.1), BF)
        args = (randn(g, *ids.shape, 768).to(BF), x, a, b, ids, scales)
        jobs.append((args, ft.lora_backward(*args)))
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in jobs], [[], []]
    for _ in range(6):
        for i, (st, (args, _)) in enumerate(zip(streams, jobs)):
            with torch.cuda.stream(st):
                got[i].append(ft.lora_backward(*args))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for i in range(2) for part in got[i] for p, q in zip(part, jobs[i][1]))


def test_nothing_between_two_calls(ft):
    """Calls one behind the other, the first without a tile of its own, the second in the same memory."""
    g, x, a, b, ids, scales = make(dict(T=3000, k=1, L=5, R=32, K=512, N=512, flat=True), BF)
    none = torch.full_like(ids, -1)
    want = ft.lora_add(x, a, b, ids, scales=scales)
    for _ in range(20):
        got = ft.lora_add(x, a, b, none, scales=scales)
        more = ft.lora_add(x, a, b, ids, scales=scales)
        assert not got.any() and torch.equal(more, want)


def test_gradients_against_differences(ft):
    g, x, a, b, ids, scales = make(dict(T=90, k=3, L=4, R=8, K=64, N=48, gap=0.1), BF)
    dy = randn(g, 90, 3, 48).to(BF)
    got = ft.lora_backward(dy, x, a, b, ids, scales=scales)
    d = [torch.randn(t.shape, generator=g, device="cuda").double() for t in (x, a, b)]

    def f(e):
        out = torch.zeros(90, 3, 48, dtype=torch.float64, device="cuda")
        X, P, Q = (t.double() + e * v for t, v in zip((x, a, b), d))
        for i in range(4):
            hit = (ids == i)[:, :, None]
            out += torch.where(hit, (X @ P[i].t() @ Q[i].t() * float(scales[i]))[:, None, :], 0.0)
        return float((out * dy.double()).sum())

    e = 1e-4
    diff = (f(e) - f(-e)) / (2 * e)
    size = sum(float((t.double() * v).abs().sum()) for t, v in zip(got, d))
    bound = sum(float((w[1] * v.abs()).sum()) for w, v in zip(A.lora_grads(dy, x, a, b, ids, scales, None), d))
    # the step's error: e^2 times the product of all three directions, of the gradients' size
    assert abs(sum(float((t.double() * v).sum()) for t, v in zip(got, d)) - diff) < bound + 100 * e * e * size


def test_far_offsets(ft):
    """Elements past the 32-bit range, in x, add, out and the gradient of x."""
    T, K, N = 140_000, 16, 16384
    g = gen(1)
    x, a, b = randn(g, T, K).to(BF), randn(g, 2, 8, K).to(BF), randn(g, 2, N, 8).to(BF)
    ids = torch.randint(0, 2, (T,), generator=g, device="cuda", dtype=torch.int32)
    got = ft.lora_add(x, a, b, ids)
    want, bound = A.lora(x[-5:], a, b, ids[-5:], None, None, BF)
    inside(got[-5:], want, bound)
    gx, ga, gb = ft.lora_backward(got, x, a, b, ids, need_b=False)
    (want, bound), _, _ = A.lora_grads(got[-5:], x[-5:], a, b, ids[-5:], None, None)
    inside(gx[-5:], want, bound)
    a2, b2 = randn(g, 2, 8, N).to(BF), randn(g, 2, K, 8).to(BF)
    out = ft.lora_add(got, a2, b2, ids, out_dtype=F32)
    inside(out[-5:], *A.lora(got[-5:], a2, b2, ids[-5:], None, None, F32))


def test_refusals(ft):
    g, x, a, b, ids, scales = make(dict(T=8, k=2, L=3, R=16, K=64, N=64), BF)
    bad = [dict(a=a[:, :12].contiguous()), dict(a=a.half()), dict(b=b[:2].contiguous()), dict(ids=ids.long()), dict(x=x[:5].contiguous()),
           dict(scales=scales[:2].contiguous()), dict(x=x.float()), dict(add=torch.zeros(8, 2, 63, device="cuda", dtype=BF)),
           dict(out_dtype=HF), dict(x=x.cpu())]
    for kw in bad:
        args = dict(x=x, a=a, b=b, ids=ids, scales=scales)
        args.update(kw)
        with pytest.raises((ValueError, TypeError)):
            ft.lora_add(args.pop("x"), args.pop("a"), args.pop("b"), args.pop("ids"), **args)
    with pytest.raises(ft.FtError):      # 60 columns
        ft.lora_add(x[:, :60].contiguous(), a[:, :, :60].contiguous(), b, ids)
    with pytest.raises(ft.FtError):      # rank 4
        ft.lora_add(x, a[:, :4].contiguous(), b[:, :, :4].contiguous(), ids)
    with pytest.raises(ft.FtError):
        ft.lora_backward(torch.zeros(8, 2, 64, device="cuda", dtype=BF), x, a, b, ids, need_x=False, need_a=False, need_b=False)
    with pytest.raises(TypeError):
        ft.lora_backward(torch.zeros(8, 2, 64, device="cuda"), x, a, b, ids)
