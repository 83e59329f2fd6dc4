"""A layer of quantized experts whose router and adapters are trained, as a user runs it: every gradient of a step against
automatic differentiation in fp64, and the trained adapters served."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import adapt_ref as A  # noqa: E402
import fp8_ref as R8  # noqa: E402

BF = torch.bfloat16


@pytest.fixture(scope="module")
def ft():
    import bit_quantized_moe_quantize_gb300 as ft
    from bit_quantized_moe_quantize_gb300 import build
    build.build()
    ft.load()
    ft.read_device_error()
    yield ft
    assert ft.read_device_error() == 0


class Layer:
    """One product of each routed expert, an adapter of its own beside it, and the weighted sum."""

    def __init__(self, ft, T, H, N, E, k, R):
        g = torch.Generator(device="cuda")
        g.manual_seed(T)
        self.ft, self.k = ft, k
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")      # noqa: E731
        self.x, self.logits = rand(T, H).to(BF), rand(T, E)
        self.logits[T // 2] = -math.inf
        self.w, self.ws = R8.weights(g, E, N, H)
        self.a, self.b = (rand(E, R, H) / math.sqrt(H)).to(BF), (rand(E, N, R) / math.sqrt(R)).to(BF)
        self.scales = torch.full((E,), 2.0, device="cuda")
        cut = torch.randint(0, T, (2,), generator=g, device="cuda").sort().values
        self.offsets = torch.cat([torch.tensor([0], device="cuda"), cut, torch.tensor([T], device="cuda")]).to(torch.int32)
        self.dy = rand(T, N).to(BF)

    def forward(self):
        ft = self.ft
        self.ids, self.weights = ft.moe_gate(self.logits, self.k)
        self.loss, self.counts, self.seq_scale = ft.moe_balance_loss(self.logits, self.ids, seq_offsets=self.offsets)
        self.base = ft.moe_fp8_fp8(self.w, self.ws, *ft.quantize_fp8(self.x), self.ids, out_dtype=BF)
        self.rows = ft.lora_add(self.x, self.a, self.b, self.ids, scales=self.scales, add=self.base)
        return ft.moe_combine(self.rows, self.weights)

    def backward(self, grad_loss):
        ft = self.ft
        grad_rows, grad_weights = ft.moe_combine_backward(self.dy, self.rows, self.weights)
        grad_logits = ft.moe_gate_backward(self.logits, self.ids, grad_weights, counts=self.counts, seq_scale=self.seq_scale,
                                           grad_loss=grad_loss, seq_offsets=self.offsets)
        return (grad_logits, *ft.lora_backward(grad_rows, self.x, self.a, self.b, self.ids, scales=self.scales))


def step64(m, grad_loss):
    """The same step in fp64 from the choices and the frozen product's rows that the layer had: (y, loss, gradients)."""
    there = m.logits.double() > -math.inf
    logits = torch.where(there, m.logits.double(), 0.0).requires_grad_()
    x, a, b = (t.double().requires_grad_() for t in (m.x, m.a, m.b))
    full = torch.where(there, logits, -math.inf)
    w = A.weights(full, m.ids, "softmax", True, 1.0)
    loss, _, _ = A.balance(full, m.ids, "softmax", m.offsets)
    T, E = logits.shape
    e = m.ids.clamp(min=0).long()
    low = torch.zeros_like(m.base, dtype=torch.float64)
    for i in range(E):
        low = low + torch.where((m.ids == i)[:, :, None], ((x @ a[i].t()) @ b[i].t() * 2.0)[:, None, :], 0.0)
    rows = m.base.double() + low
    y = (torch.where(m.ids >= 0, w, 0.0)[:, :, None] * rows).sum(1)
    total = (y * m.dy.double()).sum() + grad_loss * loss
    assert e.shape == m.ids.shape
    return y, loss, torch.autograd.grad(total, (logits, x, a, b))


def far(got, want):
    return float((got.double() - want.detach()).norm() / want.detach().norm())


@pytest.mark.parametrize("size", [(37, 256, 128, 8, 2, 8), (700, 512, 264, 16, 4, 16)])
def test_training_step(ft, size):
    T, H, N, E, k, R = size
    m = Layer(ft, *size)
    y = m.forward()
    gl = torch.tensor(5.0, device="cuda")
    grads = m.backward(gl)
    wy, wloss, want = step64(m, 5.0)
    # rows, their gradients and y are rounded to bf16: 2^-8 at most each, in rows, y, rows' gradient and x's gradient
    # one after the other at most three of them, and sums keep that relative to their terms
    assert far(y, wy) < 3 * 2.0 ** -8
    assert abs(float(m.loss) - float(wloss.detach())) < 256 * A.U32 * float(wloss.detach())
    for name, got, ref in zip(("logits", "x", "a", "b"), grads, want):
        assert far(got, ref) < 4 * 2.0 ** -8, name
    assert not grads[0][T // 2].any() and (m.ids[T // 2] == -1).all()


def test_step_from_a_graph(ft):
    """Forward and backward captured together, replayed with other inputs: the eager step's bits."""
    m = Layer(ft, 300, 256, 128, 8, 2, 16)
    gl = torch.ones((), device="cuda")

    def step():
        return (m.forward(), m.loss, *m.backward(gl))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    m.x.copy_(m.x.flip(0))
    m.logits.copy_(m.logits.roll(1, 1))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in got]
    assert all(torch.equal(p, q) for p, q in zip(got, step()))


def test_requests_beside_a_dense_product(ft):
    """Requests of different adapters in one decoding batch: each gets what it would get alone."""
    m = Layer(ft, 24, 512, 256, 1, 1, 16)
    L = 5
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    a, b = torch.randn(L, 16, 512, generator=g, device="cuda").to(BF), torch.randn(L, 256, 16, generator=g, device="cuda").to(BF)
    which = (torch.arange(24, device="cuda") % (L + 1) - 1).to(torch.int32)
    base = ft.matmul_fp8_fp8(m.w[0], m.ws[0], *ft.quantize_fp8(m.x), out_dtype=BF)
    both = ft.lora_add(m.x, a, b, which, add=base)
    assert torch.equal(both[which < 0], base[which < 0])
    for t in range(24):
        alone = ft.lora_add(m.x[t:t + 1].clone(), a, b, which[t:t + 1].clone(), add=base[t:t + 1].clone())
        assert torch.equal(alone[0], both[t])
    want, bound = A.lora(m.x, a, b, which, None, base, BF)
    A.inside(both, want, bound)
