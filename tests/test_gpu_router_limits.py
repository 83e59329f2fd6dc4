"""The router's gradient where reciprocals of vanishing sums meet large gradients, as a scaled loss gives them."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import adapt_ref as A  # noqa: E402
from adapt_ref import inside  # noqa: E402


@pytest.fixture(scope="module")
def ft():
    import bit_quantized_moe_quantize_gb300 as ft
    from bit_quantized_moe_quantize_gb300 import build
    build.build()
    ft.load()
    ft.read_device_error()
    yield ft
    assert ft.read_device_error() == 0


def rows(E, n, seed=1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g, torch.randn(n, E, generator=g, device="cuda")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k", [(5, 1), (128, 1), (128, 8), (700, 2)])
@pytest.mark.parametrize("grad", [2.0 ** 22, 2.0 ** 40])
def test_padding_beside_a_large_gradient_of_the_loss(ft, score, dtype, E, k, grad):
    """One row that counts and rows of padding, masked by -inf and by NaN: the sum of a padding row's scores is 0."""
    g, x = rows(E, 4)
    x[1], x[2, :], x[3, 1:] = -math.inf, math.nan, -math.inf
    x = x.to(dtype)
    off = torch.tensor([0, 3, 4], dtype=torch.int32, device="cuda")
    ids = torch.arange(k, dtype=torch.int32, device="cuda").repeat(4, 1)
    ids[1:3] = -1
    ids[3, 1:] = -1
    _, counts, scale = ft.moe_balance_loss(x, ids, score=score, seq_offsets=off)
    gl = torch.tensor(grad, device="cuda")
    gw = torch.randn(4, k, generator=g, device="cuda")
    for w in (None, gw):
        got = ft.moe_gate_backward(x, ids, w, score=score, counts=counts, seq_scale=scale, grad_loss=gl, seq_offsets=off)
        assert not got[1].any() and not got[2].any() and not got[3, 1:].any(), got
        inside(got, *A.gate_grad(x, ids, w, score, True, 1.0, (counts, scale, gl, off)))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("grad", [math.inf, math.nan])
def test_padding_beside_a_gradient_that_is_no_number(ft, score, grad):
    _, x = rows(24, 70)
    x[::3] = -math.inf
    ids = torch.tensor([[0, 5]], dtype=torch.int32, device="cuda").repeat(70, 1)
    ids[::3] = -1
    _, counts, scale = ft.moe_balance_loss(x, ids, score=score)
    got = ft.moe_gate_backward(x, ids, torch.ones(70, 2, device="cuda"), score=score, counts=counts, seq_scale=scale,
                               grad_loss=torch.tensor(grad, device="cuda"))
    assert not got[::3].any() and not torch.isfinite(got[1::3]).any()


@pytest.mark.parametrize("grad", [1.0, 2.0 ** 30])
def test_loss_of_scores_below_the_smallest_divisor(ft, grad):
    """Sigmoid scores e^-75: their sum is under 1e-30, which divides them, and 1e30 times the loss' gradient is out of range."""
    g, x = rows(128, 6)
    x = x * 0.25 - 75.0
    x[2, ::3] = -math.inf
    ids = torch.tensor([[3, 4]], dtype=torch.int32, device="cuda").repeat(6, 1)
    _, counts, scale = ft.moe_balance_loss(x, ids, score="sigmoid")
    gl = torch.tensor(grad, device="cuda")
    got = ft.moe_gate_backward(x, ids, None, score="sigmoid", counts=counts, seq_scale=scale, grad_loss=gl)
    # |l| < 77 gives the exponential 120 roundings, and some 20 follow: within the 256 that the bound has
    inside(got, *A.gate_grad(x, ids, None, "sigmoid", True, 1.0, (counts, scale, gl, None)))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("k", [2, 40])
@pytest.mark.parametrize("renorm", [True, False])
def test_large_gradients_of_weights_without_a_score(ft, score, k, renorm):
    """Chosen experts whose scores are 0 in fp32: the smallest divisor's 1e30 times their gradients is out of range."""
    _, x = rows(64, 5)
    x -= 250.0
    if score == "softmax":
        x[:, 63] = 1.0
    x[4] = torch.linspace(-3, 3, 64, device="cuda")      # an ordinary row among them
    ids = torch.arange(k, dtype=torch.int32, device="cuda").repeat(5, 1)
    gw = torch.linspace(-1e10, 2e10, k, device="cuda").repeat(5, 1)
    got = ft.moe_gate_backward(x, ids, gw, score=score, renormalize=renorm)
    want, bound = A.gate_grad(x, ids, gw, score, renorm, 1.0)
    inside(got, want, bound)
