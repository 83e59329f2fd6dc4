"""The 64-bit forms that the router's gradients are tested against, against differences (CPU)."""

import math

import pytest
import torch

import adapt_ref as A


def case(seed, T=6, E=7, k=3):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, E, generator=g, dtype=torch.float64)
    x[torch.rand(T, E, generator=g) < 0.15] = -math.inf
    x[2] = -math.inf
    ids = torch.rand(T, E, generator=g).argsort(1)[:, :k].to(torch.int32)
    ids[4, 1] = ids[4, 0]                       # one that repeats
    ids[1, 0] = -1
    return g, x, ids


def directional(f, x, d):
    e = 1e-6
    return (f(x + e * d) - f(x - e * d)) / (2 * e)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gate_gradient_against_differences(score, renorm):
    g, x, ids = case(3)
    gw = torch.randn(ids.shape, generator=g, dtype=torch.float64)
    there = x > -math.inf
    d = torch.randn(x.shape, generator=g, dtype=torch.float64) * there
    ids = torch.where(there.gather(1, ids.clamp(min=0).long()), ids, -1)

    def f(v):
        return float((A.weights(v, ids, score, renorm, 1.7) * torch.where(ids >= 0, gw, 0.0)).sum())

    grad, _ = A.gate_grad(x, ids, gw, score, renorm, 1.7)
    # differences of functions of size 10 and steps of 1e-6: 2^-52 * 10 / 1e-6 from rounding, as much from the step
    assert abs(float((grad * d).sum()) - directional(f, x, d)) < 1e-7


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient_against_differences(score):
    g, x, ids = case(5, T=9)
    offsets = torch.tensor([1, 3, 3, 8], dtype=torch.int32)
    _, counts, scale = A.balance(x, ids, score, offsets)
    d = torch.randn(x.shape, generator=g, dtype=torch.float64) * (x > -math.inf)
    grad, _ = A.gate_grad(x, ids, None, score, True, 1.0, (counts, scale, torch.tensor(0.7), offsets))
    diff = directional(lambda v: 0.7 * float(A.balance(v, ids, score, offsets)[0]), x, d)
    assert abs(float((grad * d).sum()) - diff) < 1e-7
    assert (grad[0] == 0).all() and (grad[8] == 0).all() and (grad[2] == 0).all()


def test_even_load_has_loss_one():
    x = torch.zeros(8, 4, dtype=torch.float64)
    ids = torch.arange(8)[:, None].remainder(4).to(torch.int32)
    loss, counts, _ = A.balance(x, ids, "softmax", None)
    assert abs(float(loss) - 1) < 1e-12 and counts.tolist() == [[2, 2, 2, 2]]
