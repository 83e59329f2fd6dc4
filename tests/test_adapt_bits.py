"""The inputs of adapt_bits.py tell two bf16 parts of a value from three (CPU)."""

import torch

import adapt_bits as D


def test_digits_are_what_the_products_make():
    d, diff = D.numbers(torch.Generator().manual_seed(1), 500, "cpu")
    w = D.wide(d)
    for dtype in (torch.bfloat16, torch.float16):
        assert torch.equal(w.to(dtype).float(), w) and torch.equal(torch.tensor(D.DIGITS).to(dtype).float(), torch.tensor(D.DIGITS))
    assert torch.equal((w.double() * torch.tensor(D.DIGITS).double()).sum(-1), D.value(d))
    assert torch.equal(D.value(d[0]) - D.value(d[1]), diff)
    assert D.value(d).max() < 2.0 ** 23 and D.value(d).min() >= 2.0 ** 22


def test_two_parts_lose_what_three_keep():
    d, diff = D.numbers(torch.Generator().manual_seed(2), 500, "cpu")
    v = D.value(d)
    assert torch.equal(D.parts(v[0], 3) - D.parts(v[1], 3), diff)
    lost = (D.parts(v[0], 2) - D.parts(v[1], 2)) != diff
    assert lost.double().mean() > 0.9
