"""Inputs whose products show how many bits the narrow side of an adapter, A x or B^T dy, keeps as a matrix operand.

A value of the narrow side is a whole number of 23 bits, a 2^16 + b 2^8 + c with a < 128 and b, c < 256, as the sum of three
products.  Two of them that agree but for c meet with opposite signs, so that a result is the difference of two c: exact in
fp32, in 16 bits, and in every sum on the way, as all of them are whole numbers below 2^24 (the products, their partial
sums, three bf16 parts, two tf32 parts, and the results).  So the results have to be equal, not near.  Two bf16 parts
hold 16 bits of 23, and the difference is lost."""

import torch

# what the three digits are multiplied with on the narrow matrix' side; the first digit stands doubled on the other
DIGITS = (2.0 ** 15, 2.0 ** 8, 1.0)


def numbers(g, n, device):
    """n pairs of whole numbers that agree but for their last digit: digits [2, n, 3] and the pairs' differences [n]."""
    d = torch.randint(0, 256, (2, n, 3), generator=g, device=device)
    d[0, :, 0] = d[0, :, 0] % 128 | 64          # 23 bits, always
    d[1, :, :2] = d[0, :, :2]
    return d, (d[0, :, 2] - d[1, :, 2]).double()


def wide(d):
    """The wide side's three values of a number (each has 8 bits)."""
    return d.float() * torch.tensor([2.0, 1.0, 1.0], device=d.device)


def value(d):
    return d[..., 0].double() * 2.0 ** 16 + d[..., 1].double() * 2.0 ** 8 + d[..., 2].double()


def parts(v, n):
    """The sum of the first n bf16 parts of fp32 values, in fp64."""
    left, total = v.float(), torch.zeros_like(v, dtype=torch.float64)
    for _ in range(n):
        p = left.to(torch.bfloat16).float()
        total += p.double()
        left = left - p
    return total
