"""The router on both sides of the batch size from which it changes its kernel: the same choices, ties included."""

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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("c", [(128, 1, 1, 1, 8), (129, 1, 1, 1, 3), (160, 1, 1, 1, 6), (256, 1, 1, 1, 5), (256, 1, 1, 1, 8), (256, 1, 1, 1, 9),
                               (257, 1, 1, 1, 8), (512, 1, 1, 1, 1), (512, 1, 1, 1, 17), (512, 1, 1, 1, 40),
                               (256, 8, 4, 2, 8), (256, 8, 4, 2, 9), (512, 8, 3, 2, 8), (512, 8, 3, 2, 12)])
@pytest.mark.parametrize("score,bias", [("softmax", False), ("sigmoid", True)])
def test_gate_long_batches(ft, c, dtype, score, bias):
    E, G, TG, GT, k = c
    T = 8192 + 3
    g = R.gen(E + 31 * G + k)
    logits = torch.randint(-12, 13, (T, E), generator=g, device="cuda").to(dtype) / 4
    logits = torch.where(torch.rand(T, E, generator=g, device="cuda") < 0.1, -math.inf, logits)
    logits[5], logits[77, 1:] = -math.inf, math.nan
    b = torch.randint(0, 3, (E,), generator=g, device="cuda").float() / 4 if bias else None
    args = dict(score=score, bias=b, n_groups=G, topk_groups=TG, group_top=GT, scale=2.5)
    ids, w = ft.moe_gate(logits, k, **args)
    want, ww, sure = R.gate(logits, k, score, b, G, TG, GT, True, 2.5)
    assert sure.float().mean() > 0.5
    assert torch.equal(ids[sure].long(), want[sure])
    # test_gate's bound: exp, sums, quotients and products of fp32
    assert ((w - ww).abs()[sure] <= 64 * R.U32 * ww[sure].abs() + 1e-30).all()
    assert (ids[5] == -1).all() and (w[5] == 0).all()
    # a few tokens of the same go by the other kernel where the two differ in their sizes
    part, wp = ft.moe_gate(logits[:8000], k, **args)
    assert torch.equal(part[sure[:8000]], ids[:8000][sure[:8000]])
    assert ((wp - w[:8000]).abs()[sure[:8000]] <= 64 * R.U32 * w[:8000].abs()[sure[:8000]] + 1e-30).all()
