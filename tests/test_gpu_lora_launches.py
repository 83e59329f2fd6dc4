"""Kernels of lora_backward that come up before the one in front of them has ended (the gradients of the matrices under the second product,
which has no tile where no slot has an adapter), call after call in the same memory."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,L,R", [(2000, 1, 16), (1500, 4, 72), (300, 40, 8)])
def test_calls_without_a_tile_between_others(dtype, T, L, R):
    import bit_quantized_moe_quantize_gb300 as ft
    from bit_quantized_moe_quantize_gb300 import build
    build.build()
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)      # noqa: E731
    a, b = rand(L, R, 512) / 16, rand(L, 768, R) / 4
    calls = []
    for kind in range(3):
        ids = torch.randint(0, L, (T,), generator=g, device="cuda", dtype=torch.int32) if kind else torch.full((T,), -1, dtype=torch.int32, device="cuda")
        calls.append((rand(T, 768), rand(T, 512), a, b, ids))
    want = []
    for c in calls:
        want.append(ft.lora_backward(*c))
        torch.cuda.synchronize()
    assert not any(t.any() for t in want[0])
    outs = [torch.empty_like(t) for t in want[0]]
    got = []
    for i in (1, 0, 2, 0, 0, 1, 2, 1, 0, 2) * 3:
        ft.lora_backward(*calls[i], grad_x=outs[0], grad_a=outs[1], grad_b=outs[2])
        got.append((i, [t.clone() for t in outs]))
    for i, r in got:
        assert all(torch.equal(p, q) for p, q in zip(r, want[i]))
