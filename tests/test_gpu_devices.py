"""Calls whose tensors lie on another device than the current one are refused, before anything is launched.

The current device is a fake here: the mismatched launch itself is never made."""

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


def fp8_calls(ft):
    g = R.gen(1)
    E, k, H, I, T = 4, 2, 256, 128, 6
    w13, s13 = R.weights(g, E, 2 * I, H)
    w2, s2 = R.weights(g, E, H, I)
    q, s = R.codes(g, T, H)
    qs, ss = R.codes(g, T * k, H)
    ids = R.ids(g, T, E, k)
    x = R.rows(g, T, H, torch.bfloat16)
    logits = torch.randn(T, E, generator=g, device="cuda")
    rows, wt = torch.randn(T, k, H, device="cuda"), torch.rand(T, k, device="cuda")
    return {
        "moe_gate": lambda: ft.moe_gate(logits, k),
        "quantize_fp8": lambda: ft.quantize_fp8(x),
        "act_mul_quantize_fp8": lambda: ft.act_mul_quantize_fp8(x, ft.ACT_SILU),
        "moe_fp8_fp8": lambda: ft.moe_fp8_fp8(w13, s13, q, s, ids),
        "moe_fp8_fp8_slots": lambda: ft.moe_fp8_fp8_slots(w13, s13, qs, ss, ids),
        "matmul_fp8_fp8": lambda: ft.matmul_fp8_fp8(w13[0], s13[0], q, s),
        "moe_combine": lambda: ft.moe_combine(rows, wt),
        "moe_layer_fp8": lambda: ft.moe_layer_fp8(x, logits, w13, s13, w2, s2, k),
    }


def test_fp8_calls_refuse_another_device(ft, monkeypatch):
    from bit_quantized_moe_quantize_gb300 import _lib
    calls = fp8_calls(ft)
    for call in calls.values():
        call()
    monkeypatch.setattr(_lib, "_current_device", lambda: torch.cuda.current_device() + 1, raising=False)
    for name, call in calls.items():
        with pytest.raises(ValueError, match="current device"):
            call()
            pytest.fail(f"{name} ran")


def test_quantized_calls_refuse_another_device(ft, monkeypatch):
    """The same of the calls on GGUF blocks."""
    from bit_quantized_moe_quantize_gb300 import _lib
    E, N, K, T = 4, 64, 64, 3
    w = torch.zeros(E, N, K // 32, 18, dtype=torch.uint8, device="cuda")
    x = torch.zeros(T, K, dtype=torch.float16, device="cuda")
    ids = torch.zeros(T, 2, dtype=torch.int32, device="cuda")
    act = ft.quantize_q8_1(x)
    calls = [lambda: ft.quantize_q8_1(x), lambda: ft.moe_q4_0_q8_1(w, act, ids), lambda: ft.moe_q4_0_fp16(w, x, ids),
             lambda: ft.route_offsets(ids, E), lambda: ft.moe_q4_0_q8_1_act(w, act, ids, ft.ACT_SILU)]
    for call in calls:
        call()
    monkeypatch.setattr(_lib, "_current_device", lambda: torch.cuda.current_device() + 1, raising=False)
    for call in calls:
        with pytest.raises(ValueError, match="current device"):
            call()
