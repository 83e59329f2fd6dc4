"""The README's lines on FP8 experts and on adapting them, run as they stand, and the gradients that they end with."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import adapt_ref as A  # noqa: E402
import fp8_ref as R8  # noqa: E402
import readme_code  # noqa: E402

BF = torch.bfloat16


def test_lines_run_and_their_gradients_are_right():
    import bit_quantized_moe_quantize_gb300 as ft
    from bit_quantized_moe_quantize_gb300 import build
    build.build()
    ft.read_device_error()
    T, H, I, E, R, L = 70, 256, 128, 64, 16, 5
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")      # noqa: E731
    w13, s13 = R8.weights(gen, E, 2 * I, H)
    w2, s2 = R8.weights(gen, E, H, I)
    v = dict(torch=torch, ft=ft, I=I, w13=w13, s13=s13, w2=w2, s2=s2, x_bf16=rand(T, H).to(BF), router_logits=rand(T, E), bias=rand(E) * 0.1,
             shared_expert_row=rand(T, H).to(BF), a=(rand(E, R, I) / 8).to(BF), b=(rand(E, H, R) / 4).to(BF),
             s=torch.rand(E, generator=gen, device="cuda") + 0.5, offsets=torch.tensor([0, 20, 70], dtype=torch.int32, device="cuda"),
             dy=rand(T, H), g=torch.tensor([3.0], device="cuda"), a1=(rand(L, R, H) / 16).to(BF), b1=(rand(L, H, R) / 4).to(BF),
             request_adapter=torch.randint(-1, L, (T,), generator=gen, device="cuda", dtype=torch.int32))
    exec(readme_code.part("FP8"), v)
    before = v["y"].clone()
    exec(readme_code.part("adapters"), v)
    assert ft.read_device_error() == 0
    A.inside(v["y"], *A.lora(v["x_bf16"], v["a1"], v["b1"], v["request_adapter"], None, before, BF))
    loss, _, _ = A.balance(v["router_logits"].double(), v["ids"], "sigmoid", v["offsets"])
    A.inside(v["loss"], loss, 256 * A.U32 * loss)
    A.inside(v["d_logits"], *A.gate_grad(v["router_logits"], v["ids"], v["d_weights"], "sigmoid", True, 2.5,
                                         (v["counts"], v["scale"], v["g"], v["offsets"])))
    want = R8.act_mul(v["h"].view(-1, 2 * I).double(), ft.ACT_SILU)
    # the activation in fp32, some ten roundings, and one to bf16
    A.inside(v["mid"], want, (A.U[BF] * 1.01 + 16 * A.U32) * want.abs() + A.LEAST[BF])
    grads = A.lora_grads(v["d_rows"].to(BF), v["mid"], v["a"], v["b"], v["ids"], v["s"], None)
    for name, (want, bound) in zip(("d_mid", "d_a", "d_b"), grads):
        A.inside(v[name], want, bound, name)
