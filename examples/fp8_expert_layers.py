"""Expert layers in FP8, from a checkpoint's matrices to decoded tokens.

Matrices are cast to e4m3 with one scale per 128 x 128 block, as FP8 checkpoints hold them.
A prompt goes through two layers in one call each; the same layer is then put together from
the operators that the call is made of, with a dense shared expert beside the routed ones; and
decoding steps run from a CUDA graph.

    python examples/fp8_expert_layers.py [--tokens 512] [--hidden 2048] [--inter 768] [--experts 64] [--top-k 8]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_quantized_moe_quantize_gb300 as ft  # noqa: E402


def to_fp8_blocks(w):
    """[..., N, K] -> (e4m3 codes, fp32 scale of every 128 x 128 block)."""
    *lead, N, K = w.shape
    nb, kb = -(-N // 128), -(-K // 128)
    p = torch.nn.functional.pad(w.float(), (0, kb * 128 - K, 0, nb * 128 - N)).view(*lead, nb, 128, kb, 128)
    scale = (p.abs().amax((-3, -1)) / 448).clamp(min=1e-12)
    q = (p / scale[..., :, None, :, None]).reshape(*lead, nb * 128, kb * 128)[..., :N, :K]
    return q.to(torch.float8_e4m3fn).contiguous(), scale.contiguous()


class Layer:
    def __init__(self, hidden, inter, experts, top_k, g):
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda") * 0.02      # noqa: E731
        self.top_k = top_k
        self.router = rand(hidden, experts).to(torch.bfloat16)
        self.w13, self.s13 = to_fp8_blocks(rand(experts, 2 * inter, hidden))
        self.w2, self.s2 = to_fp8_blocks(rand(experts, hidden, inter))
        self.shared13, self.shared_s13 = to_fp8_blocks(rand(2 * inter, hidden))
        self.shared2, self.shared_s2 = to_fp8_blocks(rand(hidden, inter))

    def __call__(self, x):
        """x plus its experts' sum, in one call."""
        return x + ft.moe_layer_fp8(x, x @ self.router, self.w13, self.s13, self.w2, self.s2, self.top_k, ft.ACT_SILU)[0]

    def with_shared_expert(self, x):
        """The routed experts' sum plus a dense expert's row, operator by operator."""
        ids, weights = ft.moe_gate(x @ self.router, self.top_k)
        xq, xs = ft.quantize_fp8(x)
        d = ft.matmul_fp8_fp8(self.shared13, self.shared_s13, xq, xs)
        d = ft.matmul_fp8_fp8(self.shared2, self.shared_s2, *ft.act_mul_quantize_fp8(d, ft.ACT_SILU), out_dtype=x.dtype)
        h = ft.moe_fp8_fp8(self.w13, self.s13, xq, xs, ids)
        a, s = ft.act_mul_quantize_fp8(h.view(-1, h.shape[2]), ft.ACT_SILU)
        rows = ft.moe_fp8_fp8_slots(self.w2, self.s2, a, s, ids, out_dtype=torch.bfloat16)
        return ft.moe_combine(rows, weights, add=d), d


def main(argv=None):
    p = argparse.ArgumentParser()
    for name, value in (("tokens", 512), ("hidden", 2048), ("inter", 768), ("experts", 64), ("top-k", 8)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args(argv)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    layers = [Layer(a.hidden, a.inter, a.experts, a.top_k, g) for _ in range(2)]
    x = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").to(torch.bfloat16)

    y = x
    for layer in layers:
        y = layer(y)
    one = ft.moe_layer_fp8(x, x @ layers[0].router, layers[0].w13, layers[0].s13, layers[0].w2, layers[0].s2, a.top_k)[0]
    both, shared = layers[0].with_shared_expert(x)
    apart = float(((both.float() - shared.float()) - one.float()).norm() / one.float().norm())

    token = y[-1:].clone()
    graph = torch.cuda.CUDAGraph()
    layers[0](token)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = layers[1](layers[0](token))
    eager = layers[1](layers[0](token))
    graph.replay()
    torch.cuda.synchronize()
    same = torch.equal(out, eager)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(100):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"{a.tokens} tokens through two layers: rms {float(y.float().square().mean().sqrt()):.3f}")
    print(f"one call against its operators: relative distance {apart:.1e}")
    print(f"decoding from a graph: {start.elapsed_time(end) * 10:.1f} us a step of two layers, the eager call's bits: {same}")
    if ft.read_device_error():
        raise RuntimeError("an expert id was out of range")
    return apart, same


if __name__ == "__main__":
    main()
