"""GB300 (sm_103a) routed Q4_0 x Q8_1 MoE expert matmul.

The computation lives in ``libft_moe.so`` (hand-written CUDA, C ABI in
``include/ft_moe.h``); this package is its thin Python binding plus the seeded
synthetic-input generator used by the tests and the benchmark.

    act = quantize_q8_1(x_fp16)                       # fp16 [T, K] -> Q8_1
    out = moe_q4_0_q8_1(weights_q4_0, act, topk_ids)  # fp32 [T, k, N]
    out = moe_q4_0_fp16(weights_q4_0, x_fp16, topk_ids)  # the same, from fp16 (one launch when decoding)
    a2 = act_mul_quantize_q8_1(out, ACT_SILU)         # Q8_1 of silu(gate) * up per slot
    y, h, a2 = moe_ffn_q4_0_q8_1(w13, w2, act, topk_ids, ACT_SILU)   # both expert layers

and of expert layers whose matrices are e4m3 with a scale per block of 128:

    ids, w = moe_gate(logits, top_k)                   # router: experts and weights of each token
    q, s = quantize_fp8(x)                             # rows -> e4m3 codes and scales
    rows = moe_fp8_fp8(weights, w_scales, q, s, ids)   # [T, k, N]
    y = moe_combine(rows, w)                           # weighted sum of each token's rows
    y, ids, w = moe_layer_fp8(x, logits, w13, s13, w2, s2, top_k)    # the whole layer

and of what adapts a layer whose matrices stay as they are, the router and low-rank adapters:

    rows = lora_add(x, a, b, ids, scales=s, add=rows)              # an adapter per expert, or per request
    loss, counts, scale = moe_balance_loss(logits, ids)            # how unevenly the experts are loaded
    d_rows, d_w = moe_combine_backward(dy, rows, w)                # gradients of moe_combine
    dx, da, db = lora_backward(d_rows.to(x.dtype), x, a, b, ids, scales=s)     # of lora_add
    d_logits = moe_gate_backward(logits, ids, d_w, counts=counts, seq_scale=scale, grad_loss=g)   # of router and loss

No call is an autograd function: what it returns has no graph, whether an input wants a gradient or not.
"""

from ._lib import (ACT_GELU_TANH, ACT_SILU, FT_DEVERR_BAD_EXPERT_ID, FT_DEVERR_WAIT_TIMEOUT,
                   FT_DEVERR_WORKSPACE_GUARD, FT_PATH_AUTO, FT_PATH_GEMM, FT_PATH_GEMV, FT_PATH_GEMV_DP4A, FtError,
                   act_mul_quantize_fp8, act_mul_quantize_q8_1, block_dots, debug_stream_read, debug_wait_timeout, ffn_reserve, last_error, load,
                   lora_add, lora_backward,
                   matmul_fp8_fp8, moe_balance_loss, moe_combine, moe_combine_backward, moe_fp8_fp8, moe_fp8_fp8_slots, moe_gate, moe_gate_backward,
                   moe_layer_fp8, quantize_fp8,
                   moe_ffn_q4_0_q8_1, moe_gguf_q8_1, moe_q4_0_fp16, moe_q4_0_q8_1, moe_q4_0_q8_1_act, moe_q4_0_q8_1_ep,
                   moe_q4_0_q8_1_slots, profile_enable,
                   profile_read, quantize_q8_1, read_device_error, repack_q4_0_soa, release, reserve, route_offsets, selected_path,
                   set_path, workspace_bytes, WEIGHT_TYPES)

__all__ = [
    "ACT_GELU_TANH", "ACT_SILU", "WEIGHT_TYPES", "moe_gguf_q8_1", "repack_q4_0_soa", "act_mul_quantize_q8_1", "moe_ffn_q4_0_q8_1", "moe_q4_0_q8_1_act", "ffn_reserve", "moe_q4_0_fp16", "FT_DEVERR_BAD_EXPERT_ID", "FT_DEVERR_WAIT_TIMEOUT", "FT_DEVERR_WORKSPACE_GUARD", "debug_wait_timeout", "debug_stream_read", "FT_PATH_AUTO", "FT_PATH_GEMM", "FT_PATH_GEMV", "FT_PATH_GEMV_DP4A", "FtError",
    "block_dots", "last_error", "load", "moe_q4_0_q8_1", "moe_q4_0_q8_1_ep", "moe_q4_0_q8_1_slots", "profile_enable", "profile_read", "quantize_q8_1", "read_device_error", "release", "reserve",
    "act_mul_quantize_fp8", "matmul_fp8_fp8", "moe_combine", "moe_fp8_fp8", "moe_fp8_fp8_slots", "moe_gate", "moe_layer_fp8", "quantize_fp8",
    "lora_add", "lora_backward", "moe_balance_loss", "moe_combine_backward", "moe_gate_backward",
    "route_offsets", "selected_path", "set_path", "workspace_bytes",
]
