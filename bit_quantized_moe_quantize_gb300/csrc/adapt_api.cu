// C entry points of the operators that adapt a layer of quantized experts: the router's training and
// low-rank adapters.  Argument checks, the layout of the caller's workspace, the order of the kernels;
// include/ft_moe.h has the contract.
#include <cuda_runtime.h>

#include "../../include/ft_moe.h"
#include "api_checks.h"
#include "ft_internal.h"

namespace ft {
namespace {

int check_router(int64_t tokens, int32_t n_experts, int32_t top_k, int32_t dtype, int64_t row_stride, int32_t score,
                 const int32_t* offsets, int32_t n_seqs) {
    int64_t n;
    if (int st = check_slots(tokens, top_k, n_experts, &n)) return st;
    if (!dtype_bytes(dtype)) return fail(FT_ERR_ARG, "unknown logits type %d", dtype);
    if (score != FT_SCORE_SOFTMAX && score != FT_SCORE_SIGMOID) return fail(FT_ERR_ARG, "unknown score %d", score);
    if (row_stride < n_experts) return fail(FT_ERR_ARG, "row_stride must be >= n_experts");
    if (!mul_ok(tokens, row_stride, &n)) return fail(FT_ERR_SIZE, "tokens * row_stride overflows");
    if (n_seqs < 1 || (!offsets && n_seqs != 1))
        return fail(FT_ERR_ARG, "n_seqs must be >= 1, and 1 without seq_offsets (got %d)", n_seqs);
    if (!aligned(offsets, 4)) return fail(FT_ERR_ALIGN, "seq_offsets must be aligned to its elements");
    return FT_OK;
}

}  // namespace
}  // namespace ft

using namespace ft;

extern "C" {

size_t ft_moe_balance_workspace_bytes(int64_t tokens, int32_t n_experts, int32_t n_seqs) {
    clear_error();
    int64_t n;
    if (check_slots(tokens, 1, n_experts, &n) || n_seqs < 1) return 0;
    return balance_workspace(tokens, n_experts, n_seqs);
}

int ft_moe_balance_loss(const void* logits, int32_t dtype, int64_t row_stride, const int32_t* topk_ids,
                        const int32_t* seq_offsets, float* loss, int32_t* counts, float* seq_scale, int64_t tokens,
                        int32_t n_experts, int32_t top_k, int32_t score, int32_t n_seqs, void* workspace,
                        size_t workspace_bytes, void* stream) {
    clear_error();
    if (int st = check_router(tokens, n_experts, top_k, dtype, row_stride, score, seq_offsets, n_seqs)) return st;
    if (!loss || !counts || !seq_scale || (tokens > 0 && (!logits || !topk_ids))) return fail(FT_ERR_ARG, "null pointer");
    if (!aligned(logits, dtype_bytes(dtype)) || !aligned(topk_ids, 4) || !aligned(loss, 4) || !aligned(counts, 4) ||
        !aligned(seq_scale, 4))
        return fail(FT_ERR_ALIGN, "logits, topk_ids, loss, counts and seq_scale must be aligned to their elements");
    if (int st = check_workspace(workspace, workspace_bytes, balance_workspace(tokens, n_experts, n_seqs))) return st;
    uint32_t* err = nullptr;
    if (int st = fp8_error_word(&err)) return st;
    const BalanceParams p{tokens, n_experts, top_k, score, n_seqs};
    return launch_balance(p, logits, dtype, row_stride, topk_ids, seq_offsets, loss, counts, seq_scale,
                          static_cast<uint8_t*>(workspace), err, static_cast<cudaStream_t>(stream));
}

int ft_moe_gate_backward(const void* logits, int32_t dtype, int64_t row_stride, const int32_t* topk_ids,
                         const float* grad_weights, const int32_t* counts, const float* seq_scale, const float* grad_loss,
                         const int32_t* seq_offsets, void* grad_logits, int64_t tokens, int32_t n_experts, int32_t top_k,
                         int32_t score, int32_t renormalize, float scale, int32_t n_seqs, void* stream) {
    clear_error();
    if (int st = check_router(tokens, n_experts, top_k, dtype, row_stride, score, seq_offsets, n_seqs)) return st;
    const int parts = (counts ? 1 : 0) + (seq_scale ? 1 : 0) + (grad_loss ? 1 : 0);
    if (parts != 0 && parts != 3) return fail(FT_ERR_ARG, "counts, seq_scale and grad_loss come together");
    if (tokens == 0) return FT_OK;
    if (!grad_weights && !parts) return fail(FT_ERR_ARG, "no gradient arrives: grad_weights and grad_loss are null");
    if (!logits || !grad_logits || (grad_weights && !topk_ids)) return fail(FT_ERR_ARG, "null pointer");
    if (!aligned(logits, dtype_bytes(dtype)) || !aligned(grad_logits, dtype_bytes(dtype)) || !aligned(topk_ids, 4) ||
        !aligned(grad_weights, 4) || !aligned(counts, 4) || !aligned(seq_scale, 4) || !aligned(grad_loss, 4))
        return fail(FT_ERR_ALIGN, "logits, gradients, topk_ids, counts and seq_scale must be aligned to their elements");
    uint32_t* err = nullptr;
    if (int st = fp8_error_word(&err)) return st;
    const GateGradParams p{tokens, n_experts, top_k, score, renormalize, n_seqs, scale, topk_ids, grad_weights, counts,
                           seq_scale, grad_loss, seq_offsets};
    return launch_gate_grad(p, logits, dtype, row_stride, grad_logits, err, static_cast<cudaStream_t>(stream));
}

int ft_moe_combine_backward(const void* grad_y, int32_t y_dtype, const void* rows, int32_t rows_dtype,
                            const float* topk_weights, void* grad_rows, float* grad_weights, int64_t tokens, int32_t top_k,
                            int64_t ncols, void* stream) {
    clear_error();
    if (tokens < 0) return fail(FT_ERR_ARG, "tokens must be >= 0 (got %lld)", (long long)tokens);
    if (top_k < 1) return fail(FT_ERR_ARG, "top_k must be >= 1 (got %d)", top_k);
    if (ncols <= 0) return fail(FT_ERR_ARG, "ncols must be > 0 (got %lld)", (long long)ncols);
    if (rows_dtype != FT_DTYPE_F32 && rows_dtype != FT_DTYPE_BF16)
        return fail(FT_ERR_ARG, "rows_dtype must be FT_DTYPE_F32 or FT_DTYPE_BF16 (got %d)", rows_dtype);
    if (!dtype_bytes(y_dtype)) return fail(FT_ERR_ARG, "unknown element type %d", y_dtype);
    int64_t n;
    if (!mul_ok(tokens, top_k, &n) || n > INT32_MAX || !mul_ok(n, ncols, &n))
        return fail(FT_ERR_SIZE, "tokens * top_k must be < 2^31 and the rows' size must not overflow");
    if (tokens == 0) return FT_OK;
    if (!grad_rows && !grad_weights) return fail(FT_ERR_ARG, "grad_rows and grad_weights are both null");
    if (!grad_y || !topk_weights || !rows) return fail(FT_ERR_ARG, "null pointer");
    if (!aligned(rows, dtype_bytes(rows_dtype)) || !aligned(grad_rows, dtype_bytes(rows_dtype)) ||
        !aligned(grad_y, dtype_bytes(y_dtype)) || !aligned(topk_weights, 4) || !aligned(grad_weights, 4))
        return fail(FT_ERR_ALIGN, "grad_y, rows, weights and their gradients must be aligned to their elements");
    return launch_combine_grad(grad_y, y_dtype, rows, rows_dtype, topk_weights, grad_rows, grad_weights, tokens, top_k, ncols,
                               static_cast<cudaStream_t>(stream));
}

}  // extern "C"
