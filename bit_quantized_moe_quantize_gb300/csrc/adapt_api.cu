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

// ------------------------------------------------------- low-rank adapters
// Slots per adapter on average that go by tiles of 16 slots, and from how many on by tiles of 128; else of 64.  From a
// graph, 128 adapters of rank 8 with 8, 16, 32 slots each: 30, 30, 38 us by 16, 32, 33, 36 by 64; gradients of 64 of rank
// 64 with 16, 32 each: 163, 181 against 171, 177.  Gradients, rank 64, 256, 512, 8192 slots each: 206, 188, 156 us by 64,
// 236, 181, 144 by 128; rank 16 forward has the same times by either.  Above rank 64 the registers hold no 128 slots.
// The mean is over all adapters of the call, as the host does not know which have slots: 8191 slots of 12 among 128 or 512 adapters
// take 67 and 86 us where 12 alone take 58.
constexpr int32_t kLoraSmallMean = 16;
constexpr int64_t kLoraWideMean = 512;

struct LoraShape {
    int64_t tokens, n_slots, ncols, nrows;
    int32_t top_k, n_adapters, rank;
};

int check_lora(int64_t tokens, int32_t top_k, int32_t n_adapters, int32_t rank, int64_t ncols, int64_t nrows, LoraShape* h) {
    if (tokens < 0) return fail(FT_ERR_ARG, "tokens must be >= 0 (got %lld)", (long long)tokens);
    if (top_k < 1) return fail(FT_ERR_ARG, "top_k must be >= 1 (got %d)", top_k);
    if (n_adapters < 1 || n_adapters > FT_MAX_EXPERTS)
        return fail(FT_ERR_ARG, "n_adapters must be in [1, %d] (got %d)", FT_MAX_EXPERTS, n_adapters);
    if (rank < 8 || rank > FT_MAX_LORA_RANK || rank % 8 != 0)
        return fail(FT_ERR_ARG, "rank must be a multiple of 8 in [8, %d] (got %d)", FT_MAX_LORA_RANK, rank);
    if (ncols <= 0 || ncols % 8 != 0 || nrows <= 0 || nrows % 8 != 0)
        return fail(FT_ERR_ARG, "ncols and nrows must be positive multiples of 8 (got %lld, %lld)", (long long)ncols, (long long)nrows);
    if (ncols > FT_MAX_NCOLS || nrows > FT_MAX_NCOLS)
        return fail(FT_ERR_SIZE, "ncols and nrows must be <= %d (got %lld, %lld)", FT_MAX_NCOLS, (long long)ncols, (long long)nrows);
    int64_t n;
    if (!mul_ok(tokens, top_k, &n) || n > INT32_MAX) return fail(FT_ERR_SIZE, "tokens * top_k = %lld * %d must be < 2^31", (long long)tokens, top_k);
    *h = LoraShape{tokens, n, ncols, nrows, top_k, n_adapters, rank};
    return FT_OK;
}

// Slots of a tile.
int lora_width(int64_t n_slots, int32_t n_adapters, int32_t rank) {
    if (n_slots <= kLoraSmallMean * n_adapters) return 16;
    return n_slots < kLoraWideMean * n_adapters || rank > 64 ? 64 : 128;
}

int64_t lora_tiles(int64_t n_slots, int32_t n_adapters, int width) {
    const int64_t some = n_slots < n_adapters ? n_slots : n_adapters;      // adapters that can have a tile that is not full
    return (n_slots + some * (width - 1)) / width;
}

// Chunks of the matrices' gradients, beside one more for each adapter: a CTA per SM, each with 256 columns.  The workspace, whose
// size is asked for without a device, has room for those of kLoraGradSms; a call makes them for the SMs that there are.
constexpr int64_t kLoraGradSms = 152;
int64_t lora_most_chunks(int64_t ncols, int64_t nrows, int64_t sms) {
    const int64_t chunks = sms / ((ncols + 255) / 256 + (nrows + 255) / 256);
    return chunks > 0 ? chunks : 1;
}

// Slots of a chunk: whole stages of 32, and no less than 64: what is left to join grows, the chain of stages shrinks.  From a
// graph, 509 slots of 6 adapters, rank 24, fp16: 32 us, of one adapter 32; with 256 at least 34 and 42, with 32 32 and 31; 512 of 4, rank
// 128, bf16: 39, 40, 42.
constexpr int64_t kLoraLeastChunk = 64;
int32_t lora_chunk(int64_t n_slots, int64_t most) {
    const int64_t slots = (n_slots + most - 1) / most;
    return static_cast<int32_t>(slots < kLoraLeastChunk ? kLoraLeastChunk : (slots + 31) / 32 * 32);
}

struct LoraWs {
    Fp8Order order;
    size_t u, v, u_parts, v_parts, rows, present, parts_a, parts_b, total;
    int width;
    int64_t n_tiles;
};

// rows: of the gradient of x, where slots share a row of x.
LoraWs lora_ws(uint8_t* base, const LoraShape& h, bool backward, bool share) {
    LoraWs L{};
    const size_t S = static_cast<size_t>(h.n_slots), R = static_cast<size_t>(h.rank);
    size_t at = 0;
    L.width = lora_width(h.n_slots, h.n_adapters, h.rank);
    L.n_tiles = lora_tiles(h.n_slots, h.n_adapters, L.width);
    if (!backward && h.n_slots <= kLoraFewSlots) return L;      // needs none
    at = al256(fp8_order_layout(base, h.n_slots, h.n_adapters, false, &L.order));
    L.u = take_bytes(&at, S * R * 4);
    if (backward) {
        L.v = take_bytes(&at, S * R * 4);
        const size_t lines = static_cast<size_t>(lora_part_kinds(h.rank)) * S * 128;
        L.u_parts = take_bytes(&at, lines);
        L.v_parts = take_bytes(&at, lines);
        const int64_t most = lora_most_chunks(h.ncols, h.nrows, kLoraGradSms), all = h.n_slots / kLoraLeastChunk;
        const size_t chunks = static_cast<size_t>((all < most ? all : most) + h.n_adapters);      // rises with the slots
        L.parts_a = take_bytes(&at, chunks * R * h.ncols * 4);
        L.parts_b = take_bytes(&at, chunks * R * h.nrows * 4);
        if (share) {
            L.rows = take_bytes(&at, S * h.ncols * 4);
            L.present = take_bytes(&at, S * 4);
        }
    }
    L.total = at;
    return L;
}

// The most that lora_ws gives for up to h.tokens tokens: what it needs rises with them but where the tiles' width, the
// order's scratch or the chunks change.
size_t lora_most(const LoraShape& h, bool backward, bool share) {
    size_t most = 0;
    auto take = [&](int64_t tokens) {
        if (tokens < 0 || tokens > h.tokens) return;
        LoraShape x = h;
        x.tokens = tokens;
        x.n_slots = tokens * h.top_k;
        const size_t n = lora_ws(nullptr, x, backward, share).total;
        most = n > most ? n : most;
    };
    take(h.tokens);
    take(static_cast<int64_t>(kLoraSmallMean) * h.n_adapters / h.top_k);
    take((kLoraWideMean * h.n_adapters - 1) / h.top_k);
    take(kFastRouteSlots / h.top_k);
    return most;
}

LoraPlan lora_plan(const LoraShape& h, const LoraWs& L, const int32_t* ids, const float* scales, uint32_t* err, bool backward) {
    LoraPlan p{};
    p.ids = ids;
    p.offsets = L.order.offsets;
    p.tiles = L.order.tiles;
    p.perm = L.order.perm;
    p.scales = scales;
    p.n_slots = static_cast<int32_t>(h.n_slots);
    p.n_adapters = h.n_adapters;
    p.rank = h.rank;
    p.width = L.width;
    p.n_tiles = L.n_tiles;
    if (backward) {
        const int64_t sms = sm_count();
        p.chunk = lora_chunk(h.n_slots, lora_most_chunks(h.ncols, h.nrows, sms < kLoraGradSms ? sms : kLoraGradSms));
    }
    p.err = err;
    p.down_jobs = backward ? 2 : 1;
    p.down_cols = static_cast<int32_t>(backward && h.nrows > h.ncols ? h.nrows : h.ncols);
    return p;
}

int check_lora_type(int32_t dtype) {
    if (dtype != FT_DTYPE_F16 && dtype != FT_DTYPE_BF16)
        return fail(FT_ERR_ARG, "dtype must be FT_DTYPE_F16 or FT_DTYPE_BF16 (got %d)", dtype);
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

size_t ft_lora_workspace_bytes(int64_t tokens, int32_t top_k, int32_t n_adapters, int32_t rank, int64_t ncols, int64_t nrows,
                               int32_t backward) {
    clear_error();
    LoraShape h;
    if (check_lora(tokens, top_k, n_adapters, rank, ncols, nrows, &h)) return 0;
    return lora_most(h, backward != 0, top_k > 1);
}

int ft_lora_add(const void* x, int32_t dtype, const void* a, const void* b, const float* scales, const int32_t* ids,
                const void* add, void* out, int32_t out_dtype, int64_t tokens, int32_t top_k, int32_t x_per_slot,
                int32_t n_adapters, int32_t rank, int64_t ncols, int64_t nrows, void* workspace, size_t workspace_bytes,
                void* stream) {
    clear_error();
    LoraShape h;
    if (int st = check_lora(tokens, top_k, n_adapters, rank, ncols, nrows, &h)) return st;
    if (int st = check_lora_type(dtype)) return st;
    if (out_dtype != FT_DTYPE_F32 && out_dtype != dtype)
        return fail(FT_ERR_ARG, "out_dtype must be FT_DTYPE_F32 or the adapters' type (got %d)", out_dtype);
    if (tokens == 0) return FT_OK;
    if (!x || !a || !b || !ids || !out) return fail(FT_ERR_ARG, "null pointer");
    if (!aligned(x, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(add, 16) || !aligned(out, 16))
        return fail(FT_ERR_ALIGN, "x, a, b, add and out must be 16-byte aligned");
    if (!aligned(scales, 4) || !aligned(ids, 4)) return fail(FT_ERR_ALIGN, "scales and ids must be aligned to their elements");
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const LoraWs L = lora_ws(ws, h, false, false);
    if (int st = check_workspace(workspace, workspace_bytes, L.total)) return st;
    uint32_t* err = nullptr;
    if (int st = fp8_error_word(&err)) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const LoraPlan p = lora_plan(h, L, ids, scales, err, false);
    const bool f32 = out_dtype == FT_DTYPE_F32;
    if (h.n_slots <= kLoraFewSlots)
        return launch_lora_few(LoraFew{x, a, b, add, out, static_cast<int32_t>(ncols), static_cast<int32_t>(nrows), x_per_slot ? 1 : top_k, f32},
                               p, dtype, s);
    if (int st = launch_lora_order(ids, h.n_slots, n_adapters, L.width, L.order, s)) return st;
    float* u = reinterpret_cast<float*>(ws + L.u);
    const LoraDown down{x, a, u, nullptr, static_cast<int32_t>(ncols), x_per_slot ? 1 : top_k, false};
    if (int st = launch_lora_down(&down, 1, p, dtype, s)) return st;
    const LoraUp up{u, b, add, out, nullptr, static_cast<int32_t>(nrows), false, f32};
    return launch_lora_up(up, p, dtype, s);
}

int ft_lora_backward(const void* grad_out, const void* x, int32_t dtype, const void* a, const void* b, const float* scales,
                     const int32_t* ids, const void* add, void* grad_x, float* grad_a, float* grad_b, int64_t tokens,
                     int32_t top_k, int32_t x_per_slot, int32_t n_adapters, int32_t rank, int64_t ncols, int64_t nrows,
                     void* workspace, size_t workspace_bytes, void* stream) {
    clear_error();
    LoraShape h;
    if (int st = check_lora(tokens, top_k, n_adapters, rank, ncols, nrows, &h)) return st;
    if (int st = check_lora_type(dtype)) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t size_a = static_cast<int64_t>(n_adapters) * rank * ncols * 4, size_b = static_cast<int64_t>(n_adapters) * rank * nrows * 4;
    if (!aligned(grad_x, 16) || !aligned(grad_a, 16) || !aligned(grad_b, 16))
        return fail(FT_ERR_ALIGN, "grad_x, grad_a and grad_b must be 16-byte aligned");
    if (tokens == 0) {      // sums over nothing
        cudaError_t e = cudaSuccess;
        if (grad_a) e = cudaMemsetAsync(grad_a, 0, static_cast<size_t>(size_a), s);
        if (grad_b && e == cudaSuccess) e = cudaMemsetAsync(grad_b, 0, static_cast<size_t>(size_b), s);
        return e == cudaSuccess ? FT_OK : fail(FT_ERR_CUDA, "cudaMemsetAsync: %s", cudaGetErrorString(e));
    }
    if (!grad_x && !grad_a && !grad_b) return fail(FT_ERR_ARG, "grad_x, grad_a and grad_b are all null");
    if (!grad_out || !x || !a || !b || !ids) return fail(FT_ERR_ARG, "null pointer");
    if (!aligned(grad_out, 16) || !aligned(x, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(add, 16))
        return fail(FT_ERR_ALIGN, "grad_out, x, a, b and add must be 16-byte aligned");
    if (!aligned(scales, 4) || !aligned(ids, 4)) return fail(FT_ERR_ALIGN, "scales and ids must be aligned to their elements");
    const bool share = top_k > 1 && !x_per_slot;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const LoraWs L = lora_ws(ws, h, true, share);
    if (int st = check_workspace(workspace, workspace_bytes, L.total)) return st;
    uint32_t* err = nullptr;
    if (int st = fp8_error_word(&err)) return st;
    LoraPlan p = lora_plan(h, L, ids, scales, err, true);
    if (int st = launch_lora_order(ids, h.n_slots, n_adapters, L.width, L.order, s)) return st;
    float *u = reinterpret_cast<float*>(ws + L.u), *v = reinterpret_cast<float*>(ws + L.v);
    const int32_t K = static_cast<int32_t>(ncols), N = static_cast<int32_t>(nrows), div = x_per_slot ? 1 : top_k;
    LoraDown down[2];
    int n = 0;
    // the matrices' gradients take u and v as fp32 (fp16 adapters) or in parts, grad_x takes v as fp32
    const bool bf = dtype == FT_DTYPE_BF16;
    void *u_parts = ws + L.u_parts, *v_parts = ws + L.v_parts;
    if (grad_b) down[n++] = LoraDown{x, a, bf ? nullptr : u, bf ? u_parts : nullptr, K, div, false};
    if (grad_x || grad_a) down[n++] = LoraDown{grad_out, b, bf && !grad_x ? nullptr : v, bf && grad_a ? v_parts : nullptr, N, 1, true};
    if (int st = launch_lora_down(down, n, p, dtype, s)) return st;
    if (grad_x) {
        float *rows = reinterpret_cast<float*>(ws + L.rows), *present = reinterpret_cast<float*>(ws + L.present);
        const LoraUp up = share ? LoraUp{v, a, nullptr, rows, present, K, true, true}
                                : LoraUp{v, a, add, grad_x, nullptr, K, true, false};
        if (int st = launch_lora_up(up, p, dtype, s)) return st;
        p.overlap_grad = !share;
        if (share)
            if (int st = launch_combine(rows, FT_DTYPE_F32, present, add, grad_x, dtype, tokens, top_k, ncols, s)) return st;
    }
    const LoraGrad grads[2] = {LoraGrad{x, v, v_parts, grad_a, reinterpret_cast<float*>(ws + L.parts_a), K, div, false},
                               LoraGrad{grad_out, u, u_parts, grad_b, reinterpret_cast<float*>(ws + L.parts_b), N, 1, true}};
    return launch_lora_grad(grads, p, dtype, s);
}

}  // extern "C"
