// C entry points of the FP8 expert-layer operators: argument checks, the
// layout of the caller's workspace, and the order of the kernels.  See
// include/ft_moe.h for the contract.
#include <algorithm>
#include <mutex>

#include <cuda_runtime.h>

#include "../../include/ft_moe.h"
#include "fp8_common.cuh"
#include "ft_internal.h"

namespace ft {

static __device__ uint32_t g_fp8_error;

// The word's address is looked up once per device; host code cannot use the
// symbol's name as a pointer.  Every call that can raise a flag looks it up.
int fp8_error_word(uint32_t** word, bool only_if_used) {
    constexpr int kMaxDevices = 64;
    static std::mutex mu;
    static uint32_t* at[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return fail(FT_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
    if (dev < 0 || dev >= kMaxDevices) return fail(FT_ERR_CUDA, "device ordinal %d out of range", dev);
    std::lock_guard<std::mutex> lk(mu);
    if (!at[dev] && !only_if_used) {
        void* p = nullptr;
        e = cudaGetSymbolAddress(&p, g_fp8_error);
        if (e != cudaSuccess || !p) return fail(FT_ERR_CUDA, "cudaGetSymbolAddress: %s", cudaGetErrorString(e));
        at[dev] = static_cast<uint32_t*>(p);
    }
    *word = at[dev];
    return FT_OK;
}

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 60;   // products of sizes stay far from overflow below this

bool mul_ok(int64_t a, int64_t b, int64_t* r) {
    if (a < 0 || b < 0 || (a != 0 && b > kMaxElems / a)) return false;
    *r = a * b;
    return true;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

size_t al256(size_t x) { return (x + 255) & ~size_t(255); }

int dtype_bytes(int32_t d) { return d == FT_DTYPE_F32 ? 4 : d == FT_DTYPE_F16 || d == FT_DTYPE_BF16 ? 2 : 0; }

int check_cols(int64_t ncols, const char* what) {
    if (ncols <= 0 || ncols % 16 != 0)
        return fail(FT_ERR_ARG, "%s must be a positive multiple of 16 (got %lld)", what, (long long)ncols);
    return FT_OK;
}

int check_slots(int64_t tokens, int32_t top_k, int32_t n_experts, int64_t* n_slots) {
    if (tokens < 0) return fail(FT_ERR_ARG, "tokens must be >= 0 (got %lld)", (long long)tokens);
    if (n_experts < 1 || n_experts > FT_MAX_EXPERTS)
        return fail(FT_ERR_ARG, "n_experts must be in [1, %d] (got %d)", FT_MAX_EXPERTS, n_experts);
    if (top_k < 1 || top_k > n_experts)
        return fail(FT_ERR_ARG, "top_k must be in [1, n_experts=%d] (got %d)", n_experts, top_k);
    if (!mul_ok(tokens, top_k, n_slots) || *n_slots > INT32_MAX)
        return fail(FT_ERR_SIZE, "tokens * top_k = %lld * %d must be < 2^31", (long long)tokens, top_k);
    return FT_OK;
}

int check_gate(int64_t tokens, int32_t n_experts, int32_t top_k, int32_t score, int32_t n_groups, int32_t topk_groups,
               int32_t group_top, int32_t dtype, int64_t row_stride, int64_t* n_slots) {
    if (int st = check_slots(tokens, top_k, n_experts, n_slots)) return st;
    if (!dtype_bytes(dtype)) return fail(FT_ERR_ARG, "unknown logits type %d", dtype);
    if (score != FT_SCORE_SOFTMAX && score != FT_SCORE_SIGMOID) return fail(FT_ERR_ARG, "unknown score %d", score);
    if (n_groups < 1 || n_experts % n_groups != 0)
        return fail(FT_ERR_ARG, "n_groups must divide n_experts=%d (got %d)", n_experts, n_groups);
    if (topk_groups < 1 || topk_groups > n_groups)
        return fail(FT_ERR_ARG, "topk_groups must be in [1, n_groups=%d] (got %d)", n_groups, topk_groups);
    if (group_top < 1 || group_top > 2 || (n_groups > 1 && group_top > n_experts / n_groups))
        return fail(FT_ERR_ARG, "group_top must be 1 or 2 and at most n_experts / n_groups (got %d)", group_top);
    if (top_k > n_experts / n_groups * topk_groups)
        return fail(FT_ERR_ARG, "top_k=%d exceeds the %d experts of the chosen groups", top_k,
                    n_experts / n_groups * topk_groups);
    int64_t n;
    if (row_stride < n_experts) return fail(FT_ERR_ARG, "row_stride must be >= n_experts");
    if (!mul_ok(tokens, row_stride, &n)) return fail(FT_ERR_SIZE, "tokens * row_stride overflows");
    return FT_OK;
}

int check_matrix(int32_t n_experts, int64_t nrows, int64_t ncols) {
    if (int st = check_cols(ncols, "ncols")) return st;
    if (ncols > FT_MAX_NCOLS) return fail(FT_ERR_SIZE, "ncols must be <= %d (got %lld)", FT_MAX_NCOLS, (long long)ncols);
    if (nrows <= 0) return fail(FT_ERR_ARG, "nrows must be > 0 (got %lld)", (long long)nrows);
    int64_t n;
    if (!mul_ok(n_experts, nrows, &n) || n > INT32_MAX) return fail(FT_ERR_SIZE, "n_experts * nrows must be < 2^31");
    return FT_OK;
}

int check_workspace(const void* workspace, size_t have, size_t need) {
    if (need && (!workspace || have < need))
        return fail(FT_ERR_WORKSPACE, "a workspace of %zu bytes is needed (got %zu)", need, workspace ? have : 0);
    if (!aligned(workspace, 256)) return fail(FT_ERR_ALIGN, "the workspace must be 256-byte aligned");
    return FT_OK;
}

size_t take_bytes(size_t* at, size_t bytes) {
    const size_t r = *at;
    *at = al256(*at + bytes);
    return r;
}

// Workspace of a routed product: router order, then (wide tiles) the activation rows and
// scales in that order.
struct ProductWs {
    Fp8Order order;
    int width;
    size_t rows, scales, total;
};

ProductWs product_ws(uint8_t* base, int64_t n_slots, int32_t n_experts, int64_t ncols) {
    ProductWs L{};
    size_t at = al256(fp8_order_layout(base, n_slots, n_experts, false, &L.order));
    L.width = fp8_tile_width(n_slots, n_experts);
    const size_t copied = L.width == kWideTile ? static_cast<size_t>(n_slots) : 0;
    L.rows = take_bytes(&at, copied * static_cast<size_t>(ncols));
    L.scales = take_bytes(&at, copied * static_cast<size_t>(fp8_scale_pitch(ncols)) * 4);
    L.total = at;
    return L;
}

int product_entry(const void* weights, const float* w_scales, const void* act, const float* act_scales,
                  const int32_t* ids, bool dense, bool per_slot, void* out, int32_t out_dtype, int64_t tokens,
                  int32_t top_k, int32_t n_experts, int64_t nrows, int64_t ncols, void* workspace,
                  size_t workspace_bytes, void* stream) {
    clear_error();
    int64_t n_slots, n;
    if (int st = check_slots(tokens, top_k, n_experts, &n_slots)) return st;
    if (int st = check_matrix(n_experts, nrows, ncols)) return st;
    if (!mul_ok(n_slots, nrows, &n) || !mul_ok(n_slots, ncols, &n)) return fail(FT_ERR_SIZE, "output size overflows");
    if (out_dtype != FT_DTYPE_F32 && out_dtype != FT_DTYPE_BF16)
        return fail(FT_ERR_ARG, "out_dtype must be FT_DTYPE_F32 or FT_DTYPE_BF16 (got %d)", out_dtype);
    if (n_slots == 0) return FT_OK;
    if (!weights || !w_scales || !act || !act_scales || !out || (!dense && !ids)) return fail(FT_ERR_ARG, "null pointer");
    if (!aligned(weights, 16) || !aligned(act, 16)) return fail(FT_ERR_ALIGN, "weights and act must be 16-byte aligned");
    if (!aligned(w_scales, 4) || !aligned(act_scales, 4) || !aligned(ids, 4) || !aligned(out, dtype_bytes(out_dtype)))
        return fail(FT_ERR_ALIGN, "scales, ids and out must be aligned to their elements");
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    ProductWs L{};
    if (!dense) {
        L = product_ws(ws, n_slots, n_experts, ncols);
        if (int st = check_workspace(workspace, workspace_bytes, L.total)) return st;
    }
    uint32_t* err = nullptr;
    if (int st = fp8_error_word(&err)) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Fp8Product p{};
    p.weights = static_cast<const uint8_t*>(weights);
    p.w_scales = w_scales;
    p.act = static_cast<const uint8_t*>(act);
    p.act_scales = act_scales;
    p.scale_pitch = static_cast<int32_t>(fp8_blocks(ncols));
    p.n_slots = n_slots;
    p.act_div = per_slot ? 1 : top_k;
    p.act_rows = per_slot ? n_slots : tokens;
    p.nrows = nrows;
    p.ncols = ncols;
    p.n_experts = n_experts;
    const int width = dense ? fp8_tile_width(n_slots, 1) : L.width;
    if (!dense) {
        p.ids = ids;
        p.order = &L.order;
        if (!fp8_orders_itself(n_slots, n_experts, width))
            if (int st = launch_fp8_order(ids, n_slots, n_experts, width, L.order, s)) return st;
        if (width == kWideTile)
            if (int st = launch_fp8_order_rows(&p, ws + L.rows, reinterpret_cast<float*>(ws + L.scales), s)) return st;
    }
    return launch_fp8_product(p, width, out, out_dtype, err, s);
}

// Workspace of a layer: router order; the gated values' codes and scales; and one place for
// what the second product does not read any more, x's codes and scales and (where the first product
// does not quantize the gated values itself: n_inter % 128 != 0, or few slots per expert) that one's
// fp32 rows, and for the rows that the second product writes.  Codes lie in router order for wide tiles
// (`spread`), else by token and by slot.
//
// The second product's rows are fp32, but bf16 for wide tiles where y is bf16: no fewer bits than y
// has, and half the bytes (8192 tokens of 8 slots, 2048 wide: 535 us, with fp32 rows 614; with
// narrower tiles, 8, 64 and 512 tokens, fp32 rows take no longer).  Their rounding, at most 2^-8 of a
// row, is far below that of the codes, 2^-4, which both products start from.
struct LayerWs {
    Fp8Order order;
    size_t mq, ms, xq, xs, h, rows, total;
    int width;
    bool spread, gated;
};

LayerWs layer_ws(uint8_t* base, int64_t tokens, int64_t n_slots, int32_t n_experts, int64_t hidden, int64_t n_inter) {
    LayerWs L{};
    L.width = fp8_tile_width(n_slots, n_experts);
    L.spread = L.width == kWideTile;
    L.gated = L.spread && n_inter % kFp8Block == 0;
    size_t at = al256(fp8_order_layout(base, n_slots, n_experts, L.spread, &L.order));
    const size_t S = static_cast<size_t>(n_slots), X = L.spread ? S : static_cast<size_t>(tokens);
    L.mq = take_bytes(&at, S * n_inter);
    L.ms = take_bytes(&at, S * fp8_scale_pitch(n_inter) * 4);
    L.rows = at;
    L.xq = take_bytes(&at, X * hidden);
    L.xs = take_bytes(&at, X * fp8_scale_pitch(hidden) * 4);
    L.h = take_bytes(&at, L.gated ? 0 : S * 2 * n_inter * 4);
    L.total = std::max(at, al256(L.rows + S * hidden * 4));
    return L;
}

// The most that `total` (tokens, slots) gives for up to `tokens` tokens.  It rises with them but where the
// products' tiles or the order of the slots change, so what counts is the last token of each of those forms.
template <typename F>
size_t most_bytes(int64_t tokens, int32_t top_k, int32_t n_experts, const F& total) {
    size_t most = total(tokens, tokens * top_k);
    auto last = [&](int64_t slots) {      // of a form that holds up to so many slots
        const int64_t t = std::min(tokens, slots / top_k);
        if (t > 0) most = std::max(most, total(t, t * top_k));
    };
    last(top_k);      // (one slot is a form of its own)
    for (const double mean : {kGemvMean, kMean16, kMean32}) last(static_cast<int64_t>(mean * n_experts));
    last(kFastRouteSlots);
    return most;
}

}  // namespace
}  // namespace ft

using namespace ft;

extern "C" {

int ft_moe_gate(const void* logits, int32_t dtype, int64_t row_stride, const float* bias, int32_t* topk_ids,
                float* topk_weights, int64_t tokens, int32_t n_experts, int32_t top_k, int32_t score, int32_t n_groups,
                int32_t topk_groups, int32_t group_top, int32_t renormalize, float scale, void* stream) {
    clear_error();
    int64_t n_slots;
    if (int st = check_gate(tokens, n_experts, top_k, score, n_groups, topk_groups, group_top, dtype, row_stride, &n_slots))
        return st;
    if (tokens == 0) return FT_OK;
    if (!logits || !topk_ids || !topk_weights) return fail(FT_ERR_ARG, "null pointer");
    if (!aligned(logits, dtype_bytes(dtype)) || !aligned(bias, 4) || !aligned(topk_ids, 4) || !aligned(topk_weights, 4))
        return fail(FT_ERR_ALIGN, "logits, bias, topk_ids and topk_weights must be aligned to their elements");
    const GateParams p{tokens, n_experts, top_k, score, n_groups, topk_groups, group_top, renormalize, scale, bias};
    return launch_gate(p, logits, dtype, row_stride, topk_ids, topk_weights, static_cast<cudaStream_t>(stream));
}

static int quantize_entry(const void* x, int32_t dtype, void* codes, float* scales, int64_t rows, int64_t ncols,
                          bool gated, int32_t act_kind, void* stream) {
    clear_error();
    if (rows < 0) return fail(FT_ERR_ARG, "rows must be >= 0 (got %lld)", (long long)rows);
    if (int st = check_cols(ncols, gated ? "n_inter" : "ncols")) return st;
    if (!dtype_bytes(dtype)) return fail(FT_ERR_ARG, "unknown element type %d", dtype);
    if (gated && act_kind != FT_ACT_SILU && act_kind != FT_ACT_GELU_TANH)
        return fail(FT_ERR_ARG, "unknown activation %d", act_kind);
    int64_t n;
    if (!mul_ok(rows, ncols, &n) || ncols / kFp8Block >= INT32_MAX) return fail(FT_ERR_SIZE, "rows * ncols overflows");
    if (rows == 0) return FT_OK;
    if (!x || !codes || !scales) return fail(FT_ERR_ARG, "null pointer");
    if (!aligned(x, 16) || !aligned(codes, 8) || !aligned(scales, 4))
        return fail(FT_ERR_ALIGN, "x must be 16-byte, codes 8-byte and scales 4-byte aligned");
    return launch_quantize_fp8(x, dtype, static_cast<uint8_t*>(codes), scales, rows, ncols, gated, act_kind,
                               static_cast<cudaStream_t>(stream));
}

int ft_quantize_fp8(const void* x, int32_t dtype, void* codes, float* scales, int64_t rows, int64_t ncols, void* stream) {
    return quantize_entry(x, dtype, codes, scales, rows, ncols, false, FT_ACT_SILU, stream);
}

int ft_act_mul_quantize_fp8(const void* h, int32_t dtype, void* codes, float* scales, int64_t rows, int64_t n_inter,
                            int32_t act_kind, void* stream) {
    return quantize_entry(h, dtype, codes, scales, rows, n_inter, true, act_kind, stream);
}

size_t ft_moe_fp8_workspace_bytes(int64_t tokens, int32_t top_k, int32_t n_experts, int64_t ncols) {
    clear_error();
    int64_t n_slots;
    int64_t n;
    if (check_slots(tokens, top_k, n_experts, &n_slots) || check_cols(ncols, "ncols") || !mul_ok(n_slots, ncols, &n)) return 0;
    return most_bytes(tokens, top_k, n_experts, [=](int64_t, int64_t slots) { return product_ws(nullptr, slots, n_experts, ncols).total; });
}

int ft_moe_fp8_fp8(const void* weights, const float* w_scales, const void* act, const float* act_scales,
                   const int32_t* topk_ids, void* out, int32_t out_dtype, int64_t tokens, int32_t top_k,
                   int32_t n_experts, int64_t nrows, int64_t ncols, void* workspace, size_t workspace_bytes,
                   void* stream) {
    return product_entry(weights, w_scales, act, act_scales, topk_ids, false, false, out, out_dtype, tokens, top_k,
                         n_experts, nrows, ncols, workspace, workspace_bytes, stream);
}

int ft_moe_fp8_fp8_slots(const void* weights, const float* w_scales, const void* act_slots, const float* act_scales,
                         const int32_t* topk_ids, void* out, int32_t out_dtype, int64_t tokens, int32_t top_k,
                         int32_t n_experts, int64_t nrows, int64_t ncols, void* workspace, size_t workspace_bytes,
                         void* stream) {
    return product_entry(weights, w_scales, act_slots, act_scales, topk_ids, false, true, out, out_dtype, tokens, top_k,
                         n_experts, nrows, ncols, workspace, workspace_bytes, stream);
}

int ft_matmul_fp8_fp8(const void* weights, const float* w_scales, const void* act, const float* act_scales, void* out,
                      int32_t out_dtype, int64_t rows, int64_t nrows, int64_t ncols, void* stream) {
    return product_entry(weights, w_scales, act, act_scales, nullptr, true, true, out, out_dtype, rows, 1, 1, nrows,
                         ncols, nullptr, 0, stream);
}

int ft_moe_combine(const void* rows, int32_t rows_dtype, const float* topk_weights, const void* add, void* y,
                   int32_t y_dtype, int64_t tokens, int32_t top_k, int64_t ncols, void* stream) {
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
    if (!rows || !topk_weights || !y) return fail(FT_ERR_ARG, "null pointer");
    if (!aligned(rows, dtype_bytes(rows_dtype)) || !aligned(topk_weights, 4) || !aligned(y, dtype_bytes(y_dtype)) ||
        !aligned(add, dtype_bytes(y_dtype)))
        return fail(FT_ERR_ALIGN, "rows, topk_weights, add and y must be aligned to their elements");
    return launch_combine(rows, rows_dtype, topk_weights, add, y, y_dtype, tokens, top_k, ncols,
                          static_cast<cudaStream_t>(stream));
}

size_t ft_moe_layer_fp8_workspace_bytes(int64_t tokens, int32_t top_k, int32_t n_experts, int64_t hidden,
                                        int64_t n_inter) {
    clear_error();
    int64_t n_slots, n;
    if (check_slots(tokens, top_k, n_experts, &n_slots)) return 0;
    if (check_matrix(n_experts, hidden, n_inter) || n_inter > FT_MAX_NCOLS || check_matrix(n_experts, 2 * n_inter, hidden))
        return 0;
    if (!mul_ok(n_slots, 8 * (hidden + n_inter), &n)) return 0;
    return most_bytes(tokens, top_k, n_experts,
                      [=](int64_t t, int64_t slots) { return layer_ws(nullptr, t, slots, n_experts, hidden, n_inter).total; });
}

int ft_moe_layer_fp8(const void* x, int32_t x_dtype, const void* logits, int32_t logits_dtype, int64_t row_stride,
                     const float* bias, const void* w13, const float* s13, const void* w2, const float* s2, void* y,
                     int32_t* topk_ids, float* topk_weights, int64_t tokens, int32_t n_experts, int32_t top_k,
                     int64_t hidden, int64_t n_inter, int32_t score, int32_t n_groups, int32_t topk_groups,
                     int32_t group_top, int32_t renormalize, float scale, int32_t act_kind, void* workspace,
                     size_t workspace_bytes, void* stream) {
    clear_error();
    int64_t n_slots, n;
    if (int st = check_gate(tokens, n_experts, top_k, score, n_groups, topk_groups, group_top, logits_dtype, row_stride,
                            &n_slots))
        return st;
    if (int st = check_cols(hidden, "hidden")) return st;
    if (int st = check_cols(n_inter, "n_inter")) return st;
    if (hidden > FT_MAX_NCOLS || n_inter > FT_MAX_NCOLS)
        return fail(FT_ERR_SIZE, "hidden and n_inter must be <= %d", FT_MAX_NCOLS);
    if (int st = check_matrix(n_experts, 2 * n_inter, hidden)) return st;
    if (int st = check_matrix(n_experts, hidden, n_inter)) return st;
    if (x_dtype != FT_DTYPE_F16 && x_dtype != FT_DTYPE_BF16)
        return fail(FT_ERR_ARG, "x_dtype must be FT_DTYPE_F16 or FT_DTYPE_BF16 (got %d)", x_dtype);
    if (act_kind != FT_ACT_SILU && act_kind != FT_ACT_GELU_TANH) return fail(FT_ERR_ARG, "unknown activation %d", act_kind);
    if (!mul_ok(n_slots, 8 * (hidden + n_inter), &n)) return fail(FT_ERR_SIZE, "workspace size overflows");
    if (tokens == 0) return FT_OK;
    if (!x || !logits || !w13 || !s13 || !w2 || !s2 || !y || !topk_ids || !topk_weights)
        return fail(FT_ERR_ARG, "null pointer");
    if (!aligned(x, 16) || !aligned(w13, 16) || !aligned(w2, 16))
        return fail(FT_ERR_ALIGN, "x, w13 and w2 must be 16-byte aligned");
    if (!aligned(logits, dtype_bytes(logits_dtype)) || !aligned(bias, 4) || !aligned(s13, 4) || !aligned(s2, 4) ||
        !aligned(y, 2) || !aligned(topk_ids, 4) || !aligned(topk_weights, 4))
        return fail(FT_ERR_ALIGN, "logits, bias, scales, y, topk_ids and topk_weights must be aligned to their elements");
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const LayerWs L = layer_ws(ws, tokens, n_slots, n_experts, hidden, n_inter);
    if (int st = check_workspace(workspace, workspace_bytes, L.total)) return st;
    uint32_t* err = nullptr;
    if (int st = fp8_error_word(&err)) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);

    const GateParams g{tokens, n_experts, top_k, score, n_groups, topk_groups, group_top, renormalize, scale, bias};
    if (int st = launch_gate(g, logits, logits_dtype, row_stride, topk_ids, topk_weights, s)) return st;
    if (L.width == 1 && fp8_token_ok(n_slots, tokens, top_k, hidden, n_inter))
        return launch_fp8_token_layer(x, x_dtype, static_cast<const uint8_t*>(w13), s13, static_cast<const uint8_t*>(w2), s2, topk_ids,
                                      topk_weights, reinterpret_cast<float*>(ws + L.h), y, tokens, top_k, n_experts, hidden, n_inter,
                                      act_kind, s);
    if (!fp8_orders_itself(n_slots, n_experts, L.width))
        if (int st = launch_fp8_order(topk_ids, n_slots, n_experts, L.width, L.order, s)) return st;
    float *xs = reinterpret_cast<float*>(ws + L.xs), *ms = reinterpret_cast<float*>(ws + L.ms);
    Fp8Product p{};
    p.ids = topk_ids;
    p.order = &L.order;
    p.n_slots = n_slots;
    p.n_experts = n_experts;
    // first product: gate and up rows
    if (L.spread) {
        p.scale_pitch = fp8_scale_pitch(hidden);
        if (int st = launch_quantize_fp8_spread(x, x_dtype, ws + L.xq, xs, tokens, hidden, false, act_kind, L.order.pos, top_k,
                                                p.scale_pitch, s))
            return st;
    } else {
        p.scale_pitch = static_cast<int32_t>(fp8_blocks(hidden));
        if (int st = launch_quantize_fp8(x, x_dtype, ws + L.xq, xs, tokens, hidden, false, act_kind, s)) return st;
    }
    p.weights = static_cast<const uint8_t*>(w13);
    p.w_scales = s13;
    p.act = ws + L.xq;
    p.act_scales = xs;
    p.ordered = L.spread;
    p.act_div = top_k;
    p.act_rows = L.spread ? n_slots : tokens;
    p.nrows = 2 * n_inter;
    p.ncols = hidden;
    if (L.gated) {
        p.mid = ws + L.mq;
        p.mid_scales = ms;
        p.mid_pitch = fp8_scale_pitch(n_inter);
        p.act_kind = act_kind;
        if (int st = launch_fp8_product(p, L.width, nullptr, FT_DTYPE_F32, err, s)) return st;
        p.mid = nullptr;
        p.ordered = true;
        p.scale_pitch = fp8_scale_pitch(n_inter);
    } else {
        if (int st = launch_fp8_product(p, L.width, ws + L.h, FT_DTYPE_F32, err, s)) return st;
        p.scale_pitch = L.spread ? fp8_scale_pitch(n_inter) : static_cast<int32_t>(fp8_blocks(n_inter));
        const int st = L.spread ? launch_quantize_fp8_spread(ws + L.h, FT_DTYPE_F32, ws + L.mq, ms, n_slots, n_inter, true, act_kind,
                                                             L.order.pos, 1, p.scale_pitch, s)
                                : launch_quantize_fp8(ws + L.h, FT_DTYPE_F32, ws + L.mq, ms, n_slots, n_inter, true, act_kind, s);
        if (st) return st;
    }
    // second product
    p.weights = static_cast<const uint8_t*>(w2);
    p.w_scales = s2;
    p.act = ws + L.mq;
    p.act_scales = ms;
    p.act_div = 1;
    p.act_rows = n_slots;
    p.nrows = hidden;
    p.ncols = n_inter;
    const int rows_dtype = x_dtype == FT_DTYPE_BF16 && L.width == kWideTile ? FT_DTYPE_BF16 : FT_DTYPE_F32;
    if (int st = launch_fp8_product(p, L.width, ws + L.rows, rows_dtype, err, s)) return st;
    return launch_combine(ws + L.rows, rows_dtype, topk_weights, nullptr, y, x_dtype, tokens, top_k, hidden, s);
}

}  // extern "C"
