// Argument checks that the C entry points with a caller's workspace share.
#pragma once

#include <cstddef>
#include <cstdint>

#include "../../include/ft_moe.h"
#include "ft_internal.h"

namespace ft {

constexpr int64_t kMaxElems = int64_t(1) << 60;   // products of sizes stay far from overflow below this

inline bool mul_ok(int64_t a, int64_t b, int64_t* r) {
    if (a < 0 || b < 0 || (a != 0 && b > kMaxElems / a)) return false;
    *r = a * b;
    return true;
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline size_t al256(size_t x) { return (x + 255) & ~size_t(255); }

inline int dtype_bytes(int32_t d) { return d == FT_DTYPE_F32 ? 4 : d == FT_DTYPE_F16 || d == FT_DTYPE_BF16 ? 2 : 0; }

inline int check_slots(int64_t tokens, int32_t top_k, int32_t n_experts, int64_t* n_slots) {
    if (tokens < 0) return fail(FT_ERR_ARG, "tokens must be >= 0 (got %lld)", (long long)tokens);
    if (n_experts < 1 || n_experts > FT_MAX_EXPERTS)
        return fail(FT_ERR_ARG, "n_experts must be in [1, %d] (got %d)", FT_MAX_EXPERTS, n_experts);
    if (top_k < 1 || top_k > n_experts)
        return fail(FT_ERR_ARG, "top_k must be in [1, n_experts=%d] (got %d)", n_experts, top_k);
    if (!mul_ok(tokens, top_k, n_slots) || *n_slots > INT32_MAX)
        return fail(FT_ERR_SIZE, "tokens * top_k = %lld * %d must be < 2^31", (long long)tokens, top_k);
    return FT_OK;
}

inline int check_workspace(const void* workspace, size_t have, size_t need) {
    if (need && (!workspace || have < need))
        return fail(FT_ERR_WORKSPACE, "a workspace of %zu bytes is needed (got %zu)", need, workspace ? have : 0);
    if (!aligned(workspace, 256)) return fail(FT_ERR_ALIGN, "the workspace must be 256-byte aligned");
    return FT_OK;
}

inline size_t take_bytes(size_t* at, size_t bytes) {
    const size_t r = *at;
    *at = al256(*at + bytes);
    return r;
}

}  // namespace ft
