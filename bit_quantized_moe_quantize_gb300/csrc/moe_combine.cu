// The weighted sum of a token's expert rows:
//
//   y[t][c] = sum_j w[t][j] rows[t][j][c]  (+ add[t][c])
//
// summed in fp32 in the order j = 0 .. k - 1, `add` last, rounded once.  A row
// whose weight is 0 is not read, so rows of slots that no expert computed may
// hold anything.
//
// Memory-bound: each thread owns V neighbouring columns of one token and reads
// them of all rows; V elements make 16 bytes of the rows' type where the
// column count and the pointers allow it, else V = 1.  A CTA works on one token, with as
// many threads as share its columns evenly (a 64-bit division per thread to find its token
// took as long as its loads).
#include "fp8_common.cuh"
#include "ft_internal.h"

namespace ft {

constexpr int kCombineThreads = 256;

template <typename T, int V>
__device__ __forceinline__ void load_cols(const T* p, float (&v)[V]) {
    if constexpr (V == 1) v[0] = to_f32<T>(p[0]);
    else load_vec<T, V>(p, v);
}

template <typename TI, typename TO, int V>
__global__ void __launch_bounds__(kCombineThreads)
    moe_combine_kernel(const TI* __restrict__ rows, const float* __restrict__ weights, const TO* __restrict__ add,
                       TO* __restrict__ y, int64_t row_vec, uint32_t per_row, int32_t top_k) {
    const uint32_t tb = blockIdx.x / per_row;
    const int64_t v = static_cast<int64_t>(blockIdx.x - tb * per_row) * blockDim.x + threadIdx.x;
    if (v >= row_vec) return;
    const int64_t t = tb, c = v * V, ncols = row_vec * V;
    float acc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.0f;
    const TI* base = rows + t * top_k * ncols + c;
#pragma unroll 4
    for (int32_t k = 0; k < top_k; ++k) {
        const float w = __ldg(weights + t * top_k + k);
        if (w != 0.0f) {
            float v[V];
            load_cols<TI, V>(base + k * ncols, v);
#pragma unroll
            for (int j = 0; j < V; ++j) acc[j] = fmaf(w, v[j], acc[j]);
        }
    }
    if (add) {
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] += to_f32<TO>(add[t * ncols + c + j]);
    }
    __align__(16) TO o[V];
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = from_f32<TO>(acc[j]);
    TO* dst = y + t * ncols + c;
    constexpr int BYTES = V * static_cast<int>(sizeof(TO));
    if constexpr (BYTES % 16 == 0) {
#pragma unroll
        for (int j = 0; j < BYTES / 16; ++j) reinterpret_cast<uint4*>(dst)[j] = reinterpret_cast<const uint4*>(o)[j];
    } else if constexpr (BYTES == 8) {
        *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(o);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) dst[j] = o[j];
    }
}

template <typename TI, typename TO>
static int launch_typed(const void* rows, const float* weights, const void* add, void* y, int64_t tokens, int32_t top_k,
                        int64_t ncols, cudaStream_t s) {
    constexpr int V = 16 / static_cast<int>(sizeof(TI));
    auto ok = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    const bool wide = ncols % V == 0 && ncols * static_cast<int64_t>(sizeof(TO)) % 16 == 0 && ok(rows) && ok(y) && ok(add);
    const int64_t row_vec = wide ? ncols / V : ncols, per_row = (row_vec + kCombineThreads - 1) / kCombineThreads;
    const int64_t threads = ((row_vec + per_row - 1) / per_row + 31) / 32 * 32;
    if (per_row > 0x7FFFFFFF / tokens) return fail(FT_ERR_SIZE, "tokens * ncols too large for one launch");
    const dim3 grid(static_cast<unsigned>(tokens * per_row)), block(static_cast<unsigned>(threads));
    const TI* r = static_cast<const TI*>(rows);
    const TO* a = static_cast<const TO*>(add);
    TO* o = static_cast<TO*>(y);
    if (wide) moe_combine_kernel<TI, TO, V><<<grid, block, 0, s>>>(r, weights, a, o, row_vec, static_cast<uint32_t>(per_row), top_k);
    else moe_combine_kernel<TI, TO, 1><<<grid, block, 0, s>>>(r, weights, a, o, row_vec, static_cast<uint32_t>(per_row), top_k);
    return check_launch("moe_combine_kernel", grid, block, 0);
}

int launch_combine(const void* rows, int rows_dtype, const float* weights, const void* add, void* y, int y_dtype,
                   int64_t tokens, int32_t top_k, int64_t ncols, cudaStream_t s) {
    if (tokens == 0) return FT_OK;
    if (rows_dtype == FT_DTYPE_F32) {
        if (y_dtype == FT_DTYPE_F32) return launch_typed<float, float>(rows, weights, add, y, tokens, top_k, ncols, s);
        if (y_dtype == FT_DTYPE_F16) return launch_typed<float, __half>(rows, weights, add, y, tokens, top_k, ncols, s);
        return launch_typed<float, __nv_bfloat16>(rows, weights, add, y, tokens, top_k, ncols, s);
    }
    if (y_dtype == FT_DTYPE_F32) return launch_typed<__nv_bfloat16, float>(rows, weights, add, y, tokens, top_k, ncols, s);
    if (y_dtype == FT_DTYPE_F16) return launch_typed<__nv_bfloat16, __half>(rows, weights, add, y, tokens, top_k, ncols, s);
    return launch_typed<__nv_bfloat16, __nv_bfloat16>(rows, weights, add, y, tokens, top_k, ncols, s);
}

}  // namespace ft
