// The weighted sum of a token's expert rows:
//
//   y[t][c] = sum_j w[t][j] rows[t][j][c]  (+ add[t][c])
//
// summed in fp32 in the order j = 0 .. k - 1, `add` last, rounded once.  A row
// whose weight is 0 is not read, so rows of slots that no expert computed may
// hold anything.
//
// Memory-bound: a thread owns the V neighbouring columns of a token that make 16 bytes of the
// rows' type and reads them of all rows.  A CTA works on one token, with as many threads as
// share its columns evenly: one thread per V columns of all tokens divided by the row length
// in 64 bits, 83 us against 75 (5.5 TB/s) for 8191 tokens, 8 rows of 2816 bf16 each.  DRAM is at 69 %
// of its peak; warps wait for rows that wait for their weights.
//
// Rows or sums that do not start at 16-byte words everywhere are read by single elements
// (moe_combine_ragged_kernel), four columns of four rows at once in a thread (8191 tokens, 8 rows
// of 2813 bf16: 103 us; one column 185; the two aligned words around eight columns, shifted, 132).
#include <type_traits>

#include "fp8_common.cuh"
#include "ft_internal.h"

namespace ft {

constexpr int kCombineThreads = 256;

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
            load_vec<TI, V>(base + k * ncols, v);
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
    } else {
        static_assert(BYTES == 8, "eight bytes or whole words");
        *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(o);
    }
}

constexpr int kRaggedCols = 4, kRaggedRows = 4;

// An element's bits in a register of their own, 0 where `there` is false: in C++ the compiler
// branches around each load, or packs 16-bit elements in pairs and waits for them to do so.
template <typename T>
__device__ __forceinline__ uint32_t load_bits(const T* p, bool there) {
    uint32_t w;
    if constexpr (sizeof(T) == 4)
        asm("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.u32 %0, 0;\n\t@p ld.global.nc.b32 %0, [%1];\n\t}"
            : "=r"(w) : "l"(p), "r"(static_cast<uint32_t>(there)));
    else
        asm("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.u32 %0, 0;\n\t@p ld.global.nc.u16 %0, [%1];\n\t}"
            : "=r"(w) : "l"(p), "r"(static_cast<uint32_t>(there)));
    return w;
}

template <typename T>
__device__ __forceinline__ float bits_value(uint32_t w) {
    static_assert(sizeof(T) == 4 || std::is_same<T, __nv_bfloat16>::value, "rows are fp32 or bf16");
    return __uint_as_float(sizeof(T) == 4 ? w : w << 16);
}

// A thread's columns lie blockDim apart.
template <typename TI, typename TO>
__global__ void __launch_bounds__(kCombineThreads)
    moe_combine_ragged_kernel(const TI* __restrict__ rows, const float* __restrict__ weights, const TO* __restrict__ add,
                              TO* __restrict__ y, int64_t ncols, uint32_t per_row, int32_t top_k) {
    const uint32_t t = blockIdx.x / per_row;
    const int64_t c0 = static_cast<int64_t>(blockIdx.x - t * per_row) * blockDim.x * kRaggedCols, left = ncols - c0;
    const TI* base = rows + static_cast<int64_t>(t) * top_k * ncols + c0;
    uint32_t c[kRaggedCols];
    bool in[kRaggedCols];
    float acc[kRaggedCols];
#pragma unroll
    for (int i = 0; i < kRaggedCols; ++i) {
        c[i] = threadIdx.x + i * blockDim.x;
        in[i] = c[i] < left;
        acc[i] = 0.0f;
    }
    // the rows k0 .. k0 + R - 1, all asked for before the first is added
    auto add_rows = [&](int32_t k0, auto count) {
        constexpr int R = decltype(count)::value;
        float w[R];
        uint32_t x[R][kRaggedCols];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            w[r] = __ldg(weights + static_cast<int64_t>(t) * top_k + k0 + r);
            const TI* row = base + (k0 + r) * ncols;
#pragma unroll
            for (int i = 0; i < kRaggedCols; ++i) x[r][i] = load_bits(row + c[i], w[r] != 0.0f && in[i]);
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < kRaggedCols; ++i) acc[i] = fmaf(w[r], bits_value<TI>(x[r][i]), acc[i]);
    };
    int32_t k0 = 0;
    for (; k0 + kRaggedRows <= top_k; k0 += kRaggedRows) add_rows(k0, std::integral_constant<int, kRaggedRows>{});
    for (; k0 < top_k; ++k0) add_rows(k0, std::integral_constant<int, 1>{});
#pragma unroll
    for (int i = 0; i < kRaggedCols; ++i) {
        if (in[i]) {
            const int64_t at = static_cast<int64_t>(t) * ncols + c0 + c[i];
            y[at] = from_f32<TO>(add ? acc[i] + to_f32<TO>(add[at]) : acc[i]);
        }
    }
}

template <typename TI, typename TO>
static int launch_typed(const void* rows, const float* weights, const void* add, void* y, int64_t tokens, int32_t top_k,
                        int64_t ncols, cudaStream_t s) {
    constexpr int V = 16 / static_cast<int>(sizeof(TI));
    auto ok = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    const bool wide = ncols % V == 0 && ncols * static_cast<int64_t>(sizeof(TO)) % 16 == 0 && ok(rows) && ok(y) && ok(add);
    const int64_t per = wide ? V : kRaggedCols, row_vec = (ncols + per - 1) / per;      // columns of a thread, threads of a row
    const int64_t per_row = (row_vec + kCombineThreads - 1) / kCombineThreads;
    const int64_t threads = ((row_vec + per_row - 1) / per_row + 31) / 32 * 32;
    if (per_row > 0x7FFFFFFF / tokens) return fail(FT_ERR_SIZE, "tokens * ncols too large for one launch");
    const dim3 grid(static_cast<unsigned>(tokens * per_row)), block(static_cast<unsigned>(threads));
    const TI* r = static_cast<const TI*>(rows);
    const TO* a = static_cast<const TO*>(add);
    TO* o = static_cast<TO*>(y);
    if (wide) moe_combine_kernel<TI, TO, V><<<grid, block, 0, s>>>(r, weights, a, o, row_vec, static_cast<uint32_t>(per_row), top_k);
    else moe_combine_ragged_kernel<TI, TO><<<grid, block, 0, s>>>(r, weights, a, o, ncols, static_cast<uint32_t>(per_row), top_k);
    return check_launch(wide ? "moe_combine_kernel" : "moe_combine_ragged_kernel", grid, block, 0);
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
