// Gradient of the weighted sum of a token's expert rows, y[t] = sum_j w[t][j] rows[t][j]:
//
//   d rows[t][j][c] = w[t][j] dy[t][c]
//   d w[t][j]       = sum_c dy[t][c] rows[t][j][c], in fp32
//
// A row whose weight is 0 took no part: it is not read, and both its gradients are 0.
//
// Memory-bound: the rows are read once and as much is written (8191 x 8 rows of 2816 bf16: 118.5 us, 785 MB at 6.6 TB/s;
// 8 x 8 of 2048: 4.3 us).  A slot is one to eight warps', as many as leave work for all of the GPU where slots are few;
// dy comes from the caches for all of a token's slots but the first.
// Where rows do not start at 16-byte words, the words inside of a row are read and written whole all the same, dy beside
// them and the elements around them one by one (combine_grad_ragged_kernel).
#include "fp8_common.cuh"
#include "ft_internal.h"

namespace ft {

namespace {

constexpr int kGradThreads = 256, kGradWarps = kGradThreads / 32;

// V neighbouring elements, 8 bytes or whole 16-byte words of them.
template <typename T, int V>
__device__ __forceinline__ void load_some(const T* p, float (&v)[V]) {
    if constexpr (V * sizeof(T) % 16 == 0) {
        load_vec<T, V>(p, v);
    } else {
        static_assert(V * sizeof(T) == 8, "eight bytes or whole words");
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
        const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = to_f32<T>(e[i]);
    }
}

// A slot's sum over its warps' lanes, in a fixed order, to its weight's gradient.
__device__ __forceinline__ void store_sum(float sum, float* part, float* grad_weights, int64_t slot, bool there, int32_t warps) {
    const int32_t warp = static_cast<int32_t>(threadIdx.x >> 5), lane = static_cast<int32_t>(lane_id());
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (warps > 1) {
        if (lane == 0) part[warp] = sum;
        __syncthreads();
        sum = 0.0f;
        for (int32_t i = 0; i < warps; ++i) sum += part[warp / warps * warps + i];
    }
    if (there && lane == 0 && warp % warps == 0) grad_weights[slot] = sum;
}

// V: elements of a 16-byte word of the rows, or 1.  grad_rows may be null.
template <typename TI, typename TY, int V>
__global__ void __launch_bounds__(kGradThreads)
    combine_grad_kernel(const TY* __restrict__ dy, const TI* __restrict__ rows, const float* __restrict__ weights,
                        TI* __restrict__ grad_rows, float* __restrict__ grad_weights, int64_t n_slots, int64_t row_vec,
                        uint32_t top_k, int32_t warps) {
    __shared__ float part[kGradWarps];
    const int32_t warp = static_cast<int32_t>(threadIdx.x >> 5), lane = static_cast<int32_t>(lane_id());
    const int64_t slot = static_cast<int64_t>(blockIdx.x) * (kGradWarps / warps) + warp / warps;
    const bool there = slot < n_slots;
    const float w = there ? __ldg(weights + slot) : 0.0f;
    float sum = 0.0f;
    if (there) {
        const int64_t ncols = row_vec * V;
        const TY* g = dy + static_cast<int64_t>(static_cast<uint32_t>(slot) / top_k) * ncols;
        const TI* r = rows + slot * ncols;
        TI* out = grad_rows ? grad_rows + slot * ncols : nullptr;
        const int64_t step = 32 * warps;
        if (w != 0.0f) {
#pragma unroll 4
            for (int64_t i = warp % warps * 32 + lane; i < row_vec; i += step) {
                float x[V], y[V];
                if constexpr (V == 1) {
                    x[0] = to_f32<TI>(r[i]);
                    y[0] = to_f32<TY>(g[i]);
                } else {
                    load_vec<TI, V>(r + i * V, x);
                    load_some<TY, V>(g + i * V, y);
                }
                __align__(16) TI o[V];
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    sum = fmaf(x[j], y[j], sum);
                    o[j] = from_f32<TI>(w * y[j]);
                }
                if (out) {
                    if constexpr (V == 1) out[i] = o[0];
                    else reinterpret_cast<uint4*>(out)[i] = *reinterpret_cast<const uint4*>(o);
                }
            }
        } else if (out) {
            for (int64_t i = warp % warps * 32 + lane; i < row_vec; i += step) {
                if constexpr (V == 1) out[i] = from_f32<TI>(0.0f);
                else reinterpret_cast<uint4*>(out)[i] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
    }
    if (grad_weights) store_sum(sum, part, grad_weights, slot, there, warps);
}

// Rows that start anywhere: V elements to a 16-byte word, `rows` and `grad_rows` as far from one as each other.
template <typename TI, typename TY, int V>
__global__ void __launch_bounds__(kGradThreads)
    combine_grad_ragged_kernel(const TY* __restrict__ dy, const TI* __restrict__ rows, const float* __restrict__ weights,
                               TI* __restrict__ grad_rows, float* __restrict__ grad_weights, int64_t n_slots, int32_t ncols,
                               uint32_t top_k, int32_t warps) {
    __shared__ float part[kGradWarps];
    const int32_t warp = static_cast<int32_t>(threadIdx.x >> 5), lane = static_cast<int32_t>(lane_id());
    const int64_t slot = static_cast<int64_t>(blockIdx.x) * (kGradWarps / warps) + warp / warps;
    const bool there = slot < n_slots;
    const float w = there ? __ldg(weights + slot) : 0.0f;
    float sum = 0.0f;
    if (there) {
        const TY* g = dy + static_cast<int64_t>(static_cast<uint32_t>(slot) / top_k) * ncols;
        const TI* r = rows + slot * ncols;
        TI* out = grad_rows ? grad_rows + slot * ncols : nullptr;
        const int32_t before = static_cast<int32_t>(reinterpret_cast<uintptr_t>(r) % 16 / sizeof(TI));      // elements of the first word that are not the row's
        const int32_t words = (before + ncols + V - 1) / V;
#pragma unroll 2
        for (int32_t i = warp % warps * 32 + lane; i < words; i += 32 * warps) {
            const int32_t c = i * V - before;
            if (c >= 0 && c + V <= ncols) {
                float x[V] = {}, y[V];
                if (w != 0.0f) load_vec<TI, V>(r + c, x);
#pragma unroll
                for (int j = 0; j < V; ++j) y[j] = w != 0.0f ? to_f32<TY>(__ldg(g + c + j)) : 0.0f;
                __align__(16) TI o[V];
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    sum = fmaf(x[j], y[j], sum);
                    o[j] = from_f32<TI>(w * y[j]);
                }
                if (out) *reinterpret_cast<uint4*>(out + c) = *reinterpret_cast<const uint4*>(o);
            } else {
                for (int32_t q = c < 0 ? 0 : c; q < ncols && q < c + V; ++q) {
                    const float y = w != 0.0f ? to_f32<TY>(g[q]) : 0.0f;
                    if (w != 0.0f) sum = fmaf(to_f32<TI>(r[q]), y, sum);
                    if (out) out[q] = from_f32<TI>(w * y);
                }
            }
        }
    }
    if (grad_weights) store_sum(sum, part, grad_weights, slot, there, warps);
}

template <typename TI, typename TY>
int launch_grad_typed(const void* dy, const void* rows, const float* weights, void* grad_rows, float* grad_weights,
                      int64_t tokens, int32_t top_k, int64_t ncols, cudaStream_t s) {
    constexpr int V = 16 / static_cast<int>(sizeof(TI));
    auto ok = [](const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; };
    constexpr unsigned DY = V * sizeof(TY) % 16 == 0 ? 16 : 8;
    const bool wide = ncols % V == 0 && ok(rows, 16) && ok(grad_rows, 16) && ok(dy, DY);
    const int64_t slots = tokens * top_k;
    int32_t warps = 1;
    while (warps < kGradWarps && slots * warps < 32 * static_cast<int64_t>(sm_count())) warps *= 2;
    const int64_t per = kGradWarps / warps, ctas = (slots + per - 1) / per;
    const dim3 grid(static_cast<unsigned>(ctas)), block(kGradThreads);
    const TY* g = static_cast<const TY*>(dy);
    const TI* r = static_cast<const TI*>(rows);
    TI* o = static_cast<TI*>(grad_rows);
    const uint32_t k = static_cast<uint32_t>(top_k);
    if (wide) combine_grad_kernel<TI, TY, V><<<grid, block, 0, s>>>(g, r, weights, o, grad_weights, slots, ncols / V, k, warps);
    else if (ncols < (1 << 30) && (!o || (reinterpret_cast<uintptr_t>(o) - reinterpret_cast<uintptr_t>(r)) % 16 == 0))
        combine_grad_ragged_kernel<TI, TY, V><<<grid, block, 0, s>>>(g, r, weights, o, grad_weights, slots, static_cast<int32_t>(ncols), k, warps);
    else combine_grad_kernel<TI, TY, 1><<<grid, block, 0, s>>>(g, r, weights, o, grad_weights, slots, ncols, k, warps);
    return check_launch(wide ? "combine_grad_kernel" : "combine_grad_kernel (ragged)", grid, block, 0);
}

}  // namespace

int launch_combine_grad(const void* dy, int dy_dtype, const void* rows, int rows_dtype, const float* weights, void* grad_rows,
                        float* grad_weights, int64_t tokens, int32_t top_k, int64_t ncols, cudaStream_t s) {
    auto go = [&](auto ti, auto ty) {
        return launch_grad_typed<decltype(ti), decltype(ty)>(dy, rows, weights, grad_rows, grad_weights, tokens, top_k, ncols, s);
    };
    if (rows_dtype == FT_DTYPE_F32) {
        if (dy_dtype == FT_DTYPE_F32) return go(float{}, float{});
        if (dy_dtype == FT_DTYPE_F16) return go(float{}, __half{});
        return go(float{}, __nv_bfloat16{});
    }
    if (dy_dtype == FT_DTYPE_F32) return go(__nv_bfloat16{}, float{});
    if (dy_dtype == FT_DTYPE_F16) return go(__nv_bfloat16{}, __half{});
    return go(__nv_bfloat16{}, __nv_bfloat16{});
}

}  // namespace ft
