// Rows -> e4m3 codes with one fp32 scale per 128 columns, and the same of the
// gated activation between the two expert products.
//
//   scale = amax / 448 (IEEE quotient of the block's largest magnitude),
//   code  = e4m3(v / scale), round to nearest even; a block whose scale is 0
//           gets codes 0
//
// Half a warp takes one block of a row: lane i its values 8 i .. 8 i + 7 (columns past the
// row's end count as 0 and are not stored), four shuffles find the largest magnitude.  The
// codes are those of the IEEE quotients; see fp8_codes for how most of them come without a
// division.  A non-finite value makes its block's scale infinite or NaN, and what is
// divided by it 0 or NaN.
#include "fp8_quant.cuh"
#include "ft_internal.h"

namespace ft {

constexpr int kQuantWarps = 8, kQuantAhead = 2;

// Eight neighbouring elements, 16-byte aligned.
template <typename T>
__device__ __forceinline__ void load_raw(const T* p, T (&v)[8]) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) reinterpret_cast<uint4*>(v)[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
}

// GATED: x holds rows of 2 ncols values, gate then up.  SPREAD: row r is a token's, and
// its codes and scales go to the rows pos[r * k ..] (-1: none) of the outputs.
template <typename T, bool GATED, bool SPREAD>
__global__ void __launch_bounds__(32 * kQuantWarps)
    quantize_fp8_kernel(const T* __restrict__ x, uint8_t* __restrict__ codes, float* __restrict__ scales,
                        uint32_t n_blocks, uint32_t nb, int64_t ncols, int kind, const int32_t* __restrict__ pos, int32_t k,
                        int32_t pitch) {
    const uint32_t sub = lane_id() & 15u;
    // both of a half warp's blocks are asked for before the first is worked on
    __align__(16) T raw[kQuantAhead][GATED ? 2 : 1][8];
    uint32_t at[kQuantAhead];
    int64_t row[kQuantAhead], col[kQuantAhead];
    bool in[kQuantAhead];
#pragma unroll
    for (int n = 0; n < kQuantAhead; ++n) {
        at[n] = ((blockIdx.x * kQuantAhead + n) * kQuantWarps + (threadIdx.x >> 5)) * 2 + (lane_id() >> 4);
        const bool there = at[n] < n_blocks;
        const uint32_t r = there ? at[n] / nb : 0u;
        row[n] = r;
        col[n] = static_cast<int64_t>(there ? at[n] - r * nb : 0u) * kFp8Block + 8 * sub;
        in[n] = there && col[n] < ncols;      // ncols % 16 == 0: a lane's eight values are all inside or all outside
        if (in[n]) {
            if constexpr (GATED) {
                load_raw(x + row[n] * 2 * ncols + col[n], raw[n][0]);
                load_raw(x + row[n] * 2 * ncols + ncols + col[n], raw[n][1]);
            } else {
                load_raw(x + row[n] * ncols + col[n], raw[n][0]);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < kQuantAhead; ++n) {
        float v[8] = {};
        if (in[n]) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (GATED) v[j] = act_mul_f32(to_f32<T>(raw[n][0][j]), to_f32<T>(raw[n][1][j]), kind);
                else v[j] = to_f32<T>(raw[n][0][j]);
            }
        }
        const float scale = fp8_block_scale(v);
        if (in[n]) {
            const uint2 q = fp8_codes(v, scale);
            if constexpr (SPREAD) {
                for (int32_t j = 0; j < k; ++j) {
                    const int64_t p = __ldg(pos + row[n] * k + j);
                    if (p >= 0) {
                        *reinterpret_cast<uint2*>(codes + p * ncols + col[n]) = q;
                        if (sub == 0) scales[p * pitch + (at[n] - static_cast<uint32_t>(row[n]) * nb)] = scale;
                    }
                }
            } else {
                if (sub == 0) scales[at[n]] = scale;
                *reinterpret_cast<uint2*>(codes + row[n] * ncols + col[n]) = q;
            }
        }
    }
}

template <typename T, bool GATED, bool SPREAD = false>
static int launch_typed(const void* x, uint8_t* codes, float* scales, int64_t rows, int64_t ncols, int kind,
                        cudaStream_t s, const int32_t* pos = nullptr, int32_t k = 0, int32_t pitch = 0) {
    const int64_t nb = fp8_blocks(ncols), n_blocks = rows * nb;
    constexpr int64_t per = 2 * kQuantWarps * kQuantAhead;
    const int64_t ctas = (n_blocks + per - 1) / per;
    if (n_blocks > 0xFFFF0000LL) return fail(FT_ERR_SIZE, "rows * ceil(ncols / 128) too large for one launch");
    const dim3 grid(static_cast<unsigned>(ctas)), block(32 * kQuantWarps);
    quantize_fp8_kernel<T, GATED, SPREAD><<<grid, block, 0, s>>>(static_cast<const T*>(x), codes, scales, static_cast<uint32_t>(n_blocks),
                                                                static_cast<uint32_t>(nb), ncols, kind, pos, k, pitch);
    return check_launch("quantize_fp8_kernel", grid, block, 0);
}

int launch_quantize_fp8(const void* x, int dtype, uint8_t* codes, float* scales, int64_t rows, int64_t ncols,
                        bool gated, int kind, cudaStream_t s) {
    if (rows == 0) return FT_OK;
    if (dtype == FT_DTYPE_F32)
        return gated ? launch_typed<float, true>(x, codes, scales, rows, ncols, kind, s)
                     : launch_typed<float, false>(x, codes, scales, rows, ncols, kind, s);
    if (dtype == FT_DTYPE_F16)
        return gated ? launch_typed<__half, true>(x, codes, scales, rows, ncols, kind, s)
                     : launch_typed<__half, false>(x, codes, scales, rows, ncols, kind, s);
    return gated ? launch_typed<__nv_bfloat16, true>(x, codes, scales, rows, ncols, kind, s)
                 : launch_typed<__nv_bfloat16, false>(x, codes, scales, rows, ncols, kind, s);
}

int launch_quantize_fp8_spread(const void* x, int dtype, uint8_t* codes, float* scales, int64_t tokens, int64_t ncols,
                               const int32_t* pos, int32_t k, int32_t pitch, cudaStream_t s) {
    if (dtype == FT_DTYPE_F16)
        return launch_typed<__half, false, true>(x, codes, scales, tokens, ncols, FT_ACT_SILU, s, pos, k, pitch);
    return launch_typed<__nv_bfloat16, false, true>(x, codes, scales, tokens, ncols, FT_ACT_SILU, s, pos, k, pitch);
}

}  // namespace ft
