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

constexpr int kQuantWarps = 8;

// GATED: x holds rows of 2 ncols values, gate then up.  SPREAD: row r is a token's, and
// its codes and scales go to the rows pos[r * k ..] (-1: none) of the outputs.
template <typename T, bool GATED, bool SPREAD>
__global__ void __launch_bounds__(32 * kQuantWarps)
    quantize_fp8_kernel(const T* __restrict__ x, uint8_t* __restrict__ codes, float* __restrict__ scales,
                        int64_t n_blocks, int32_t nb, int64_t ncols, int kind, const int32_t* __restrict__ pos, int32_t k,
                        int32_t pitch) {
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * kQuantWarps + (threadIdx.x >> 5)) * 2 + (lane_id() >> 4);
    const uint32_t sub = lane_id() & 15u;
    const bool there = i < n_blocks;
    const int64_t row = there ? i / nb : 0;
    const int64_t c = (there ? i - row * nb : 0) * kFp8Block + 8 * static_cast<int64_t>(sub);
    const bool in = there && c < ncols;      // ncols % 16 == 0: a lane's eight values are all inside or all outside
    float v[8] = {};
    if (in) {
        if constexpr (GATED) {
            float g[8], u[8];
            load_vec<T, 8>(x + row * 2 * ncols + c, g);
            load_vec<T, 8>(x + row * 2 * ncols + ncols + c, u);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = act_mul_f32(g[j], u[j], kind);
        } else {
            load_vec<T, 8>(x + row * ncols + c, v);
        }
    }
    const float scale = fp8_block_scale(v);
    if (!in) return;
    const uint2 q = fp8_codes(v, scale);
    if constexpr (SPREAD) {
        for (int32_t j = 0; j < k; ++j) {
            const int64_t p = __ldg(pos + row * k + j);
            if (p >= 0) {
                *reinterpret_cast<uint2*>(codes + p * ncols + c) = q;
                if (sub == 0) scales[p * pitch + (i - row * nb)] = scale;
            }
        }
    } else {
        if (sub == 0) scales[i] = scale;
        *reinterpret_cast<uint2*>(codes + row * ncols + c) = q;
    }
}

template <typename T, bool GATED, bool SPREAD = false>
static int launch_typed(const void* x, uint8_t* codes, float* scales, int64_t rows, int64_t ncols, int kind,
                        cudaStream_t s, const int32_t* pos = nullptr, int32_t k = 0, int32_t pitch = 0) {
    const int64_t nb = fp8_blocks(ncols), n_blocks = rows * nb;
    const int64_t ctas = (n_blocks + 2 * kQuantWarps - 1) / (2 * kQuantWarps);
    if (ctas > 0x7FFFFFFF) return fail(FT_ERR_SIZE, "rows * ncols too large for one launch");
    const dim3 grid(static_cast<unsigned>(ctas)), block(32 * kQuantWarps);
    quantize_fp8_kernel<T, GATED, SPREAD><<<grid, block, 0, s>>>(static_cast<const T*>(x), codes, scales, n_blocks,
                                                                static_cast<int32_t>(nb), ncols, kind, pos, k, pitch);
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
