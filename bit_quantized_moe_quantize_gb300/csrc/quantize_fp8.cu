// Rows -> e4m3 codes with one fp32 scale per 128 columns, and the same of the
// gated activation between the two expert products.
//
//   scale = amax / 448 (IEEE quotient of the block's largest magnitude),
//   code  = e4m3(v / scale), round to nearest even; a block whose scale is 0
//           gets codes 0
//
// A warp takes one block of a row: lane i its values 4 i .. 4 i + 3 (columns
// past the row's end count as 0 and are not stored), five shuffles find the
// largest magnitude.  Both quotients are IEEE divisions, so the codes are those
// of any IEEE evaluation of the formula.  A non-finite value makes its block's
// scale infinite or NaN, and what is divided by it 0 or NaN.
#include "fp8_common.cuh"
#include "ft_internal.h"

namespace ft {

constexpr int kQuantWarps = 8;

// The gated activation of one value: act(g) * up with act(g) = g / (1 + exp(-z)),
// z = g for SiLU and 2 sqrt(2/pi) (g + 0.044715 g^3) for the tanh form of GELU.
__device__ __forceinline__ float act_mul_f32(float g, float up, int kind) {
    const float cube = __fmul_rn(__fmul_rn(__fmul_rn(0.044715f, g), g), g);
    const float z = kind == FT_ACT_SILU ? g : __fmul_rn(1.5957691216057308f, __fadd_rn(g, cube));
    return __fdiv_rn(g, 1.0f + expf(-z)) * up;
}

// GATED: x holds rows of 2 ncols values, gate then up.  SPREAD: row r is a token's, and
// its codes and scales go to the rows pos[r * k ..] (-1: none) of the outputs.
template <typename T, bool GATED, bool SPREAD>
__global__ void __launch_bounds__(32 * kQuantWarps)
    quantize_fp8_kernel(const T* __restrict__ x, uint8_t* __restrict__ codes, float* __restrict__ scales,
                        int64_t n_blocks, int32_t nb, int64_t ncols, int kind, const int32_t* __restrict__ pos, int32_t k,
                        int32_t pitch) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kQuantWarps + (threadIdx.x >> 5);
    if (i >= n_blocks) return;
    const int64_t row = i / nb;
    const int64_t c = (i - row * nb) * kFp8Block + 4 * static_cast<int64_t>(lane_id());
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < ncols) {      // ncols % 16 == 0: a lane's four values are all inside or all outside
        if constexpr (GATED) {
            float g[4], u[4];
            load_vec<T, 4>(x + row * 2 * ncols + c, g);
            load_vec<T, 4>(x + row * 2 * ncols + ncols + c, u);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = act_mul_f32(g[j], u[j], kind);
        } else {
            load_vec<T, 4>(x + row * ncols + c, v);
        }
    }
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) amax = fmaxf(amax, fabsf(v[j]));
    bool nan = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) nan |= v[j] != v[j];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    if (__any_sync(0xFFFFFFFFu, nan)) amax = NAN;
    const float scale = __fdiv_rn(amax, kFp8Max);
    uint32_t q = 0;
    if (c < ncols && scale != 0.0f)
        q = e4m3x4(__fdiv_rn(v[0], scale), __fdiv_rn(v[1], scale), __fdiv_rn(v[2], scale), __fdiv_rn(v[3], scale));
    if constexpr (SPREAD) {
        for (int32_t j = 0; j < k; ++j) {
            const int64_t p = __ldg(pos + row * k + j);
            if (p >= 0) {
                if (c < ncols) *reinterpret_cast<uint32_t*>(codes + p * ncols + c) = q;
                if (lane_id() == 0) scales[p * pitch + (i - row * nb)] = scale;
            }
        }
    } else {
        if (lane_id() == 0) scales[i] = scale;
        if (c < ncols) *reinterpret_cast<uint32_t*>(codes + row * ncols + c) = q;
    }
}

template <typename T, bool GATED, bool SPREAD = false>
static int launch_typed(const void* x, uint8_t* codes, float* scales, int64_t rows, int64_t ncols, int kind,
                        cudaStream_t s, const int32_t* pos = nullptr, int32_t k = 0, int32_t pitch = 0) {
    const int64_t nb = fp8_blocks(ncols), n_blocks = rows * nb;
    const int64_t ctas = (n_blocks + kQuantWarps - 1) / kQuantWarps;
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
