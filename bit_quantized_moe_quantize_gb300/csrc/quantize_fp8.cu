// Rows -> e4m3 codes with one fp32 scale per 128 columns, and the same of the
// gated activation between the two expert products.
//
//   scale = amax / 448 (IEEE quotient of the block's largest magnitude),
//   code  = e4m3(v / scale), round to nearest even; a block whose scale is 0
//           gets codes 0
//
// Eight lanes take one block of a row: lane i its values 8 i .. and 64 + 8 i .. (columns past
// the row's end count as 0 and are not stored), three shuffles find the largest magnitude.
// The codes are those of the IEEE quotients; see fp8_codes for how most of them come without a
// division.  A non-finite value makes its block's scale infinite or NaN, and what is
// divided by it 0 or NaN.
//
// 16-bit rows are bound by instructions (65528 rows x 1408 gated bf16: 100 us, 4.6 TB/s, issue slots
// 85 % taken, with an activation within 10 * 2^-24 instead of act_mul_f32 78; rows of 2816 bf16 120 us,
// 4.4 TB/s, 71 %), fp32 ones by memory (6.3 and 6.6 TB/s).  CTAs that stay and fetch ahead took longer
// for 16-bit rows: small ones that come and go hide the loads as well, with half the registers.
#include "fp8_quant.cuh"
#include "ft_internal.h"

namespace ft {

constexpr int kQuantWarps = 4, kQuantHalves = 2;      // of a block: eight values of each in a lane

// Eight neighbouring elements, 16-byte aligned.
template <typename T>
__device__ __forceinline__ void load_raw(const T* p, T (&v)[8]) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) reinterpret_cast<uint4*>(v)[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
}

constexpr int kNoAct = -1;

// n / d for 32-bit n as the top of n * (floor((2^64 - 1) / d) + 1), exact for d > 1: a 32-bit
// division takes as many instructions as a lane's eight values.
struct Divider {
    uint32_t d, hi, lo;
    explicit Divider(uint32_t by) : d(by) {
        const uint64_t m = ~uint64_t(0) / by + 1;
        hi = static_cast<uint32_t>(m >> 32);
        lo = static_cast<uint32_t>(m);
    }
    __device__ uint32_t operator()(uint32_t n) const {
        const uint64_t top = static_cast<uint64_t>(n) * hi + __umulhi(n, lo);
        return d == 1 ? n : static_cast<uint32_t>(top >> 32);
    }
};

// ACT: kNoAct, or FT_ACT_*: x holds rows of 2 ncols values, gate then up (a template: both
// activations and a choice took a fifth of the instructions).  SPREAD: the codes and scales of
// row r, a token's (or, k = 1, a slot's), go to the rows pos[r * k ..] (-1: none) of the outputs.
template <typename T, int ACT, bool SPREAD>
__global__ void __launch_bounds__(32 * kQuantWarps)
    quantize_fp8_kernel(const T* __restrict__ x, uint8_t* __restrict__ codes, float* __restrict__ scales,
                        uint32_t n_blocks, const Divider nb, int64_t ncols, const int32_t* __restrict__ pos, int32_t k, int32_t pitch) {
    constexpr bool GATED = ACT != kNoAct;
    const uint32_t sub = lane_id() & 7u;
    const uint32_t at = (blockIdx.x * kQuantWarps + (threadIdx.x >> 5)) * 4 + (lane_id() >> 3);
    const uint32_t r = at < n_blocks ? nb(at) : 0u, b = at < n_blocks ? at - r * nb.d : 0u;
    const int64_t row = r, col = static_cast<int64_t>(b) * kFp8Block + 8 * sub;
    // all values are asked for before the first is worked on; ncols % 16 == 0: eight are all inside or all outside
    __align__(16) T raw[kQuantHalves][GATED ? 2 : 1][8];
    bool in[kQuantHalves];
#pragma unroll
    for (int n = 0; n < kQuantHalves; ++n) {
        in[n] = at < n_blocks && col + 64 * n < ncols;
        if (in[n]) {
            const T* src = x + row * (GATED ? 2 : 1) * ncols + col + 64 * n;
            load_raw(src, raw[n][0]);
            if constexpr (GATED) load_raw(src + ncols, raw[n][1]);
        }
    }
    float v[kQuantHalves][8] = {};
#pragma unroll
    for (int n = 0; n < kQuantHalves; ++n) {
        if (in[n]) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (GATED) v[n][j] = act_mul_f32(to_f32<T>(raw[n][0][j]), to_f32<T>(raw[n][1][j]), ACT);
                else v[n][j] = to_f32<T>(raw[n][0][j]);
            }
        }
    }
    const float scale = fp8_block_scale(v), inv = rcp_approx(scale);
    uint2 q[kQuantHalves];
#pragma unroll
    for (int n = 0; n < kQuantHalves; ++n) q[n] = fp8_codes(v[n], scale, inv);
    if (at >= n_blocks) return;
    if constexpr (SPREAD) {
        for (int32_t j = 0; j < k; ++j) {
            const int64_t p = __ldg(pos + row * k + j);
            if (p < 0) continue;
#pragma unroll
            for (int n = 0; n < kQuantHalves; ++n)
                if (in[n]) *reinterpret_cast<uint2*>(codes + p * ncols + col + 64 * n) = q[n];
            if (sub == 0) scales[p * pitch + b] = scale;
        }
    } else {
#pragma unroll
        for (int n = 0; n < kQuantHalves; ++n)
            if (in[n]) *reinterpret_cast<uint2*>(codes + row * ncols + col + 64 * n) = q[n];
        if (sub == 0) scales[at] = scale;
    }
}

template <typename T, int ACT, bool SPREAD = false>
static int launch_typed(const void* x, uint8_t* codes, float* scales, int64_t rows, int64_t ncols, cudaStream_t s,
                        const int32_t* pos = nullptr, int32_t k = 0, int32_t pitch = 0) {
    const int64_t nb = fp8_blocks(ncols), n_blocks = rows * nb;
    constexpr int64_t per = 4 * kQuantWarps;
    const int64_t ctas = (n_blocks + per - 1) / per;
    if (n_blocks > 0xFFFF0000LL) return fail(FT_ERR_SIZE, "rows * ceil(ncols / 128) too large for one launch");
    const dim3 grid(static_cast<unsigned>(ctas)), block(32 * kQuantWarps);
    quantize_fp8_kernel<T, ACT, SPREAD><<<grid, block, 0, s>>>(static_cast<const T*>(x), codes, scales, static_cast<uint32_t>(n_blocks),
                                                              Divider(static_cast<uint32_t>(nb)), ncols, pos, k, pitch);
    return check_launch("quantize_fp8_kernel", grid, block, 0);
}

template <typename T>
static int launch_act(const void* x, uint8_t* codes, float* scales, int64_t rows, int64_t ncols, bool gated, int kind, cudaStream_t s) {
    if (!gated) return launch_typed<T, kNoAct>(x, codes, scales, rows, ncols, s);
    return kind == FT_ACT_SILU ? launch_typed<T, FT_ACT_SILU>(x, codes, scales, rows, ncols, s)
                               : launch_typed<T, FT_ACT_GELU_TANH>(x, codes, scales, rows, ncols, s);
}

int launch_quantize_fp8(const void* x, int dtype, uint8_t* codes, float* scales, int64_t rows, int64_t ncols,
                        bool gated, int kind, cudaStream_t s) {
    if (rows == 0) return FT_OK;
    if (dtype == FT_DTYPE_F32) return launch_act<float>(x, codes, scales, rows, ncols, gated, kind, s);
    if (dtype == FT_DTYPE_F16) return launch_act<__half>(x, codes, scales, rows, ncols, gated, kind, s);
    return launch_act<__nv_bfloat16>(x, codes, scales, rows, ncols, gated, kind, s);
}

int launch_quantize_fp8_spread(const void* x, int dtype, uint8_t* codes, float* scales, int64_t rows, int64_t ncols,
                               bool gated, int kind, const int32_t* pos, int32_t k, int32_t pitch, cudaStream_t s) {
    if (dtype == FT_DTYPE_F32) {      // the gated rows between the products; x itself is 16-bit
        if (!gated) return fail(FT_ERR_ARG, "rows spread to router order are 16-bit, or gated fp32");
        return kind == FT_ACT_SILU ? launch_typed<float, FT_ACT_SILU, true>(x, codes, scales, rows, ncols, s, pos, k, pitch)
                                   : launch_typed<float, FT_ACT_GELU_TANH, true>(x, codes, scales, rows, ncols, s, pos, k, pitch);
    }
    if (gated) return fail(FT_ERR_ARG, "gated rows spread to router order are fp32");
    if (dtype == FT_DTYPE_F16) return launch_typed<__half, kNoAct, true>(x, codes, scales, rows, ncols, s, pos, k, pitch);
    return launch_typed<__nv_bfloat16, kNoAct, true>(x, codes, scales, rows, ncols, s, pos, k, pitch);
}

}  // namespace ft
