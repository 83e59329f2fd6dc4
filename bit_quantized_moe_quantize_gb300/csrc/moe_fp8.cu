// Routed expert products in 8-bit floating point with a scale per block of 128:
//
//   out[s][r] = sum_b sa[row(s)][b] sw[e][r / 128][b] sum_{i in block b} w[e][r][i] a[row(s)][i]
//
// with e = topk_ids[s] and row(s) = s / act_div (act_div = top_k: one
// activation row per token; 1: one per slot), and the dense product (one
// matrix, slot s = row s).  Products of e4m3 values are summed in fp32.
//
// A warp takes kRows weight rows of one slot's expert; in each step its lanes
// cover one scale block, lane i the values 4 i .. 4 i + 3.
#include "fp8_common.cuh"
#include "ft_internal.h"

namespace ft {

constexpr int kFp8Warps = 8, kFp8Rows = 8;

__device__ __forceinline__ void e4m3x4_to_f32(uint32_t q, float (&v)[4]) {
    uint32_t lo, hi;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(static_cast<uint16_t>(q & 0xFFFFu)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(static_cast<uint16_t>(q >> 16)));
    const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo)), b = __half22float2(*reinterpret_cast<__half2*>(&hi));
    v[0] = a.x;
    v[1] = a.y;
    v[2] = b.x;
    v[3] = b.y;
}

template <typename TO>
__global__ void __launch_bounds__(32 * kFp8Warps) moe_fp8_kernel(const Fp8Product p, TO* __restrict__ out,
                                                                uint32_t* err) {
    const uint32_t lane = lane_id();
    const int64_t s = blockIdx.x;
    const int64_t r0 = (static_cast<int64_t>(blockIdx.y) * kFp8Warps + (threadIdx.x >> 5)) * kFp8Rows;
    const int32_t e = p.ids ? p.ids[s] : 0;
    if (e < 0 || e >= p.n_experts) {
        if (e != -1 && threadIdx.x == 0) atomicOr(err, FT_DEVERR_BAD_EXPERT_ID);
        for (int64_t r = r0 + lane; r < min(p.nrows, r0 + kFp8Rows); r += 32) out[s * p.nrows + r] = from_f32<TO>(0.0f);
        return;
    }
    const int64_t nb = fp8_blocks(p.ncols), a_row = s / p.act_div;
    const uint8_t* act = p.act + a_row * p.ncols;
    const uint8_t* w = p.weights + static_cast<int64_t>(e) * p.nrows * p.ncols;
    const float* sw = p.w_scales + static_cast<int64_t>(e) * fp8_blocks(p.nrows) * nb;
    float acc[kFp8Rows] = {};
    for (int64_t b = 0; b < nb; ++b) {
        const int64_t c = b * kFp8Block + 4 * lane;
        if (c >= p.ncols) break;
        float x[4], v[4];
        e4m3x4_to_f32(__ldg(reinterpret_cast<const uint32_t*>(act + c)), x);
        const float sa = p.act_scales[a_row * nb + b];
#pragma unroll
        for (int i = 0; i < kFp8Rows; ++i) {
            const int64_t r = r0 + i;
            if (r < p.nrows) {
                e4m3x4_to_f32(__ldg(reinterpret_cast<const uint32_t*>(w + r * p.ncols + c)), v);
                const float d = x[0] * v[0] + x[1] * v[1] + x[2] * v[2] + x[3] * v[3];
                acc[i] = fmaf(d, sa * sw[r / kFp8Block * nb + b], acc[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kFp8Rows; ++i) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc[i] += __shfl_xor_sync(0xFFFFFFFFu, acc[i], o);
        if (lane == 0 && r0 + i < p.nrows) out[s * p.nrows + r0 + i] = from_f32<TO>(acc[i]);
    }
}

size_t fp8_product_workspace(int64_t n_slots, int32_t n_experts) { return 0; }

int launch_fp8_product(const Fp8Product& p, void* out, int out_dtype, void* workspace, uint32_t* err, cudaStream_t s) {
    const int64_t row_ctas = (p.nrows + kFp8Warps * kFp8Rows - 1) / (kFp8Warps * kFp8Rows);
    if (row_ctas > 65535) return fail(FT_ERR_SIZE, "nrows too large");
    const dim3 grid(static_cast<unsigned>(p.n_slots), static_cast<unsigned>(row_ctas)), block(32 * kFp8Warps);
    if (out_dtype == FT_DTYPE_F32) moe_fp8_kernel<float><<<grid, block, 0, s>>>(p, static_cast<float*>(out), err);
    else moe_fp8_kernel<__nv_bfloat16><<<grid, block, 0, s>>>(p, static_cast<__nv_bfloat16*>(out), err);
    return check_launch("moe_fp8_kernel", grid, block, 0);
}

}  // namespace ft
