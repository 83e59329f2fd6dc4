// The FP8 products for a handful of slots (one decoded token): every slot by itself on the
// CUDA cores, without ordering, barriers or a pipeline to fill.
//
// A warp takes four weight rows of one slot's expert; a step covers 512 columns, 16 of each
// row per lane in one 16-byte load, so that a lane's 16 lie within one scale block: their
// dot product times 16 sa sw (fp8_dot.cuh) goes to the row's sum.
//
// Bound by latency and by reading the matrices once: 8 slots, 768 x 2048 of 128 experts: 3.8 us
// in a graph, 8.1 with cold caches (12.6 MB: 1.9 us at the copy's rate).
#include "fp8_dot.cuh"
#include "ft_internal.h"

namespace ft {

constexpr int kGemvWarps = 4, kGemvRows = 4;

template <typename TO>
__global__ void __launch_bounds__(32 * kGemvWarps) moe_fp8_gemv_kernel(const Fp8Product p, TO* __restrict__ out, uint32_t* err) {
    const uint32_t lane = lane_id();
    const int64_t s = blockIdx.y;
    const int32_t r0 = (static_cast<int32_t>(blockIdx.x) * kGemvWarps + static_cast<int32_t>(threadIdx.x >> 5)) * kGemvRows;
    const int32_t nrows = static_cast<int32_t>(p.nrows), ncols = static_cast<int32_t>(p.ncols);
    if (r0 >= nrows) return;
    TO* o = out + s * p.nrows + r0;
    const int32_t e = p.ids ? __ldg(p.ids + s) : 0;
    if (e < 0 || e >= p.n_experts) {      // no expert: zeros, and the flag if it is not -1
        if (e != -1 && lane == 0) atomicOr(err, FT_DEVERR_BAD_EXPERT_ID);
        if (static_cast<int32_t>(lane) < min(kGemvRows, nrows - r0)) o[lane] = from_f32<TO>(0.0f);
        return;
    }
    const int32_t nb = (ncols + kFp8Block - 1) / kFp8Block;
    const int64_t a_row = s / p.act_div;
    const uint8_t* act = p.act + a_row * ncols + 16 * lane;
    const float* sa = p.act_scales + a_row * p.scale_pitch;
    const uint8_t* w[kGemvRows];
    const float* sw[kGemvRows];
#pragma unroll
    for (int i = 0; i < kGemvRows; ++i) {      // rows past the end read the last one
        const int32_t r = min(r0 + i, nrows - 1);
        w[i] = p.weights + (static_cast<int64_t>(e) * nrows + r) * ncols + 16 * lane;
        sw[i] = p.w_scales + (static_cast<int64_t>(e) * ((nrows + kFp8Block - 1) / kFp8Block) + r / kFp8Block) * nb;
    }
    float acc[kGemvRows] = {};
#pragma unroll 2
    for (int32_t c = 0; c < ncols; c += 512) {
        if (c + 16 * static_cast<int32_t>(lane) < ncols) {      // ncols % 16 == 0: 16 columns are all inside or all outside
            const uint4 x = __ldg(reinterpret_cast<const uint4*>(act + c));
            uint4 q[kGemvRows];
#pragma unroll
            for (int i = 0; i < kGemvRows; ++i) q[i] = __ldg(reinterpret_cast<const uint4*>(w[i] + c));
            const int32_t b = (c + 16 * static_cast<int32_t>(lane)) / kFp8Block;
            const float scale = __ldg(sa + b) * kActUp;
            uint32_t a[8];
            act_to_f16(x, a);
#pragma unroll
            for (int i = 0; i < kGemvRows; ++i) acc[i] = fmaf(dot16(q[i], a), scale * __ldg(sw[i] + b), acc[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < kGemvRows; ++i)
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) acc[i] += __shfl_xor_sync(0xFFFFFFFFu, acc[i], k);
    if (lane < static_cast<uint32_t>(kGemvRows) && r0 + static_cast<int32_t>(lane) < nrows)
        o[lane] = from_f32<TO>(lane == 0 ? acc[0] : lane == 1 ? acc[1] : lane == 2 ? acc[2] : acc[3]);
}

int launch_fp8_gemv(const Fp8Product& p, void* out, int out_dtype, uint32_t* err, cudaStream_t s) {
    const int64_t per = kGemvWarps * kGemvRows;
    const dim3 grid(static_cast<unsigned>((p.nrows + per - 1) / per), static_cast<unsigned>(p.n_slots)), block(32 * kGemvWarps);
    if (out_dtype == FT_DTYPE_F32) moe_fp8_gemv_kernel<float><<<grid, block, 0, s>>>(p, static_cast<float*>(out), err);
    else moe_fp8_gemv_kernel<__nv_bfloat16><<<grid, block, 0, s>>>(p, static_cast<__nv_bfloat16*>(out), err);
    return check_launch("moe_fp8_gemv_kernel", grid, block, 0);
}

}  // namespace ft
