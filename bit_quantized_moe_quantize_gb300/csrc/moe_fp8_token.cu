// An expert layer for a few decoded tokens, after the router, in two launches.
//
//   token_gated: quantizes the token's row of x (in every CTA, into shared memory), takes its
//     dot products with gate and up rows of one slot's expert, and writes act(gate) * up in fp32
//   token_down: quantizes each slot's activated row (a warp per slot, into shared memory),
//     takes its dot products with rows of w2, four at a time, and adds the slots' sums with
//     their weights, in the order of the slots
//
// The grids hold a few CTAs per SM, and a CTA goes over several groups of rows: with one
// group each, quantizing the row again and again took eight tokens 130 us.
//
// Reading the experts' matrices once is what is left to wait for, beside the launches: the
// same pieces as separate launches (quantizer, product, quantizer, product, weighted sum)
// take six.  Every value is rounded as those do, with the second product's rows in fp32.  One
// token, 8 of 128 experts, 2048 and 768 wide: 19 us with the router in a graph, 30 with cold caches
// (38 MB: 5.6 us at the copy's rate).
//
// Each launch may start before the one before it has ended (programmatic dependent launch):
// what it reads of that one's results comes after griddepcontrol.wait, and nothing is
// written before it.
#include "fp8_dot.cuh"
#include "fp8_quant.cuh"
#include "ft_internal.h"

namespace ft {

// CTAs per SM: 2, 3, 4 take (us) 36.5, 30.5, 31.6 for one token, 8 slots, 2048 and 768 wide; 30.8, 27.6,
// 29.7 for 4 tokens, 8 slots, 1024 and 384.
constexpr int kTokenWarps = 8, kPairs = 2, kDownRows = 4, kCtasPerSm = 3;

__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Quantizes n values (a multiple of 16) by `warps` warps into codes and scales in shared memory.
// fp32 rows are the launch before's results.
template <typename T>
__device__ __forceinline__ void quantize_row(const T* x, int32_t n, uint8_t* codes, float* scales, uint32_t warp,
                                             uint32_t warps) {
    const uint32_t sub = lane_id() & 15u;
    const int32_t nb = (n + kFp8Block - 1) / kFp8Block;
    constexpr int AHEAD = 4;      // block pairs whose values are on their way at once
    for (int32_t b0 = 2 * static_cast<int32_t>(warp); b0 < nb; b0 += 2 * AHEAD * static_cast<int32_t>(warps)) {
        float v[AHEAD][1][8] = {};
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int32_t c = (b0 + 2 * i * static_cast<int32_t>(warps) + static_cast<int32_t>(lane_id() >> 4)) * kFp8Block + 8 * static_cast<int32_t>(sub);
            if (c < n) {
                if constexpr (sizeof(T) == 4) load_vec_plain<8>(x + c, v[i][0]);
                else load_vec<T, 8>(x + c, v[i][0]);
            }
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int32_t b = b0 + 2 * i * static_cast<int32_t>(warps) + static_cast<int32_t>(lane_id() >> 4);
            const int32_t c = b * kFp8Block + 8 * static_cast<int32_t>(sub);
            if (b0 + 2 * i * static_cast<int32_t>(warps) < nb) {      // the whole warp
                const float scale = fp8_block_scale(v[i]);
                if (c < n) *reinterpret_cast<uint2*>(codes + c) = fp8_codes(v[i][0], scale, rcp_approx(scale));
                if (sub == 0 && b < nb) scales[b] = scale;
            }
        }
    }
}

// Dot products of R rows (w: with the lane's offset; sw: their scales) with a quantized row in shared memory.
template <int R>
__device__ __forceinline__ void dot_rows(const uint8_t* const (&w)[R], const float* const (&sw)[R], int32_t n, const uint8_t* codes,
                                         const float* scales, float (&acc)[R]) {
    const int32_t l = 16 * static_cast<int32_t>(lane_id());
#pragma unroll 2
    for (int32_t c = 0; c < n; c += 512) {
        if (c + l < n) {
            uint4 q[R];
#pragma unroll
            for (int i = 0; i < R; ++i) q[i] = __ldg(reinterpret_cast<const uint4*>(w[i] + c));
            const int32_t b = (c + l) / kFp8Block;
            const float scale = scales[b] * kActUp;
            uint32_t a[8];
            act_to_f16(*reinterpret_cast<const uint4*>(codes + c + l), a);
#pragma unroll
            for (int i = 0; i < R; ++i) acc[i] = fmaf(dot16(q[i], a), scale * __ldg(sw[i] + b), acc[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) acc[i] += __shfl_xor_sync(0xFFFFFFFFu, acc[i], k);
}

// grid: (CTAs per slot, slots)
template <typename T>
__global__ void __launch_bounds__(32 * kTokenWarps)
    token_gated_kernel(const T* __restrict__ x, const uint8_t* __restrict__ w13, const float* __restrict__ s13,
                       const int32_t* ids, float* mid, int32_t n_experts, int32_t top_k, int32_t hidden,
                       int32_t n_inter, int kind) {
    extern __shared__ __align__(16) uint8_t row_smem[];
    float* scales = reinterpret_cast<float*>(row_smem + hidden);
    const uint32_t warp = threadIdx.x >> 5;
    const int64_t s = blockIdx.y;
    grid_launch_dependents();
    quantize_row<T>(x + s / top_k * hidden, hidden, row_smem, scales, warp, kTokenWarps);
    __syncthreads();
    grid_dependency_wait();      // the router's choice
    const int32_t e = ids[s];
    if (e < 0 || e >= n_experts) return;
    const int32_t nb = (hidden + kFp8Block - 1) / kFp8Block, blocks = (2 * n_inter + kFp8Block - 1) / kFp8Block;
    const int32_t step = static_cast<int32_t>(gridDim.x) * kTokenWarps * kPairs;
    for (int32_t i0 = (static_cast<int32_t>(blockIdx.x) * kTokenWarps + static_cast<int32_t>(warp)) * kPairs; i0 < n_inter; i0 += step) {
        const uint8_t* w[2 * kPairs];
        const float* sw[2 * kPairs];
#pragma unroll
        for (int i = 0; i < 2 * kPairs; ++i) {      // gate rows, then up rows; past the end the last one again
            const int32_t r = min(i0 + i % kPairs, n_inter - 1) + (i < kPairs ? 0 : n_inter);
            w[i] = w13 + (static_cast<int64_t>(e) * 2 * n_inter + r) * hidden + 16 * lane_id();
            sw[i] = s13 + (static_cast<int64_t>(e) * blocks + r / kFp8Block) * nb;
        }
        float acc[2 * kPairs] = {};
        dot_rows<2 * kPairs>(w, sw, hidden, row_smem, scales, acc);
#pragma unroll
        for (int i = 0; i < kPairs; ++i)
            if (lane_id() == static_cast<uint32_t>(i) && i0 + i < n_inter)
                mid[s * n_inter + i0 + i] = act_mul_f32(acc[i], acc[kPairs + i], kind);
    }
}

// grid: (CTAs per token, tokens); a CTA takes `groups` neighbouring groups of rows.
template <typename TO>
__global__ void __launch_bounds__(32 * kTokenWarps)
    token_down_kernel(const float* mid, const uint8_t* __restrict__ w2, const float* __restrict__ s2,
                      const int32_t* ids, const float* weights, TO* y, int32_t n_experts,
                      int32_t top_k, int32_t hidden, int32_t n_inter, int32_t warp_bytes, int32_t groups) {
    extern __shared__ __align__(16) uint8_t row_smem[];      // per warp codes[n_inter], scales; then sums[groups][top_k][kDownRows]
    const uint32_t warp = threadIdx.x >> 5, lane = lane_id();
    uint8_t* codes = row_smem + warp * static_cast<uint32_t>(warp_bytes);
    float* scales = reinterpret_cast<float*>(codes + n_inter);
    float* sums = reinterpret_cast<float*>(row_smem + kTokenWarps * static_cast<uint32_t>(warp_bytes));
    const int64_t t = blockIdx.y;
    const int32_t r0 = static_cast<int32_t>(blockIdx.x) * groups * kDownRows;
    const int32_t nb = (n_inter + kFp8Block - 1) / kFp8Block, blocks = (hidden + kFp8Block - 1) / kFp8Block;
    grid_dependency_wait();
    for (int32_t j = static_cast<int32_t>(warp); j < top_k; j += kTokenWarps) {
        const int64_t s = t * top_k + j;
        const int32_t e = ids[s];
        const bool routed = e >= 0 && e < n_experts;
        if (routed) {
            __syncwarp();
            quantize_row<float>(mid + s * n_inter, n_inter, codes, scales, 0, 1);
            __syncwarp();
        }
        for (int32_t g = 0; g < groups; ++g) {
            const int32_t rg = r0 + g * kDownRows;
            if (rg >= hidden) break;
            float acc[kDownRows] = {};
            if (routed) {
                const uint8_t* w[kDownRows];
                const float* sw[kDownRows];
#pragma unroll
                for (int i = 0; i < kDownRows; ++i) {
                    const int32_t r = min(rg + i, hidden - 1);
                    w[i] = w2 + (static_cast<int64_t>(e) * hidden + r) * n_inter + 16 * lane;
                    sw[i] = s2 + (static_cast<int64_t>(e) * blocks + r / kFp8Block) * nb;
                }
                dot_rows<kDownRows>(w, sw, n_inter, codes, scales, acc);
            }
#pragma unroll
            for (int i = 0; i < kDownRows; ++i)
                if (lane == static_cast<uint32_t>(i)) sums[(g * top_k + j) * kDownRows + i] = acc[i];
        }
    }
    __syncthreads();
    for (int32_t i = static_cast<int32_t>(threadIdx.x); i < groups * kDownRows; i += 32 * kTokenWarps) {
        const int32_t r = r0 + i;
        if (r >= hidden) break;
        float sum = 0.0f;
        for (int32_t j = 0; j < top_k; ++j) {
            const float wj = weights[t * top_k + j];
            if (wj != 0.0f) sum = fmaf(wj, sums[(i / kDownRows * top_k + j) * kDownRows + i % kDownRows], sum);
        }
        y[t * hidden + r] = from_f32<TO>(sum);
    }
}

// ------------------------------------------------------------------- host
namespace {

int32_t down_warp_bytes(int64_t n_inter) { return static_cast<int32_t>((n_inter + 4 * fp8_blocks(n_inter) + 15) / 16 * 16); }

// Groups of rows of w2 per CTA: as many as leave a few CTAs per SM.
int32_t down_groups(int64_t tokens, int64_t hidden) {
    const int64_t all = (hidden + kDownRows - 1) / kDownRows;
    int64_t ctas = kCtasPerSm * static_cast<int64_t>(sm_count()) / tokens;
    ctas = ctas < 1 ? 1 : ctas < all ? ctas : all;
    return static_cast<int32_t>((all + ctas - 1) / ctas);
}

size_t down_smem(int64_t n_inter, int32_t top_k, int32_t groups) {
    return static_cast<size_t>(kTokenWarps) * down_warp_bytes(n_inter) + static_cast<size_t>(groups) * top_k * kDownRows * 4;
}

template <typename... A>
int launch_dependent(void (*kernel)(A...), const char* name, dim3 grid, size_t smem, cudaStream_t s, A... args) {
    if (smem > 48 * 1024)
        if (int st = set_smem_limit(reinterpret_cast<const void*>(kernel), static_cast<int>(smem))) return st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(32 * kTokenWarps);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    c.attrs = at;
    c.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&c, kernel, args...);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(FT_ERR_LAUNCH, "launch of %s failed: %s", name, cudaGetErrorString(e));
    }
    return check_launch(name, grid, c.blockDim, smem);
}

}  // namespace

bool fp8_token_ok(int64_t n_slots, int64_t tokens, int32_t top_k, int64_t hidden, int64_t n_inter) {
    // The more the matrices' reading takes, the less the launches saved count, and the separate
    // kernels' warps, which are not tied to slots, read them faster.  Times (us, cold, these kernels /
    // separate; tokens x slots, hidden, n_inter):
    //   6 MB   1x1 2048 1024 25/27;   13 MB  4x2 1024 512 20/25, 1x1 4096 1024 35/31;   14 MB 1x8 768 768 22/29
    //   25 MB  1x8 2048 512 25/29, 8x8 512 256 22/31, 1x2 2048 1792 33/30 (22 MB)
    //   38 MB  1x8 2048 768 30/32, 1x8 1024 1536 28/33, 2x8 2048 384 28/34, 1x4 2048 1536 32/33, 1x2 4096 1536 41/37
    //   50 MB  1x8 2048 1024 36/33, 1x8 1024 2048 34/38, 4x8 1024 512 30/36, 1x4 4096 1024 39/38, 1x2 4096 2048 46/40
    //   75 MB  1x8 4096 768 43/46, 8x8 1024 384 37/43;  65 MB 1x6 2560 1408 43/40, 63 MB 1x10 2048 1024 46/45
    //   100 MB 4x8 2048 512 47/49;  113 MB 3x8 2048 768 53/51;  142 MB 1x6 5120 1536 71/58
    // From 25 to 100 MB neither is ahead for all shapes, by 10 % or so either way (with few slots of
    // large matrices the separate ones); 40 MB lies between.
    if (3 * n_slots * hidden * n_inter > 40'000'000) return false;
    return n_slots <= 65535 && tokens <= 65535 && hidden + 4 * fp8_blocks(hidden) <= 200 * 1024 &&
           down_smem(n_inter, top_k, down_groups(tokens, hidden)) <= 200 * 1024;
}

int launch_fp8_token_layer(const void* x, int x_dtype, const uint8_t* w13, const float* s13, const uint8_t* w2, const float* s2,
                           const int32_t* ids, const float* weights, float* mid, void* y, int64_t tokens, int32_t top_k,
                           int32_t n_experts, int64_t hidden, int64_t n_inter, int kind, cudaStream_t s) {
    const int32_t H = static_cast<int32_t>(hidden), I = static_cast<int32_t>(n_inter);
    const int64_t slots = tokens * top_k, most = (n_inter + kTokenWarps * kPairs - 1) / (kTokenWarps * kPairs);
    const int64_t fit = kCtasPerSm * static_cast<int64_t>(sm_count()) / slots, ctas = fit > 0 ? fit : 1;
    const int32_t groups = down_groups(tokens, hidden);
    const int64_t per = static_cast<int64_t>(groups) * kDownRows;
    const dim3 g1(static_cast<unsigned>(ctas < most ? ctas : most), static_cast<unsigned>(slots));
    const dim3 g2(static_cast<unsigned>((hidden + per - 1) / per), static_cast<unsigned>(tokens));
    const size_t sm1 = static_cast<size_t>(hidden + 4 * fp8_blocks(hidden)), sm2 = down_smem(n_inter, top_k, groups);
    const int32_t wb = down_warp_bytes(n_inter);
    int st;
    if (x_dtype == FT_DTYPE_F16)
        st = launch_dependent(token_gated_kernel<__half>, "token_gated_kernel", g1, sm1, s, static_cast<const __half*>(x), w13, s13, ids,
                              mid, n_experts, top_k, H, I, kind);
    else
        st = launch_dependent(token_gated_kernel<__nv_bfloat16>, "token_gated_kernel", g1, sm1, s, static_cast<const __nv_bfloat16*>(x),
                              w13, s13, ids, mid, n_experts, top_k, H, I, kind);
    if (st) return st;
    const float* m = mid;
    if (x_dtype == FT_DTYPE_F16)
        return launch_dependent(token_down_kernel<__half>, "token_down_kernel", g2, sm2, s, m, w2, s2, ids, weights,
                                static_cast<__half*>(y), n_experts, top_k, H, I, wb, groups);
    return launch_dependent(token_down_kernel<__nv_bfloat16>, "token_down_kernel", g2, sm2, s, m, w2, s2, ids, weights,
                            static_cast<__nv_bfloat16*>(y), n_experts, top_k, H, I, wb, groups);
}

}  // namespace ft
