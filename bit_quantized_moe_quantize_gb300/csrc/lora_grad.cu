// Gradients of the adapters' matrices, sums over the slots of an adapter:
//
//   dA[r][k] = sum_s v[s][r] x[s][k]      v = scale B^T dy
//   dB[n][r] = sum_s dy[s][n] u[s][r]     u = scale A x
//
// for fp16 adapters, and what follows for all: lora_grad_tc.cu has the kernel for bf16.
//
// A CTA takes a chunk of an adapter's slots and 256 columns (128 for ranks above 64).  z's rows come by cp.async, 32 slots a
// stage; the narrow side's fp32 values go through shared memory as they are and are split into two tf32 parts in
// registers, beside fp16 turned to tf32, which is exact: the narrow side needs more exponents than fp16 has.  The sums lie in
// registers; an adapter with several chunks leaves them in the workspace, where a second launch adds them up in order.
// That launch also writes the zeros of adapters without a slot.
//
// 509 slots, rank 24, 1000 and 1416 columns, 6 adapters: 9 us, 5 more to join: a chunk's chain of two stages and
// little to do beside it.
//
// Chunk j of adapter e has number offsets[e] / per + e + j: chunks of `per` slots never need more numbers than that leaves.
#include <algorithm>

#include "lora_grad.cuh"

namespace ft {

namespace {

constexpr int kGradSlots = 32, kGradStages = 3, kGradRing = 8;

// MR: tiles of 16 ranks that there is room for; NJ: tiles of eight columns that a warp has.
template <int MR, int NJ>
__global__ void __launch_bounds__(kGradThreads, 2) lora_grad_kernel(const __grid_constant__ GradArgs<__half> a) {
    using T = __half;
    constexpr int CC = 8 * NJ * (kGradThreads / 32), ZP = CC + 8;      // columns of the CTA, their pitch
    constexpr int PAIRS = MR;      // pairs of ranks that a thread has of a stage
    extern __shared__ __align__(16) uint8_t grad_smem[];
    const int32_t tid = static_cast<int32_t>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    const bool second = static_cast<int32_t>(blockIdx.y) >= a.blocks0;
    const GradJob<T>& job = a.job[second ? 1 : 0];
    const int32_t col0 = (static_cast<int32_t>(blockIdx.y) - (second ? a.blocks0 : 0)) * CC;
    const Chunk ck = find_chunk<kGradThreads>(a.slots, static_cast<int32_t>(blockIdx.x), a.per);
    if (ck.n == 0) {
        wait_for_prior_grid();
        return;
    }
    const int32_t R = a.rank, r16 = (R + 15) / 16 * 16, mr = r16 / 16, cols = job.cols;
    const int32_t wf = r16 + 4, w_bytes = kGradSlots * wf * 4;      // pitch of w's rows: lanes' pairs of slots in different banks
    T* zs_all = reinterpret_cast<T*>(grad_smem);
    uint8_t* ws_all = grad_smem + kGradStages * kGradSlots * ZP * sizeof(T);
    __shared__ int32_t ring[kGradRing][kGradSlots];      // slots of the stages from the one at work on
    const int32_t* perm = a.slots.perm + ck.first;
    const float scale = a.scales ? __ldg(a.scales + ck.adapter) : 1.0f;
    const int32_t steps = (ck.n + kGradSlots - 1) / kGradSlots;

    // z: thread by 16-byte words of a row
    constexpr int ZW = CC / 8, ZROWS = kGradThreads / ZW, ZI = kGradSlots / ZROWS;
    const int32_t zc = tid % ZW * 8;
    auto load_z = [&](int32_t i) {
        T* zs = zs_all + i % kGradStages * kGradSlots * ZP;
#pragma unroll
        for (int j = 0; j < ZI; ++j) {
            const int32_t row = tid / ZW + ZROWS * j, s = i * kGradSlots + row;
            const bool there = s < ck.n && col0 + zc < cols;
            const T* src = there ? job.z + static_cast<int64_t>(ring[i % kGradRing][row] / job.div) * cols + col0 + zc : job.z;
            copy16(zs + row * ZP + zc, src, there);
        }
    };
    // w: pairs of ranks, by slot and then by pair
    float2 wreg[PAIRS];
    auto load_w = [&](int32_t i) {
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) {
            const int32_t at = tid + j * kGradThreads, row = at / (8 * mr), r = (at - row * 8 * mr) * 2, s = i * kGradSlots + row;
            wreg[j] = make_float2(0.0f, 0.0f);
            if (j < mr && s < ck.n && r < R) {
                const float2 v = *reinterpret_cast<const float2*>(job.w + static_cast<int64_t>(ring[i % kGradRing][row]) * R + r);
                wreg[j] = make_float2(v.x * scale, v.y * scale);
            }
        }
    };
    auto store_w = [&](int32_t i) {
        uint8_t* ws = ws_all + i % 2 * w_bytes;
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) {
            if (j >= mr) break;
            const int32_t at = tid + j * kGradThreads, row = at / (8 * mr), r = (at - row * 8 * mr) * 2;
            float* f = reinterpret_cast<float*>(ws) + row * wf + r;
            f[0] = wreg[j].x;
            f[1] = wreg[j].y;
        }
    };

    // the slots are asked for four stages ahead of the rows they name
    constexpr int AHEAD = 4;
    if (tid < AHEAD * kGradSlots && tid < ck.n) ring[tid / kGradSlots][tid % kGradSlots] = __ldg(perm + tid);
    auto slot_of = [&](int32_t i) { return tid < kGradSlots && i * kGradSlots + tid < ck.n ? __ldg(perm + i * kGradSlots + tid) : 0; };
    int32_t next = slot_of(AHEAD);
    __syncthreads();
    float acc[MR][NJ][4] = {};
#pragma unroll
    for (int i = 0; i < kGradStages - 1; ++i) {
        if (i < steps) load_z(i);
        copies_commit();
    }
    load_w(0);
    store_w(0);
    if (steps > 1) load_w(1);
    for (int32_t i = 0; i < steps; ++i) {
        copies_wait<kGradStages - 2>();
        __syncthreads();
        if (i + kGradStages - 1 < steps) load_z(i + kGradStages - 1);
        copies_commit();
        if (tid < kGradSlots) ring[(i + AHEAD) % kGradRing][tid] = next;
        next = slot_of(i + AHEAD + 1);
        if (i + 1 < steps) store_w(i + 1);      // the buffer that the step before last read
        if (i + 2 < steps) load_w(i + 2);
        const T* zs = zs_all + i % kGradStages * kGradSlots * ZP;
        const uint8_t* ws = ws_all + i % 2 * w_bytes;
        uint32_t b[kGradSlots / 16][NJ][2];
#pragma unroll
        for (int k = 0; k < kGradSlots / 16; ++k)
#pragma unroll
            for (int j = 0; j < NJ; j += 2) {
                uint32_t x[4];
                ldsm4(x, zs + (k * 16 + lane % 16) * ZP + warp * 8 * NJ + (j + lane / 16) * 8, true);
                b[k][j][0] = x[0];
                b[k][j][1] = x[1];
                b[k][j + 1][0] = x[2];
                b[k][j + 1][1] = x[3];
            }
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            if (m >= mr) break;
            float sum[NJ][4] = {};      // of the stage: a chain of few additions that cut off (lora_down.cu)
#pragma unroll
            for (int k = 0; k < kGradSlots / 16; ++k) {
                const float* f = reinterpret_cast<const float*>(ws) + (k * 16 + lane % 4 * 2) * wf + m * 16 + lane / 4;
                float v[8];      // ranks by h, slots 2 q (+1) and 2 q + 8 (+1)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        v[2 * (h + 2 * x)] = f[8 * x * wf + 8 * h];
                        v[2 * (h + 2 * x) + 1] = f[(8 * x + 1) * wf + 8 * h];
                    }
                Wide16<T> wide;
                wide.set(v);
                wide.mul(sum, b[k]);
            }
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int x = 0; x < 4; ++x) acc[m][j][x] += sum[j][x];
        }
    }
    copies_wait<0>();
    const int64_t size = static_cast<int64_t>(R) * cols;
    float* out = ck.alone ? job.out + ck.adapter * size : job.parts + blockIdx.x * size;
#pragma unroll
    for (int m = 0; m < MR; ++m) {
        if (m >= mr) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int32_t r = m * 16 + lane / 4 + 8 * h;
            if (r >= R) continue;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int32_t c = col0 + warp * 8 * NJ + j * 8 + lane % 4 * 2;
                if (c >= cols) continue;
                if (job.turned) {
                    out[static_cast<int64_t>(c) * R + r] = acc[m][j][2 * h];
                    out[static_cast<int64_t>(c + 1) * R + r] = acc[m][j][2 * h + 1];
                } else {
                    *reinterpret_cast<float2*>(out + static_cast<int64_t>(r) * cols + c) = make_float2(acc[m][j][2 * h], acc[m][j][2 * h + 1]);
                }
            }
        }
    }
    wait_for_prior_grid();
}

// Adds up the chunks of adapters that have several, and zeroes those that have none.
struct JoinArgs {
    float* out[2];
    const float* parts[2];
    int64_t size4[2];      // in words of 16 bytes
    const int32_t* offsets;
    int32_t per;
};

__global__ void __launch_bounds__(kGradThreads) lora_join_kernel(const JoinArgs a) {
    const int32_t e = static_cast<int32_t>(blockIdx.x);
    const int32_t o0 = __ldg(a.offsets + e), n = __ldg(a.offsets + e + 1) - o0;
    if (n > 0 && n <= a.per) return;
    const int32_t chunks = n / a.per + (n % a.per != 0);
    const int64_t first = o0 / a.per + e;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (!a.out[j]) continue;
        const int64_t size = a.size4[j];
        const float4* parts = reinterpret_cast<const float4*>(a.parts[j]) + first * size;
        float4* out = reinterpret_cast<float4*>(a.out[j]) + e * size;
        for (int64_t i = static_cast<int64_t>(blockIdx.y) * kGradThreads + threadIdx.x; i < size; i += static_cast<int64_t>(gridDim.y) * kGradThreads) {
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
            for (int32_t c = 0; c < chunks; ++c) {
                const float4 x = __ldg(parts + c * size + i);
                v.x += x.x;
                v.y += x.y;
                v.z += x.z;
                v.w += x.w;
            }
            out[i] = v;
        }
    }
}

int launch_grad_fp16(const LoraGrad* jobs, const LoraPlan& p, cudaStream_t s) {
    const int32_t cc = p.rank <= 64 ? 256 : 128, r16 = (p.rank + 15) / 16 * 16;
    int64_t blocks;
    const GradArgs<__half> a = grad_args<__half>(jobs, p, cc, &blocks);
    const dim3 grid(static_cast<unsigned>(lora_chunks(p.n_slots, p.n_adapters, p.chunk)), static_cast<unsigned>(blocks)), block(kGradThreads);
    const size_t sm = kGradStages * kGradSlots * static_cast<size_t>(cc + 8) * 2 + 2 * static_cast<size_t>(kGradSlots * (r16 + 4) * 4);
    auto go = [&](auto k) { return launch_with(k, "lora_grad_kernel", grid, block, sm, p.overlap_grad, 1, s, a); };
    if (p.rank <= 16) return go(lora_grad_kernel<1, 4>);
    if (p.rank <= 32) return go(lora_grad_kernel<2, 4>);
    if (p.rank <= 64) return go(lora_grad_kernel<4, 4>);
    return go(lora_grad_kernel<8, 2>);
}

}  // namespace

int launch_lora_grad(const LoraGrad* jobs, const LoraPlan& p, int dtype, cudaStream_t s) {
    JoinArgs j{};
    for (int i = 0; i < 2; ++i) {
        j.out[i] = jobs[i].out;
        j.parts[i] = jobs[i].parts;
        j.size4[i] = jobs[i].out ? static_cast<int64_t>(p.rank) * jobs[i].cols / 4 : 0;
    }
    if (!j.out[0] && !j.out[1]) return FT_OK;
    if (int st = dtype == FT_DTYPE_F16 ? launch_grad_fp16(jobs, p, s) : launch_lora_grad_tc(jobs, p, s)) return st;
    j.offsets = p.offsets;
    j.per = p.chunk;
    int64_t y = 4 * static_cast<int64_t>(sm_count()) / p.n_adapters;
    const int64_t most = (std::max(j.size4[0], j.size4[1]) + kGradThreads - 1) / kGradThreads;
    y = y < 1 ? 1 : y < most ? y : most;
    const dim3 jgrid(static_cast<unsigned>(p.n_adapters), static_cast<unsigned>(y)), block(kGradThreads);
    lora_join_kernel<<<jgrid, block, 0, s>>>(j);
    return check_launch("lora_join_kernel", jgrid, block, 0);
}

}  // namespace ft
