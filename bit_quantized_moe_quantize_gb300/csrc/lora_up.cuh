// Second product of a low-rank adapter: out[s] = add[s] + scale W u[s], for slots s that share an adapter.
//
//   forward   u = A x,          W = B [N][R]                out = add + scale B A x
//   backward  u = B^T dy,       W = A^T of A [R][K]         the gradient of x, per slot
//
// Memory-bound on out and add.  A CTA takes 64 slots (16 where adapters have few) and a run of
// columns; u stays in registers as a matrix operand that keeps its 24 bits (lora.cuh).  W and add pass through a
// ring of stages in shared memory, add's words at the place of the thread that wants them.  A thread's results are made
// eight neighbours, by where W's columns are put or by an exchange between four lanes, and written as whole 16-byte words.
//
// Rows without an adapter are copied (or zeroed) by CTAs of their own.
//
// 8191 slots of 4096 bf16, rank 16, add: 27 us, 134 MB at 4.9 TB/s; 16384 of 1536 fp32, rank 8: 39 us, 201 MB at
// 5.2; 8192 of 4096, rank 64, W turned, no add: 42.5 us, whose MMAs (three for a product, 47 % of the tensor cores' cycles) and
// the matrices' way to the registers bound it.  (With two parts of u, 16 bits, the first and last took 26 and 35 us.)
//
// All ranks and parts of a result, 24 MMAs at rank 128, go through one accumulator, which cuts off what it adds (lora_down.cu): some
// 24 2^-25 of the sum, too short a chain for sums that start anew.
#pragma once

#include <type_traits>

#include "lora.cuh"
#include "ft_internal.h"
#include "launch.cuh"

namespace ft {

// Stages: what two or more CTAs of an SM have room for.
template <typename YT>
__host__ __device__ constexpr int up_stages() { return sizeof(YT) == 4 ? 3 : 4; }
constexpr int kUpFill = 64;      // slots that a CTA looks through for such without an adapter

template <typename T>
struct UpArgs {
    LoraSlots slots;
    const float *u, *scales;
    const T* w;
    const void* add;
    void* out;
    float* present;      // instead of copying rows without an adapter: 1 or 0 per slot
    int32_t rank, cols, per, fills;
    bool trans;          // W's values of one rank are neighbours ([R][cols])
};

// Columns 8 j + 2 q + {0, 1} of lane q (of four neighbours) -> columns 8 q + 2 i + {0, 1}: a 4 x 4 transpose of pairs.
__device__ __forceinline__ void turn_pairs(float (&v)[8], int32_t lane) {
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int lo = o == 1 ? 2 * m : m, hi = lo + o;      // pairs that this step exchanges
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float got = __shfl_xor_sync(0xFFFFFFFFu, up ? v[2 * lo + i] : v[2 * hi + i], o);
                v[2 * lo + i] = up ? got : v[2 * lo + i];
                v[2 * hi + i] = up ? v[2 * hi + i] : got;
            }
        }
    }
}

// out := add or 0, columns [c0, c1) of n slots without an adapter, by the whole CTA.
template <typename YT, int THREADS>
__device__ __forceinline__ void up_pass(const void* add, void* out, int32_t cols, const int32_t* slots, int32_t n, int32_t c0, int32_t c1) {
    if (add == out) return;
    constexpr int V = 16 / static_cast<int>(sizeof(YT));
    const uint32_t words = static_cast<uint32_t>(c1 - c0) / V;
#pragma unroll 8
    for (uint32_t i = threadIdx.x; i < n * words; i += THREADS) {
        const uint32_t row = i / words;
        const int64_t at = static_cast<int64_t>(slots[row]) * cols + c0 + (i - row * words) * V;
        const uint4 v = add ? __ldg(reinterpret_cast<const uint4*>(static_cast<const YT*>(add) + at)) : make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(static_cast<YT*>(out) + at) = v;
    }
}

// KS: steps of 16 ranks that there is room for.
template <typename T, typename YT, int MT, int KS>
__global__ void __launch_bounds__(kLoraThreads) lora_up_kernel(const __grid_constant__ UpArgs<T> a) {
    constexpr bool SMALL = MT == kLoraSmallTile;
    constexpr bool FP32 = sizeof(YT) == 4;
    constexpr int STAGES = up_stages<YT>();
    constexpr int THREADS = kLoraThreads;
    constexpr int CW = SMALL ? 128 : 64;                // columns of a stage
    constexpr int GROUPS = SMALL ? 1 : 2;               // of 32 columns, that a warp has of a stage
    constexpr int WORDS = static_cast<int>(sizeof(YT)) * 8 / 16, ADDS = GROUPS * 2 * WORDS;      // 16-byte words of eight results; of a stage's
    extern __shared__ __align__(16) uint8_t up_smem[];
    __shared__ int32_t slots[MT > kUpFill ? MT : kUpFill];
    const int32_t tid = static_cast<int32_t>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    const int32_t R = a.rank, ks = (R + 15) / 16, cols = a.cols;
    const int32_t c0 = static_cast<int32_t>(blockIdx.y) * a.per, c1 = min(cols, c0 + a.per);
    if (static_cast<int32_t>(blockIdx.x) < a.fills) {
        __shared__ int32_t n_none;
        const int32_t s = static_cast<int32_t>(blockIdx.x) * kUpFill + tid;
        const bool there = tid < kUpFill && s < a.slots.n_slots;
        const int32_t id = there ? __ldg(a.slots.ids + s) : 0;
        const bool none = id < 0 || id >= a.slots.n_adapters;
        if (a.present) {
            if (blockIdx.y == 0 && there) a.present[s] = none ? 0.0f : 1.0f;
        } else {
            if (tid == 0) n_none = 0;
            __syncthreads();
            if (none) slots[atomicAdd(&n_none, 1)] = s;      // rows of their own: the order does not show
            __syncthreads();
            up_pass<YT, THREADS>(a.add, a.out, cols, slots, n_none, c0, c1);
        }
        // What starts behind this grid, early or not, takes the first products and the order for made (lora_grad.cuh).  CTAs with a tile wait
        // for them before they let it start, others end without; where no slot has an adapter this one alone waits.
        if (blockIdx.x == 0 && blockIdx.y == 0) wait_for_prior_grid();
        return;
    }
    const LoraTile tile = find_tile<MT>(a.slots, static_cast<int32_t>(blockIdx.x) - a.fills, slots);
    if (tile.n == 0) return;
    T* smem = reinterpret_cast<T*>(up_smem);
    const T* w = a.w + static_cast<int64_t>(tile.adapter) * R * cols;
    // this thread's two rows, and the first column of its words of a group's 32
    const int32_t row0 = SMALL ? 0 : warp * 16, group0 = SMALL ? warp : 0, mycol = lane % 4 * (FP32 ? 4 : 8);
    const bool busy = row0 < tile.n;
    int64_t at[2];
    bool mine[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int32_t row = row0 + lane / 4 + 8 * h;
        mine[h] = row < tile.n;
        at[h] = slots[mine[h] ? row : 0];
    }
    const int64_t uat[2] = {at[0] * R, at[1] * R};
#pragma unroll
    for (int h = 0; h < 2; ++h) at[h] = at[h] * cols + mycol;
    const YT* add = static_cast<const YT*>(a.add);
    YT* out = static_cast<YT*>(a.out);
    const int32_t steps = (c1 - c0 + CW - 1) / CW;

    auto product = [&](auto turned) {
        constexpr bool TRANS = decltype(turned)::value;
        const int32_t pitch = TRANS ? CW + 8 : odd_pitch(16 * ks), w_elems = TRANS ? 16 * ks * (CW + 8) : CW * pitch;
        const int32_t stage_elems = w_elems + (add ? ADDS * THREADS * 16 / static_cast<int>(sizeof(T)) : 0);
        auto load = [&](int32_t i) {
            const int32_t col = c0 + i * CW;
            T* ws = smem + i % STAGES * stage_elems;
            if constexpr (TRANS) {
                constexpr int WORDS = CW / 8;
#pragma unroll
                for (int j = 0; j < (16 * KS * WORDS + THREADS - 1) / THREADS; ++j) {
                    const int32_t x = tid + j * THREADS, r = x / WORDS, c = x % WORDS * 8;
                    const bool there = r < R && col + c < c1;
                    if (r < 16 * ks) copy16(ws + r * pitch + c, there ? w + static_cast<int64_t>(r) * cols + col + c : w, there);
                }
            } else {
                constexpr int SHARE = SMALL ? 2 : THREADS / CW;      // threads of a column
#pragma unroll
                for (int h = 0; h < (SMALL ? 2 : 1); ++h) {
                    const int32_t c = tid / SHARE + 64 * h;
                    const bool in = col + c < c1;
                    const T* src = w + static_cast<int64_t>(in ? col + c : 0) * R;
                    T* dst = ws + spread_col<FP32>(c) * pitch;
                    for (int32_t ch = tid % SHARE; ch < 2 * ks; ch += SHARE) {
                        const bool there = in && ch * 8 < R;
                        copy16(dst + ch * 8, there ? src + ch * 8 : w, there);
                    }
                }
            }
            if (add) {      // every thread's own words
                uint8_t* as = reinterpret_cast<uint8_t*>(ws + w_elems) + tid * 16;
#pragma unroll
                for (int g = 0; g < GROUPS; ++g)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int x = 0; x < WORDS; ++x) {
                            const int32_t c = col + (group0 + g) * 32 + x * 16;
                            const bool there = mine[h] && c + mycol < c1;
                            copy16(as + ((g * 2 + h) * WORDS + x) * THREADS * 16, there ? add + at[h] + c : add, there);
                        }
            }
        };
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) {
            if (i < steps) load(i);
            copies_commit();
        }
        wait_for_prior_grid();
        let_next_grid_start();      // behind the wait: the matrices' gradients come up early and read the first products
        Wide16<T> u[KS];
        const float scale = a.scales ? __ldg(a.scales + tile.adapter) : 1.0f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            float v[8];      // rows by h, ranks 2 q (+1) and 2 q + 8 (+1): mma's registers 0, 2 and 1, 3
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int32_t r = k * 16 + lane % 4 * 2 + 8 * i;
                    const float2 x = mine[h] && r < R ? *reinterpret_cast<const float2*>(a.u + uat[h] + r) : make_float2(0.0f, 0.0f);
                    v[2 * (h + 2 * i)] = scale * x.x;
                    v[2 * (h + 2 * i) + 1] = scale * x.y;
                }
            u[k].set(v);
        }
        // what this lane gives the address of: pairs of eight columns by 16 ranks
        int32_t wat[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int32_t n = group0 * 32 + (2 * j + lane / 16) * 8, r = lane / 8 % 2 * 8, l = lane % 8;
            wat[j] = TRANS ? (r + l) * pitch + n : (n + l) * pitch + r;
        }
        const int32_t kstep = TRANS ? 16 * pitch : 16, gstep = TRANS ? 32 : 32 * pitch;
        for (int32_t i = 0; i < steps; ++i) {
            copies_wait<STAGES - 2>();
            __syncthreads();
            if (i + STAGES - 1 < steps) load(i + STAGES - 1);
            copies_commit();
            if (!busy) continue;
            const int32_t col = c0 + i * CW + group0 * 32;
            const T* ws = smem + i % STAGES * stage_elems;
            const uint8_t* as = reinterpret_cast<const uint8_t*>(ws + w_elems) + tid * 16;
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                float acc[4][4] = {};
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    if (k >= ks) break;
                    uint32_t b[4][2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t x[4];
                        ldsm4(x, ws + wat[j] + k * kstep + g * gstep, TRANS);
                        b[2 * j][0] = x[0];
                        b[2 * j][1] = x[1];
                        b[2 * j + 1][0] = x[2];
                        b[2 * j + 1][1] = x[3];
                    }
                    u[k].mul(acc, b);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[2 * j] = acc[j][2 * h];
                        v[2 * j + 1] = acc[j][2 * h + 1];
                    }
                    if constexpr (TRANS && FP32) {      // rows of the workspace: pairs of columns, whole sectors for four lanes
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (mine[h] && col + g * 32 + j * 8 + lane % 4 * 2 < c1)
                                *reinterpret_cast<float2*>(out + at[h] - mycol + lane % 4 * 2 + col + g * 32 + j * 8) = make_float2(v[2 * j], v[2 * j + 1]);
                        continue;
                    }
                    if constexpr (TRANS) turn_pairs(v, lane);
                    constexpr int PER = 8 / WORDS;      // results of a word
#pragma unroll
                    for (int x = 0; x < WORDS; ++x) {
                        if (!mine[h] || col + g * 32 + x * 16 + mycol >= c1) continue;
                        __align__(16) YT o[PER];
                        if (add) *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(as + ((g * 2 + h) * WORDS + x) * THREADS * 16);
#pragma unroll
                        for (int j = 0; j < PER; ++j) o[j] = from_f32<YT>(add ? v[x * PER + j] + to_f32<YT>(o[j]) : v[x * PER + j]);
                        *reinterpret_cast<uint4*>(out + at[h] + col + g * 32 + x * 16) = *reinterpret_cast<const uint4*>(o);
                    }
                }
            }
        }
        copies_wait<0>();
    };
    if (a.trans) product(std::true_type());
    else product(std::false_type());
}

template <typename T, typename YT, int MT>
int launch_up_typed(UpArgs<T> a, const LoraPlan& p, cudaStream_t s) {
    constexpr int CW = MT == kLoraSmallTile ? 128 : 64;
    const int64_t blocks = (a.cols + CW - 1) / CW, tiles = p.n_tiles * (p.width / MT);
    // Runs of columns: CTAs enough to fill the GPU some times over, each of six stages or more (calls of 8191 slots, bf16, and 16384,
    // fp32, from a graph: 58 and 65 us; with half as many CTAs 60 and 69, twice 58 and 65; runs of three stages 58 and 67, of twelve 60 and 71).
    const int64_t some = p.n_slots / MT + 1;      // tiles that there are, about
    int64_t parts = 12 * static_cast<int64_t>(sm_count()) / some, most = (blocks + 5) / 6;
    if (tiles * blocks < 8 * static_cast<int64_t>(sm_count())) most = blocks;
    parts = parts < 1 ? 1 : parts < most ? parts : most;
    a.per = static_cast<int32_t>((blocks + parts - 1) / parts * CW);
    parts = (a.cols + a.per - 1) / a.per;
    a.fills = static_cast<int32_t>((static_cast<int64_t>(p.n_slots) + kUpFill - 1) / kUpFill);
    const dim3 grid(static_cast<unsigned>(tiles + a.fills), static_cast<unsigned>(parts)), block(kLoraThreads);
    const int32_t r16 = (a.rank + 15) / 16 * 16;
    const size_t adds = a.add ? static_cast<size_t>(kLoraThreads) * (MT == kLoraSmallTile ? 1 : 2) * 2 * sizeof(YT) * 8 : 0;
    const size_t sm = up_stages<YT>() * (sizeof(T) * static_cast<size_t>(a.trans ? r16 * (CW + 8) : CW * odd_pitch(r16)) + adds);
    auto go = [&](auto k) { return launch_with(k, "lora_up_kernel", grid, block, sm, true, 1, s, a); };
    if (a.rank <= 16) return go(lora_up_kernel<T, YT, MT, 1>);
    if (a.rank <= 32) return go(lora_up_kernel<T, YT, MT, 2>);
    if (a.rank <= 64) return go(lora_up_kernel<T, YT, MT, 4>);
    return go(lora_up_kernel<T, YT, MT, 8>);
}

template <typename T>
int launch_up(const LoraUp& j, const LoraPlan& p, cudaStream_t s) {
    UpArgs<T> a{};
    a.slots = LoraSlots{p.ids, p.offsets, p.tiles, p.perm, p.n_slots, p.n_adapters, p.width};
    a.u = j.u;
    a.scales = p.scales;
    a.w = static_cast<const T*>(j.w);
    a.add = j.add;
    a.out = j.out;
    a.present = j.present;
    a.rank = p.rank;
    a.cols = j.cols;
    a.trans = j.trans;
    if (j.out_f32)
        return p.width == kLoraSmallTile ? launch_up_typed<T, float, kLoraSmallTile>(a, p, s) : launch_up_typed<T, float, 64>(a, p, s);
    return p.width == kLoraSmallTile ? launch_up_typed<T, T, kLoraSmallTile>(a, p, s) : launch_up_typed<T, T, 64>(a, p, s);
}

}  // namespace ft
