// Second product of a low-rank adapter: out[s] = add[s] + scale W u[s], for slots s that share an adapter.
//
//   forward   u = A x,          W = B [N][R]                out = add + scale B A x
//   backward  u = B^T dy,       W = A^T of A [R][K]         the gradient of x, per slot
//
// Memory-bound on out and add.  A CTA takes a tile of 64 slots (16 where adapters have few) and a run of
// columns; u stays in registers as a matrix operand of 16 or 24 significant bits (lora.cuh), W passes through a ring of
// three stages in shared memory, its columns placed so that a thread's eight results are neighbours: add is read
// and out written by whole 16-byte words.  add's words are asked for before W's stage is waited for.
//
// Rows without an adapter are copied (or zeroed) by CTAs of their own, or, where CTAs find their tiles among
// the ids, by the slot's own CTA.
#pragma once

#include "lora.cuh"
#include "ft_internal.h"
#include "launch.cuh"

namespace ft {

constexpr int kUpStages = 3;

template <typename T>
struct UpArgs {
    LoraSlots slots;
    const float *u, *scales;
    const T* w;
    const void* add;
    void* out;
    float* present;      // instead of copying rows without an adapter: 1 or 0 per slot
    int32_t rank, cols, per, n_tiles;
    bool trans;          // W's values of one rank are neighbours ([R][cols])
};

template <typename T>
__device__ __forceinline__ void up_store8(T* p, const float (&v)[8]) {
    __align__(16) T o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = from_f32<T>(v[i]);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(o) / 16); ++i) reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(o)[i];
}

// out := add or 0, columns [c0, c1) of a slot without an adapter.
template <typename T, typename YT>
__device__ void up_pass(const UpArgs<T>& a, int64_t slot, int32_t c0, int32_t c1) {
    if (a.add == a.out) return;
    constexpr int V = 16 / static_cast<int>(sizeof(YT));
    for (int32_t c = c0 + static_cast<int32_t>(threadIdx.x) * V; c < c1; c += kLoraThreads * V) {
        const int64_t at = slot * a.cols + c;
        const uint4 v = a.add ? __ldg(reinterpret_cast<const uint4*>(static_cast<const YT*>(a.add) + at)) : make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(static_cast<YT*>(a.out) + at) = v;
    }
}

// KS: steps of 16 ranks that there is room for.
template <typename T, typename YT, int MT, int KS>
__global__ void __launch_bounds__(kLoraThreads) lora_up_kernel(const __grid_constant__ UpArgs<T> a) {
    constexpr int CW = MT == kLoraTile ? 64 : 128;      // columns of a stage
    constexpr int GROUPS = MT == kLoraTile ? 2 : 1;     // of 32 columns, that a warp has of a stage
    constexpr int TERMS = sizeof(YT) == 4 ? 3 : 2;      // 2^-17 of u's product is far below a 16-bit result's rounding
    constexpr int WORDS = static_cast<int>(sizeof(YT)) * 8 / 16;
    extern __shared__ __align__(16) uint8_t up_smem[];
    __shared__ int32_t slots[kLoraThreads];
    const int32_t tid = static_cast<int32_t>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    const int32_t R = a.rank, ks = (R + 15) / 16, cols = a.cols;
    const int32_t c0 = static_cast<int32_t>(blockIdx.y) * a.per, c1 = min(cols, c0 + a.per);
    if (static_cast<int32_t>(blockIdx.x) >= a.n_tiles) {
        __shared__ int32_t n_none;
        const int32_t s = (static_cast<int32_t>(blockIdx.x) - a.n_tiles) * kLoraThreads + tid;
        if (tid == 0) n_none = 0;
        __syncthreads();
        const int32_t id = s < a.slots.n_slots ? __ldg(a.slots.ids + s) : 0;
        const bool none = id < 0 || id >= a.slots.n_adapters;
        if (a.present) {
            if (blockIdx.y == 0 && s < a.slots.n_slots) a.present[s] = none ? 0.0f : 1.0f;
            return;
        }
        if (none) slots[atomicAdd(&n_none, 1)] = s;      // rows of their own: the order does not show
        __syncthreads();
        for (int32_t i = 0; i < n_none; ++i) up_pass<T, YT>(a, slots[i], c0, c1);
        return;
    }
    const LoraTile tile = find_tile<MT>(a.slots, static_cast<int32_t>(blockIdx.x), slots, kLoraThreads);
    if (tile.n == 0) {
        if (tile.adapter < 0) up_pass<T, YT>(a, tile.first, c0, c1);
        return;
    }
    const int32_t pitch = a.trans ? CW + 8 : odd_pitch(16 * ks), stage_elems = a.trans ? 16 * ks * (CW + 8) : CW * pitch;
    T* smem = reinterpret_cast<T*>(up_smem);
    const T* w = a.w + static_cast<int64_t>(tile.adapter) * R * cols;
    auto load = [&](int32_t i) {
        const int32_t col = c0 + i * CW;
        T* ws = smem + i % kUpStages * stage_elems;
        if (a.trans) {
            // pairs of columns to their places
            for (int32_t at = tid; at < 16 * ks * (CW / 2); at += kLoraThreads) {
                const int32_t r = at / (CW / 2), c = at % (CW / 2) * 2;
                const bool there = r < R && col + c < c1;
                copy4(ws + r * pitch + spread_col(c), there ? w + static_cast<int64_t>(r) * cols + col + c : w, there);
            }
        } else {
#pragma unroll
            for (int h = 0; h < CW / 64; ++h) {
                const int32_t c = tid / 2 + 64 * h;
                for (int32_t ch = tid % 2; ch < 2 * ks; ch += 2) {
                    const bool there = ch * 8 < R && col + c < c1;
                    copy16(ws + spread_col(c) * pitch + ch * 8, there ? w + static_cast<int64_t>(col + c) * R + ch * 8 : w, there);
                }
            }
        }
    };
    const int32_t steps = (c1 - c0 + CW - 1) / CW;
#pragma unroll
    for (int i = 0; i < kUpStages - 1; ++i) {
        if (i < steps) load(i);
        copies_commit();
    }
    // this thread's two rows
    const int32_t row0 = MT == kLoraTile ? warp * 16 : 0, group0 = MT == kLoraTile ? 0 : warp;
    const bool busy = row0 < tile.n;
    int64_t at[2];
    bool mine[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int32_t row = row0 + lane / 4 + 8 * h;
        mine[h] = row < tile.n;
        at[h] = slots[mine[h] ? row : 0];
    }
    wait_for_prior_grid();
    Wide16<T, TERMS> u[KS];
    const float scale = a.scales ? __ldg(a.scales + tile.adapter) : 1.0f;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
        float v[8];      // rows by h, ranks 2 q (+1) and 2 q + 8 (+1): mma's registers 0, 2 and 1, 3
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int32_t r = k * 16 + lane % 4 * 2 + 8 * i;
                const float2 x = mine[h] && r < R ? *reinterpret_cast<const float2*>(a.u + at[h] * R + r) : make_float2(0.0f, 0.0f);
                v[2 * (h + 2 * i)] = scale * x.x;
                v[2 * (h + 2 * i) + 1] = scale * x.y;
            }
        u[k].set(v);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) at[h] = at[h] * cols + lane % 4 * 8;
    const YT* add = static_cast<const YT*>(a.add);
    YT* out = static_cast<YT*>(a.out);
    for (int32_t i = 0; i < steps; ++i) {
        const int32_t col = c0 + i * CW + group0 * 32;
        uint4 sum[GROUPS][2][WORDS];
        if (add) {
#pragma unroll
            for (int g = 0; g < GROUPS; ++g)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int x = 0; x < WORDS; ++x)
                        sum[g][h][x] = mine[h] && col + g * 32 + lane % 4 * 8 < c1
                                           ? *(reinterpret_cast<const uint4*>(add + at[h] + col + g * 32) + x) : make_uint4(0u, 0u, 0u, 0u);
        }
        copies_wait<kUpStages - 2>();
        __syncthreads();
        if (i + kUpStages - 1 < steps) load(i + kUpStages - 1);
        copies_commit();
        if (!busy) continue;
        const T* ws = smem + i % kUpStages * stage_elems;
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            const int32_t first = (group0 + g) * 32;
            float acc[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int x = 0; x < 4; ++x) acc[j][x] = 0.0f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                if (k >= ks) break;
                uint32_t b[4][2];
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    const int32_t n = first + (j + lane / 16) * 8, r = k * 16 + lane / 8 % 2 * 8;
                    uint32_t x[4];
                    if (a.trans) ldsm4(x, ws + (r + lane % 8) * pitch + n, true);
                    else ldsm4(x, ws + (n + lane % 8) * pitch + r, false);
                    b[j][0] = x[0];
                    b[j][1] = x[1];
                    b[j + 1][0] = x[2];
                    b[j + 1][1] = x[3];
                }
                u[k].mul(acc, b);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (!mine[h] || col + g * 32 + lane % 4 * 8 >= c1) continue;
                float v[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[2 * j] = acc[j][2 * h];
                    v[2 * j + 1] = acc[j][2 * h + 1];
                }
                if (add) {
                    const YT* e = reinterpret_cast<const YT*>(&sum[g][h][0]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] += to_f32<YT>(e[j]);
                }
                up_store8<YT>(out + at[h] + col + g * 32, v);
            }
        }
    }
    copies_wait<0>();
}

template <typename T, typename YT, int MT>
int launch_up_typed(UpArgs<T> a, bool fill, cudaStream_t s) {
    constexpr int CW = MT == kLoraTile ? 64 : 128;
    const int64_t blocks = (a.cols + CW - 1) / CW, most = 6 * static_cast<int64_t>(sm_count());
    int64_t parts = most / (a.n_tiles > 0 ? a.n_tiles : 1);      // runs of columns: as many CTAs as fill the GPU a few times
    parts = parts < 1 ? 1 : parts < blocks ? parts : blocks;
    a.per = static_cast<int32_t>((blocks + parts - 1) / parts * CW);
    parts = (a.cols + a.per - 1) / a.per;
    const int64_t fills = fill ? (static_cast<int64_t>(a.slots.n_slots) + kLoraThreads - 1) / kLoraThreads : 0;
    const dim3 grid(static_cast<unsigned>(a.n_tiles + fills), static_cast<unsigned>(parts)), block(kLoraThreads);
    const int32_t r16 = (a.rank + 15) / 16 * 16;
    const size_t sm = kUpStages * sizeof(T) * static_cast<size_t>(a.trans ? r16 * (CW + 8) : CW * odd_pitch(r16));
    auto go = [&](auto k) { return launch_with(k, "lora_up_kernel", grid, block, sm, true, 1, s, a); };
    if (a.rank <= 16) return go(lora_up_kernel<T, YT, MT, 1>);
    if (a.rank <= 32) return go(lora_up_kernel<T, YT, MT, 2>);
    if (a.rank <= 64) return go(lora_up_kernel<T, YT, MT, 4>);
    return go(lora_up_kernel<T, YT, MT, 8>);
}

template <typename T>
int launch_up(const LoraUp& j, const LoraPlan& p, cudaStream_t s) {
    UpArgs<T> a{};
    a.slots = LoraSlots{p.ids, p.offsets, p.tiles, p.perm, p.n_slots, p.n_adapters};
    a.u = j.u;
    a.scales = p.scales;
    a.w = static_cast<const T*>(j.w);
    a.add = j.add;
    a.out = j.out;
    a.present = j.present;
    a.rank = p.rank;
    a.cols = j.cols;
    a.n_tiles = static_cast<int32_t>(p.n_tiles);
    a.trans = j.trans;
    const bool fill = p.perm != nullptr;
    if (j.out_f32)
        return p.width == kLoraTile ? launch_up_typed<T, float, kLoraTile>(a, fill, s) : launch_up_typed<T, float, kLoraSmallTile>(a, fill, s);
    return p.width == kLoraTile ? launch_up_typed<T, T, kLoraTile>(a, fill, s) : launch_up_typed<T, T, kLoraSmallTile>(a, fill, s);
}

}  // namespace ft
