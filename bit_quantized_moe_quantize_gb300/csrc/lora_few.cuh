// Low-rank adapters of few slots, in one launch and without a workspace: out[s] = add[s] + scale B (A x).
//
// Bound by latency.  A cluster of up to eight CTAs takes up to 16 slots that share an adapter, which it finds among the
// ids.  Its CTAs share the columns of x and A, add their sums up through each other's shared memory, in a fixed
// order, so that each has the whole of u = A x, and then share the rows of B.  The first of B's stages are on their way
// while A x is summed.  In the first product the four warps share a stage's values, in the second its columns;
// lora_down.cu and lora_up.cuh have the same steps for many slots, where a launch of its own for each is no loss.
//
// 1 slot of 2048 x 2048, rank 16: 7.8 us (the three launches: 19 from a graph against 11); 64 slots of as many adapters,
// 4096 x 4096: 11.2 us, 17 MB of adapters at 1.5 TB/s: ids, then A and x, two meetings of the cluster, and B's first words behind A's last,
// each a wait of its own.
#pragma once

#include "lora_up.cuh"

namespace ft {

constexpr int kFewSlots = 16, kFewStages = 4, kFewDownCols = 64, kFewUpCols = 128;
__host__ __device__ constexpr int few_up_stages(int nt) { return nt > 8 ? 2 : 3; }

template <typename T>
struct FewArgs {
    LoraSlots slots;
    const T *x, *a, *b;
    const float* scales;
    const void* add;
    void* out;
    uint32_t* err;
    int32_t rank, ncols, nrows, div, per;      // per: rows of B that a CTA takes
};

// NT: tiles of eight ranks that there is room for.
template <typename T, typename YT, int NT>
__global__ void __launch_bounds__(kLoraThreads) lora_few_kernel(const __grid_constant__ FewArgs<T> a) {
    constexpr int THREADS = kLoraThreads, WARPS = THREADS / 32, KS = NT / 2, UPS = few_up_stages(NT);
    constexpr bool FP32 = sizeof(YT) == 4;
    constexpr int WORDS = static_cast<int>(sizeof(YT)) * 8 / 16;
    extern __shared__ __align__(128) uint8_t few_smem[];
    __shared__ int32_t slots[kFewSlots];
    const uint32_t size = cluster_size(), rank = cluster_rank();
    const int32_t tid = static_cast<int32_t>(threadIdx.x), warp = tid >> 5, lane = tid & 31, l = lane % 8;
    const int32_t s0 = static_cast<int32_t>(blockIdx.x / size), R = a.rank, nt = R / 8, ks = (R + 15) / 16, K = a.ncols, N = a.nrows;
    const int32_t c0 = static_cast<int32_t>(rank) * a.per, c1 = min(N, c0 + a.per);
    const LoraTile tile = find_tile<kFewSlots>(a.slots, s0, slots);
    if (tile.n == 0) {      // all of the cluster
        if (tile.adapter < 0) {
            const int32_t id = __ldg(a.slots.ids + s0);
            if (tid == 0) {
                slots[0] = s0;
                if (rank == 0 && id != -1) atomicOr(a.err, FT_DEVERR_BAD_EXPERT_ID);
            }
            __syncthreads();
            if (c0 < c1) up_pass<YT, THREADS>(a.add, a.out, N, slots, 1, c0, c1);
        }
        return;
    }
    const int32_t down_elems = (kFewSlots + R) * kFewDownCols, pitch = odd_pitch(16 * ks);
    T* down = reinterpret_cast<T*>(few_smem);                                              // [stages][16 + R][64]
    float* sums = reinterpret_cast<float*>(down);                                          // [warps][16][R], after the first product
    float* mine = reinterpret_cast<float*>(down + kFewStages * down_elems);                // [16][R]
    float* u_all = mine + kFewSlots * R;                                                   // [16][R]
    T* up = reinterpret_cast<T*>(u_all + kFewSlots * R);                                   // [stages][128][pitch], add's words
    const int32_t w_elems = kFewUpCols * pitch, up_elems = w_elems + (a.add ? 2 * WORDS * THREADS * 16 / static_cast<int>(sizeof(T)) : 0);
    const T* wa = a.a + static_cast<int64_t>(tile.adapter) * R * K;
    const T* wb = a.b + static_cast<int64_t>(tile.adapter) * R * N;

    // second product: this thread's two slots, and the first column of its words of a warp's 32
    const int32_t mycol = lane % 4 * (FP32 ? 4 : 8);
    const YT* add = static_cast<const YT*>(a.add);
    YT* out = static_cast<YT*>(a.out);
    int64_t at[2];
    bool there2[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int32_t row = lane / 4 + 8 * h;
        there2[h] = row < tile.n;
        at[h] = static_cast<int64_t>(slots[there2[h] ? row : 0]) * N + mycol;
    }
    const int32_t up_steps = c0 < c1 ? (c1 - c0 + kFewUpCols - 1) / kFewUpCols : 0;
    auto load_up = [&](int32_t i) {
        const int32_t col = c0 + i * kFewUpCols;
        T* ws = up + i % UPS * up_elems;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int32_t c = tid / 2 + 64 * h;
            const bool in = col + c < c1;
            const T* src = wb + static_cast<int64_t>(in ? col + c : 0) * R;
            T* dst = ws + spread_col<FP32>(c) * pitch;
            for (int32_t ch = tid % 2; ch < 2 * ks; ch += 2) {
                const bool there = in && ch * 8 < R;
                copy16(dst + ch * 8, there ? src + ch * 8 : wb, there);
            }
        }
        if (add) {
            uint8_t* as = reinterpret_cast<uint8_t*>(ws + w_elems) + tid * 16;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int x = 0; x < WORDS; ++x) {
                    const int32_t c = col + warp * 32 + x * 16;
                    const bool there = there2[h] && c + mycol < c1;
                    copy16(as + (h * WORDS + x) * THREADS * 16, there ? add + at[h] + c : add, there);
                }
        }
    };

    // first product: this CTA's runs of 64 values
    const int32_t chunks = (K + kFewDownCols - 1) / kFewDownCols, per = (chunks + static_cast<int32_t>(size) - 1) / static_cast<int32_t>(size);
    const int32_t k0 = static_cast<int32_t>(rank) * per, steps = max(0, min(chunks - k0, per));
    const int32_t row = tid / 8, part = tid % 8 * 8, word = (tid % 8 ^ row % 8) * 8;      // 16 rows at a time
    const T* x = row < tile.n ? a.x + static_cast<int64_t>(slots[row] / a.div) * K : nullptr;
    auto load_down = [&](int32_t i) {
        const int32_t col = (k0 + i) * kFewDownCols + part;
        T* st = down + i % kFewStages * down_elems + row * kFewDownCols + word;
        const bool in = col < K;
        copy16(st, in && x ? x + col : a.x, in && x);
#pragma unroll
        for (int j = 0; j < KS; ++j)
            if (j * 16 + row < R) copy16(st + (j + 1) * 16 * kFewDownCols, in ? wa + static_cast<int64_t>(j * 16 + row) * K + col : wa, in);
    };
#pragma unroll
    for (int i = 0; i < kFewStages - 1; ++i) {
        if (i < steps) load_down(i);
        copies_commit();
    }
    float acc[NT][4] = {};
    const int32_t zat = lane % 16 * kFewDownCols + (2 * warp + lane / 16 ^ l) * 8, wword = (2 * warp + lane / 8 % 2 ^ l) * 8;
    for (int32_t i = 0; i < steps; ++i) {
        copies_wait<kFewStages - 2>();
        __syncthreads();
        if (i + kFewStages - 1 < steps) load_down(i + kFewStages - 1);
        copies_commit();
        const T* zs = down + i % kFewStages * down_elems;
        uint32_t z[4];
        ldsm4(z, zs + zat, false);
#pragma unroll
        for (int j = 0; j < NT / 2; ++j) {
            if (2 * j >= nt) break;
            const int32_t n = min(2 * j + lane / 16, nt - 1);      // an odd last tile stands in for its neighbour
            uint32_t w[4];
            ldsm4(w, zs + (kFewSlots + n * 8 + l) * kFewDownCols + wword, false);
            float sum[2][4] = {};      // a step's sums start from 0 (lora_down.cu)
            mma16(sum[0], z, w[0], w[1], T());
            mma16(sum[1], z, w[2], w[3], T());
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                acc[2 * j][q] += sum[0][q];
                acc[2 * j + 1][q] += sum[1][q];
            }
        }
    }
    copies_wait<0>();
    __syncthreads();
    // B's first stages, while the sums meet
#pragma unroll
    for (int i = 0; i < UPS - 1; ++i) {
        if (i < up_steps) load_up(i);
        copies_commit();
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        if (j >= nt) break;
        float* to = sums + (warp * kFewSlots + lane / 4) * R + j * 8 + lane % 4 * 2;
        *reinterpret_cast<float2*>(to) = make_float2(acc[j][0], acc[j][1]);
        *reinterpret_cast<float2*>(to + 8 * R) = make_float2(acc[j][2], acc[j][3]);
    }
    __syncthreads();
    for (int32_t i = tid; i < tile.n * R; i += THREADS) {
        float v = 0.0f;
#pragma unroll
        for (int p = 0; p < WARPS; ++p) v += sums[p * kFewSlots * R + i];
        mine[i] = v;
    }
    cluster_sync();
    const float scale = a.scales ? __ldg(a.scales + tile.adapter) : 1.0f;
    for (int32_t i = tid; i < tile.n * R; i += THREADS) {
        float v = 0.0f;
        for (uint32_t q = 0; q < size; ++q) v += cluster_load(mine + i, q);
        u_all[i] = scale * v;
    }
    cluster_sync();      // no CTA leaves while others read its sums

    Wide16<T> u[KS];
#pragma unroll
    for (int k = 0; k < KS; ++k) {
        float v[8];      // rows by h, ranks 2 q (+1) and 2 q + 8 (+1): mma's registers 0, 2 and 1, 3
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int32_t r = k * 16 + lane % 4 * 2 + 8 * i;
                const bool in = there2[h] && r < R;
                v[2 * (h + 2 * i)] = in ? u_all[(lane / 4 + 8 * h) * R + r] : 0.0f;
                v[2 * (h + 2 * i) + 1] = in ? u_all[(lane / 4 + 8 * h) * R + r + 1] : 0.0f;
            }
        u[k].set(v);
    }
    for (int32_t i = 0; i < up_steps; ++i) {
        copies_wait<UPS - 2>();
        __syncthreads();
        if (i + UPS - 1 < up_steps) load_up(i + UPS - 1);
        copies_commit();
        const int32_t col = c0 + i * kFewUpCols + warp * 32;
        const T* ws = up + i % UPS * up_elems;
        const uint8_t* as = reinterpret_cast<const uint8_t*>(ws + w_elems) + tid * 16;
        float sum[4][4] = {};
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            if (k >= ks) break;
            uint32_t w[4][2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t y[4];
                ldsm4(y, ws + (warp * 32 + (2 * j + lane / 16) * 8 + l) * pitch + k * 16 + lane / 8 % 2 * 8, false);
                w[2 * j][0] = y[0];
                w[2 * j][1] = y[1];
                w[2 * j + 1][0] = y[2];
                w[2 * j + 1][1] = y[3];
            }
            u[k].mul(sum, w);
        }
        constexpr int PER = 8 / WORDS;      // results of a word
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int y = 0; y < WORDS; ++y) {
                if (!there2[h] || col + y * 16 + mycol >= c1) continue;
                __align__(16) YT o[PER];
                if (add) *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(as + (h * WORDS + y) * THREADS * 16);
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const float v = sum[(y * PER + j) / 2][2 * h + j % 2];
                    o[j] = from_f32<YT>(add ? v + to_f32<YT>(o[j]) : v);
                }
                *reinterpret_cast<uint4*>(out + at[h] + col + y * 16) = *reinterpret_cast<const uint4*>(o);
            }
    }
    copies_wait<0>();
}

template <typename T, typename YT>
int launch_few_typed(FewArgs<T> a, cudaStream_t s) {
    const int32_t k_runs = (a.ncols + kFewDownCols - 1) / kFewDownCols, n_runs = (a.nrows + kFewUpCols - 1) / kFewUpCols;
    const int32_t most = k_runs > n_runs ? k_runs : n_runs;
    unsigned cluster = 1;
    while (cluster < 8 && static_cast<int32_t>(cluster) < most) cluster *= 2;
    a.per = (n_runs + static_cast<int32_t>(cluster) - 1) / static_cast<int32_t>(cluster) * kFewUpCols;
    const dim3 grid(static_cast<unsigned>(a.slots.n_slots) * cluster), block(kLoraThreads);
    const int32_t R = a.rank, pitch = odd_pitch((R + 15) / 16 * 16);
    auto go = [&](auto k, int nt) {
        size_t sm = static_cast<size_t>(kFewStages) * (kFewSlots + R) * kFewDownCols * 2 + 2 * static_cast<size_t>(kFewSlots) * R * 4;
        sm += static_cast<size_t>(few_up_stages(nt)) * (kFewUpCols * static_cast<size_t>(pitch) * 2 + (a.add ? 2 * sizeof(YT) * 8 * kLoraThreads : 0));
        return launch_with(k, "lora_few_kernel", grid, block, sm, false, cluster, s, a);
    };
    if (R <= 16) return go(lora_few_kernel<T, YT, 2>, 2);
    if (R <= 32) return go(lora_few_kernel<T, YT, 4>, 4);
    if (R <= 64) return go(lora_few_kernel<T, YT, 8>, 8);
    return go(lora_few_kernel<T, YT, 16>, 16);
}

template <typename T>
int launch_few(const LoraFew& f, const LoraPlan& p, cudaStream_t s) {
    FewArgs<T> a{};
    a.slots = LoraSlots{p.ids, nullptr, nullptr, nullptr, p.n_slots, p.n_adapters, kFewSlots};
    a.x = static_cast<const T*>(f.x);
    a.a = static_cast<const T*>(f.a);
    a.b = static_cast<const T*>(f.b);
    a.scales = p.scales;
    a.add = f.add;
    a.out = f.out;
    a.err = p.err;
    a.rank = p.rank;
    a.ncols = f.ncols;
    a.nrows = f.nrows;
    a.div = f.div;
    return f.out_f32 ? launch_few_typed<T, float>(a, s) : launch_few_typed<T, T>(a, s);
}

}  // namespace ft
