// First product of a low-rank adapter: u[s] = W z[s], rank R, for slots s that share an adapter.
//
//   forward   z = x [rows][K], W = A [R][K]                 u = A x
//   backward  z = dy [slots][N], W = B^T of B [N][R]        B^T dy, beside the forward's u once more
//
// Memory-bound on z.  A tile of 64 slots (16 where adapters have few) by all R columns is a cluster's work: its
// CTAs share the inner dimension, and add their sums up through each other's shared memory, in a fixed order.
// z and W come by cp.async, four stages of 64 values; in tiles of 16 slots the four warps share a
// stage's values instead of its slots.
#include "lora.cuh"
#include "ft_internal.h"
#include "launch.cuh"

namespace ft {

namespace {

constexpr int kDownCols = 64, kDownPitch = kDownCols + 8, kDownStages = 4;

template <typename T>
struct DownJob {
    const T *z, *w;
    float* u;
    int32_t cols, div;      // row of slot s: s / div
    bool trans;             // W's values of one column are neighbours ([cols][R])
};

template <typename T>
struct DownArgs {
    DownJob<T> job[2];
    LoraSlots slots;
    uint32_t* err;
    int32_t rank;
};

__host__ __device__ inline int32_t down_w_elems(int32_t rank) {
    const int32_t a = rank * kDownPitch, b = kDownCols * odd_pitch(rank);
    return a > b ? a : b;
}

// NT: tiles of eight ranks that there is room for.
template <typename T, int MT, int NT>
__global__ void __launch_bounds__(kLoraThreads) lora_down_kernel(const __grid_constant__ DownArgs<T> a) {
    constexpr int PARTS = MT == kLoraTile ? 1 : kLoraThreads / 32;      // warps that share a tile's sums
    constexpr int ZR = MT / 16;
    extern __shared__ __align__(16) uint8_t down_smem[];
    __shared__ int32_t slots[MT];
    let_next_grid_start();
    const uint32_t size = cluster_size(), rank = cluster_rank();
    const DownJob<T>& job = a.job[blockIdx.y];
    const int32_t tid = static_cast<int32_t>(threadIdx.x), warp = tid >> 5, lane = tid & 31, b = static_cast<int32_t>(blockIdx.x / size);
    if (blockIdx.y == 0 && rank == 0) {      // the tiles are no fewer than the slots' MTs, or than the slots
        const int64_t s = a.slots.perm ? static_cast<int64_t>(b) * MT + tid : b;
        if (tid < (a.slots.perm ? MT : 1) && s < a.slots.n_slots) {
            const int32_t id = __ldg(a.slots.ids + s);
            if (id < -1 || id >= a.slots.n_adapters) atomicOr(a.err, FT_DEVERR_BAD_EXPERT_ID);
        }
    }
    const LoraTile tile = find_tile<MT>(a.slots, b, slots, kLoraThreads);
    if (tile.n == 0) return;      // all of the cluster
    const int32_t R = a.rank, nt = R / 8, cols = job.cols, pitch = odd_pitch(R);
    const int32_t stage_elems = MT * kDownPitch + down_w_elems(R);
    T* smem = reinterpret_cast<T*>(down_smem);
    const T* w = job.w + static_cast<int64_t>(tile.adapter) * R * cols;
    const int32_t chunks = (cols + kDownCols - 1) / kDownCols, per = (chunks + static_cast<int32_t>(size) - 1) / static_cast<int32_t>(size);
    const int32_t c0 = static_cast<int32_t>(rank) * per, n_chunks = max(0, min(chunks - c0, per));

    const int32_t part = tid % 8 * 8;      // of a row's 64 values
    const T* z[ZR];
#pragma unroll
    for (int i = 0; i < ZR; ++i) {
        const int32_t row = tid / 8 + 16 * i;
        z[i] = row < tile.n ? job.z + static_cast<int64_t>(slots[row] / job.div) * cols : nullptr;
    }
    auto load = [&](int32_t i) {
        const int32_t col = (c0 + i) * kDownCols;
        T* zs = smem + i % kDownStages * stage_elems;
        T* ws = zs + MT * kDownPitch;
        const bool in = col + part < cols;
#pragma unroll
        for (int j = 0; j < ZR; ++j) {
            const bool there = in && z[j] != nullptr;
            copy16(zs + (tid / 8 + 16 * j) * kDownPitch + part, there ? z[j] + col + part : job.z, there);
        }
        if (job.trans) {
            const int32_t words = R / 8;
#pragma unroll
            for (int j = 0; j < NT / 2; ++j) {
                const int32_t at = tid + j * kLoraThreads, row = at / words, ch = at - row * words;
                if (row < kDownCols) {
                    const bool there = col + row < cols;
                    copy16(ws + row * pitch + ch * 8, there ? w + static_cast<int64_t>(col + row) * R + ch * 8 : w, there);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < NT / 2; ++j) {
                const int32_t r = tid / 8 + 16 * j;
                if (r < R) copy16(ws + r * kDownPitch + part, in ? w + static_cast<int64_t>(r) * cols + col + part : w, in);
            }
        }
    };

    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
#pragma unroll
    for (int i = 0; i < kDownStages - 1; ++i) {
        if (i < n_chunks) load(i);
        copies_commit();
    }
    for (int32_t c = 0; c < n_chunks; ++c) {
        copies_wait<kDownStages - 2>();
        __syncthreads();
        if (c + kDownStages - 1 < n_chunks) load(c + kDownStages - 1);
        copies_commit();
        const T* zs = smem + c % kDownStages * stage_elems;
        const T* ws = zs + MT * kDownPitch;
        auto step = [&](int32_t k0, int32_t row0) {      // 16 values of 16 slots
            uint32_t x[4];
            ldsm4(x, zs + (row0 + lane % 16) * kDownPitch + k0 + lane / 16 * 8, false);
            const int32_t k = k0 + lane / 8 % 2 * 8, l = lane % 8;
#pragma unroll
            for (int j = 0; j < NT; j += 2) {
                if (j >= nt) break;
                const int32_t n = min(j + lane / 16, nt - 1);      // an odd last tile stands in for its neighbour
                uint32_t b[4];
                if (job.trans) ldsm4(b, ws + (k + l) * pitch + n * 8, true);
                else ldsm4(b, ws + (n * 8 + l) * kDownPitch + k, false);
                mma16(acc[j], x, b[0], b[1], T());
                if (j + 1 < nt) mma16(acc[j + 1], x, b[2], b[3], T());
            }
        };
        if constexpr (PARTS == 1) {
#pragma unroll
            for (int k = 0; k < kDownCols; k += 16) step(k, warp * 16);
        } else {
            step(warp * 16, 0);
        }
    }
    copies_wait<0>();
    __syncthreads();

    float* sums = reinterpret_cast<float*>(down_smem);      // [PARTS][MT][R]
    const int32_t row = (PARTS == 1 ? warp * 16 : warp * MT) + lane / 4;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        if (j >= nt) break;
        const int32_t col = j * 8 + lane % 4 * 2;
        *reinterpret_cast<float2*>(sums + row * R + col) = make_float2(acc[j][0], acc[j][1]);
        *reinterpret_cast<float2*>(sums + (row + 8) * R + col) = make_float2(acc[j][2], acc[j][3]);
    }
    cluster_sync();
    for (int32_t i = static_cast<int32_t>(rank) * kLoraThreads + tid; i < tile.n * R; i += static_cast<int32_t>(size) * kLoraThreads) {
        float v = 0.0f;
        for (uint32_t q = 0; q < size; ++q)
#pragma unroll
            for (int p = 0; p < PARTS; ++p) v += cluster_load(sums + p * MT * R + i, q);
        const int32_t s = i / R;
        job.u[static_cast<int64_t>(slots[s]) * R + (i - s * R)] = v;
    }
    cluster_sync();      // no CTA leaves while others read its sums
}

template <typename T, int MT>
int launch_down_typed(const DownArgs<T>& a, int64_t n_tiles, int jobs, unsigned cluster, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(n_tiles * cluster), static_cast<unsigned>(jobs)), block(kLoraThreads);
    size_t sm = static_cast<size_t>(kDownStages) * (MT * kDownPitch + down_w_elems(a.rank)) * sizeof(T);
    const size_t sums = static_cast<size_t>(MT == kLoraTile ? MT : 4 * MT) * a.rank * 4;
    if (sums > sm) sm = sums;
    auto go = [&](auto k) { return launch_with(k, "lora_down_kernel", grid, block, sm, false, cluster, s, a); };
    if (a.rank <= 16) return go(lora_down_kernel<T, MT, 2>);
    if (a.rank <= 32) return go(lora_down_kernel<T, MT, 4>);
    if (a.rank <= 64) return go(lora_down_kernel<T, MT, 8>);
    return go(lora_down_kernel<T, MT, 16>);
}

template <typename T>
int launch_down(const LoraDown* jobs, int n_jobs, const LoraPlan& p, cudaStream_t s) {
    DownArgs<T> a{};
    for (int i = 0; i < n_jobs; ++i)
        a.job[i] = DownJob<T>{static_cast<const T*>(jobs[i].z), static_cast<const T*>(jobs[i].w), jobs[i].u, jobs[i].cols,
                              jobs[i].div, jobs[i].trans};
    a.slots = LoraSlots{p.ids, p.offsets, p.tiles, p.perm, p.n_slots, p.n_adapters};
    a.rank = p.rank;
    a.err = p.err;
    // as many CTAs as fill the GPU a few times, each with four stages or more; the same for one of a call's
    // products as for both, so that leaving one out changes no bit of the other
    unsigned cluster = 1;
    while (cluster < 8 && p.n_tiles * p.down_jobs * cluster < 3 * static_cast<int64_t>(sm_count()) &&
           p.down_cols >= static_cast<int32_t>(2 * cluster) * 4 * kDownCols)
        cluster *= 2;
    return p.width == kLoraTile ? launch_down_typed<T, kLoraTile>(a, p.n_tiles, n_jobs, cluster, s)
                                : launch_down_typed<T, kLoraSmallTile>(a, p.n_tiles, n_jobs, cluster, s);
}

}  // namespace

int launch_lora_down(const LoraDown* jobs, int n_jobs, const LoraPlan& p, int dtype, cudaStream_t s) {
    return dtype == FT_DTYPE_F16 ? launch_down<__half>(jobs, n_jobs, p, s) : launch_down<__nv_bfloat16>(jobs, n_jobs, p, s);
}

}  // namespace ft
