// First product of a low-rank adapter: u[s] = W z[s], rank R, for slots s that share an adapter.
//
//   forward   z = x [rows][K], W = A [R][K]                 u = A x
//   backward  z = dy [slots][N], W = B^T of B [N][R]        B^T dy, beside the forward's u once more
//
// Memory-bound on z.  A tile of 64 or 128 slots (16 where adapters have few) by all R columns is a cluster's work: its
// CTAs share the inner dimension, and add their sums up through each other's shared memory, in a fixed order.
// z and W come by cp.async, four stages of 64 values; in tiles of 16 slots the four warps share a
// stage's values instead of its slots.  A row of a stage is one line of 128 bytes whose 16-byte words are exchanged by
// word ^ row % 8: the copies fill whole lines (64 MB through shared memory 8.4 us; rows 144 bytes apart 11.8, words by
// themselves 22), and a column of eight rows lies in all banks.
//
// The tensor cores cut what they add to an accumulator off at its last bit: after n additions a sum is too small
// by some n 2^-25 of itself.  So a stage's sums start from 0 and are added to the others by the CUDA cores.
#include <type_traits>

#include "lora.cuh"
#include "ft_internal.h"
#include "launch.cuh"

namespace ft {

namespace {

constexpr int kDownCols = 64, kDownStages = 4;

template <typename T>
struct DownJob {
    const T *z, *w;
    float* u;               // or null
    __nv_bfloat16* parts;   // or null
    int32_t cols, div;      // row of slot s: s / div
    bool trans;             // W's values of one column are neighbours ([cols][R])
};

template <typename T>
struct DownArgs {
    DownJob<T> job[2];
    LoraSlots slots;
    const float* scales;
    uint32_t* err;
    int32_t rank;
};

// Elements between the rows of W's stage where they are the inner dimension's: whole lines at rank 64, else an odd number of words.
__host__ __device__ inline int32_t down_turned_pitch(int32_t rank) { return rank % 64 == 0 ? rank : odd_pitch(rank); }
__host__ __device__ inline int32_t down_w_elems(int32_t rank) { return kDownCols * down_turned_pitch(rank) > rank * kDownCols ? kDownCols * down_turned_pitch(rank) : rank * kDownCols; }

// NT: tiles of eight ranks that there is room for.
template <typename T, int MT, int NT>
__global__ void __launch_bounds__(kLoraThreads) lora_down_kernel(const __grid_constant__ DownArgs<T> a) {
    constexpr int THREADS = kLoraThreads, PARTS = MT == kLoraSmallTile ? THREADS / 32 : 1;      // PARTS: warps that share a tile's sums
    constexpr int MS = MT == 128 ? 2 : 1, WARP_ROWS = 16 * MS;                                      // a warp's runs of 16 slots
    constexpr int ZS = THREADS / 8, ZR = (MT + ZS - 1) / ZS;                                        // rows that a copy of a word per thread takes
    extern __shared__ __align__(128) uint8_t down_smem[];
    __shared__ int32_t slots[MT];
    wait_for_prior_grid();
    let_next_grid_start();      // behind the wait: what comes up early may read the order
    const uint32_t size = cluster_size(), rank = cluster_rank();
    const DownJob<T>& job = a.job[blockIdx.y];
    const int32_t tid = static_cast<int32_t>(threadIdx.x), warp = tid >> 5, lane = tid & 31, b = static_cast<int32_t>(blockIdx.x / size);
    if (blockIdx.y == 0 && rank == 0 && tid < MT) {      // the tiles are no fewer than the slots' MTs
        const int64_t s = static_cast<int64_t>(b) * MT + tid;
        if (s < a.slots.n_slots) {
            const int32_t id = __ldg(a.slots.ids + s);
            if (id < -1 || id >= a.slots.n_adapters) atomicOr(a.err, FT_DEVERR_BAD_EXPERT_ID);
        }
    }
    const LoraTile tile = find_tile<MT>(a.slots, b, slots);
    if (tile.n == 0) return;      // all of the cluster
    const int32_t R = a.rank, nt = R / 8, cols = job.cols, pitch = down_turned_pitch(R);
    const int32_t stage_elems = MT * kDownCols + down_w_elems(R);
    T* smem = reinterpret_cast<T*>(down_smem);
    const T* w = job.w + static_cast<int64_t>(tile.adapter) * R * cols;
    const int32_t chunks = (cols + kDownCols - 1) / kDownCols, per = (chunks + static_cast<int32_t>(size) - 1) / static_cast<int32_t>(size);
    const int32_t c0 = static_cast<int32_t>(rank) * per, n_chunks = max(0, min(chunks - c0, per));

    const int32_t part = tid % 8 * 8, z_word = (tid % 8 ^ tid / 8 % 8) * 8;      // of a row's 64 values, where they go
    const T* z[ZR];
#pragma unroll
    for (int i = 0; i < ZR; ++i) {
        const int32_t row = tid / 8 + ZS * i;
        z[i] = row < tile.n ? job.z + static_cast<int64_t>(slots[row] / job.div) * cols : nullptr;
    }
    constexpr int WJ = (NT * 64 + THREADS - 1) / THREADS;      // 16-byte words of W's stage that a thread copies
    const int32_t nt8 = R * 8;                                 // words of the stage: 64 values of R rows
    float acc[MS][NT][4] = {};
    auto product = [&](auto turned) {
        constexpr bool TRANS = decltype(turned)::value;
        int32_t from[WJ], to[WJ], edge[WJ];      // where a word comes from and goes; its first value along the inner dimension
#pragma unroll
        for (int j = 0; j < WJ; ++j) {
            const int32_t at = tid + j * THREADS, words = TRANS ? R / 8 : kDownCols / 8, row = at / words, ch = at - row * words;
            from[j] = TRANS ? row * R + ch * 8 : row * cols + ch * 8;
            to[j] = TRANS ? row * pitch + (R % 64 == 0 ? ch ^ row % 8 : ch) * 8 : row * kDownCols + (ch ^ row % 8) * 8;
            edge[j] = at >= nt8 ? 1 << 30 : TRANS ? row : ch * 8;
        }
        auto load = [&](int32_t i) {
            const int32_t col = (c0 + i) * kDownCols;
            T* zs = smem + i % kDownStages * stage_elems;
            T* ws = zs + MT * kDownCols;
#pragma unroll
            for (int j = 0; j < ZR; ++j) {
                const bool there = col + part < cols && z[j] != nullptr;
                copy16(zs + (tid / 8 + ZS * j) * kDownCols + z_word, there ? z[j] + col + part : job.z, there);
            }
            const T* wc = w + static_cast<int64_t>(col) * (TRANS ? R : 1);
#pragma unroll
            for (int j = 0; j < WJ; ++j) {
                const bool there = col + edge[j] < cols;
                if (edge[j] < kDownCols) copy16(ws + to[j], there ? wc + from[j] : w, there);
            }
        };
#pragma unroll
        for (int i = 0; i < kDownStages - 1; ++i) {
            if (i < n_chunks) load(i);
            copies_commit();
        }
        // what this lane gives the address of: 16 slots by 16 values of z, pairs of W's tiles by 16 values
        constexpr int KK = PARTS == 1 ? kDownCols / 16 : 1;
        const int32_t row0 = PARTS == 1 ? warp * WARP_ROWS : 0, first = PARTS == 1 ? 0 : warp, l = lane % 8;      // first: step of 16 values
        const int32_t zat = (row0 + lane % 16) * kDownCols;
        int32_t zword[KK], wword[KK], wat[NT / 2];
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            zword[kk] = (2 * (first + kk) + lane / 16 ^ l) * 8;
            wword[kk] = TRANS ? 16 * (first + kk) * pitch : (2 * (first + kk) + lane / 8 % 2 ^ l) * 8;
        }
#pragma unroll
        for (int j = 0; j < NT / 2; ++j) {
            const int32_t n = min(2 * j + lane / 16, nt - 1);      // an odd last tile stands in for its neighbour
            wat[j] = TRANS ? (lane / 8 % 2 * 8 + l) * pitch + (R % 64 == 0 ? n ^ l : n) * 8 : (n * 8 + l) * kDownCols;
        }
        for (int32_t c = 0; c < n_chunks; ++c) {
            copies_wait<kDownStages - 2>();
            __syncthreads();
            if (c + kDownStages - 1 < n_chunks) load(c + kDownStages - 1);
            copies_commit();
            const T* zs = smem + c % kDownStages * stage_elems;
            const T* ws = zs + MT * kDownCols;
            uint32_t x[MS][KK][4];
#pragma unroll
            for (int m = 0; m < MS; ++m)
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) ldsm4(x[m][kk], zs + zat + m * 16 * kDownCols + zword[kk], false);
#pragma unroll
            for (int j = 0; j < NT / 2; ++j) {
                if (2 * j >= nt) break;
                float sum[MS][2][4] = {};
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) {
                    uint32_t b[4];
                    ldsm4(b, ws + wat[j] + wword[kk], TRANS);
#pragma unroll
                    for (int m = 0; m < MS; ++m) {
                        mma16(sum[m][0], x[m][kk], b[0], b[1], T());
                        mma16(sum[m][1], x[m][kk], b[2], b[3], T());      // behind an odd last tile: not looked at
                    }
                }
#pragma unroll
                for (int m = 0; m < MS; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        acc[m][2 * j][i] += sum[m][0][i];
                        acc[m][2 * j + 1][i] += sum[m][1][i];
                    }
            }
        }
    };
    if (job.trans) product(std::true_type());
    else product(std::false_type());
    copies_wait<0>();
    __syncthreads();

    float* sums = reinterpret_cast<float*>(down_smem);      // [PARTS][MT][R]
#pragma unroll
    for (int m = 0; m < MS; ++m) {
        const int32_t row = (PARTS == 1 ? warp * WARP_ROWS + m * 16 : warp * MT) + lane / 4;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if (j >= nt) break;
            const int32_t col = j * 8 + lane % 4 * 2;
            *reinterpret_cast<float2*>(sums + row * R + col) = make_float2(acc[m][j][0], acc[m][j][1]);
            *reinterpret_cast<float2*>(sums + (row + 8) * R + col) = make_float2(acc[m][j][2], acc[m][j][3]);
        }
    }
    const float scale = a.scales ? __ldg(a.scales + tile.adapter) : 1.0f;
    cluster_sync();
    for (int32_t i = static_cast<int32_t>(rank) * THREADS + tid; i < tile.n * R; i += static_cast<int32_t>(size) * THREADS) {
        float v = 0.0f;
        for (uint32_t q = 0; q < size; ++q)
#pragma unroll
            for (int p = 0; p < PARTS; ++p) v += cluster_load(sums + p * MT * R + i, q);
        const int32_t s = i / R, r = i - s * R;
        if (job.u) job.u[static_cast<int64_t>(slots[s]) * R + r] = v;
        if (job.parts) {
            v *= scale;
            __nv_bfloat16* to = job.parts + static_cast<int64_t>(tile.first + s) * 3 * R + r;
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                const __nv_bfloat16 h = __float2bfloat16_rn(v);
                *to = h;
                v -= __bfloat162float(h);
                to += R;
            }
        }
    }
    cluster_sync();      // no CTA leaves while others read its sums
}

template <typename T, int MT>
int launch_down_typed(const DownArgs<T>& a, const LoraPlan& p, int jobs, cudaStream_t s) {
    size_t sm = static_cast<size_t>(kDownStages) * (MT * kDownCols + down_w_elems(a.rank)) * sizeof(T);
    const size_t sums = static_cast<size_t>(MT == kLoraSmallTile ? 4 * MT : MT) * a.rank * 4;
    if (sums > sm) sm = sums;
    // As many CTAs as the GPU holds at once, with four stages of work or more each.  By what a call can have, not what it has:
    // leaving out one product changes no bit of the other.
    const int64_t per_sm = static_cast<int64_t>(220 * 1024 / (sm + 1024)), fit = (per_sm < 8 ? per_sm : 8) * sm_count();
    unsigned cluster = 1;
    while (cluster < 8 && p.n_tiles * p.down_jobs * 2 * cluster <= fit * 5 / 4 && p.down_cols >= static_cast<int32_t>(2 * cluster) * 4 * kDownCols)
        cluster *= 2;
    const dim3 grid(static_cast<unsigned>(p.n_tiles * cluster), static_cast<unsigned>(jobs)), block(kLoraThreads);
    auto go = [&](auto k) { return launch_with(k, "lora_down_kernel", grid, block, sm, true, cluster, s, a); };
    if (a.rank <= 16) return go(lora_down_kernel<T, MT, 2>);
    if (a.rank <= 32) return go(lora_down_kernel<T, MT, 4>);
    if (a.rank <= 64) return go(lora_down_kernel<T, MT, 8>);
    return go(lora_down_kernel<T, MT, 16>);
}

template <typename T>
int launch_down(const LoraDown* jobs, int n_jobs, const LoraPlan& p, cudaStream_t s) {
    DownArgs<T> a{};
    for (int i = 0; i < n_jobs; ++i)
        a.job[i] = DownJob<T>{static_cast<const T*>(jobs[i].z), static_cast<const T*>(jobs[i].w), jobs[i].u, static_cast<__nv_bfloat16*>(jobs[i].parts), jobs[i].cols,
                              jobs[i].div, jobs[i].trans};
    a.slots = LoraSlots{p.ids, p.offsets, p.tiles, p.perm, p.n_slots, p.n_adapters, p.width};
    a.rank = p.rank;
    a.err = p.err;
    a.scales = p.scales;
    if (p.width == 128) return launch_down_typed<T, 128>(a, p, n_jobs, s);
    if (p.width == 64) return launch_down_typed<T, 64>(a, p, n_jobs, s);
    return launch_down_typed<T, kLoraSmallTile>(a, p, n_jobs, s);
}

}  // namespace

int launch_lora_down(const LoraDown* jobs, int n_jobs, const LoraPlan& p, int dtype, cudaStream_t s) {
    return dtype == FT_DTYPE_F16 ? launch_down<__half>(jobs, n_jobs, p, s) : launch_down<__nv_bfloat16>(jobs, n_jobs, p, s);
}

}  // namespace ft
