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
// themselves 22), and a column of eight rows lies in all banks.  Where a tile's rows of z are neighbours, as in prompts and in
// training, and where W's lines are 128 bytes, a fifth warp has them brought by TMA instead.
//
// The tensor cores cut what they add to an accumulator off at its last bit: after n additions a sum is too small
// by some n 2^-25 of itself.  So a stage's sums start from 0 and are added to the others by the CUDA cores.
//
// 8191 slots of 4096 values, rank 16: 18 us, 3.7 TB/s of x; 16384 of 2048, rank 8: 16 us (the rows from L2 for all
// of a token's slots but the first: what copies bring into an SM, 32 bytes a clock, bounds it).  8192 slots, both products
// of 4096 x 64: 46 us, 2.9 TB/s; the additions by the CUDA cores, one for every 64 products, cost there as much as the MMAs.
#include <type_traits>

#include "gemm_common.cuh"
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
    uint8_t* parts;         // or null
    int32_t cols, div;      // row of slot s: s / div
    bool trans;             // W's values of one column are neighbours ([cols][R])
};

template <typename T>
struct DownArgs {
    CUtensorMap zmap[2], wmap[2];      // boxes of MT rows, of a stage of W
    bool tma[2], w_tma[2];
    DownJob<T> job[2];
    LoraSlots slots;
    const float* scales;
    uint32_t* err;
    int32_t rank;
};

// Elements between the rows of W's stage where they are the inner dimension's: whole lines at rank 64, else an odd number of words.
__host__ __device__ inline int32_t down_turned_pitch(int32_t rank) { return rank % 64 == 0 ? rank : odd_pitch(rank); }
__host__ __device__ inline int32_t down_w_elems(int32_t rank) { return kDownCols * down_turned_pitch(rank) > rank * kDownCols ? kDownCols * down_turned_pitch(rank) : rank * kDownCols; }

// NT: tiles of eight ranks that there is room for.  TMA: a fifth warp has neighbouring rows brought.
template <typename T, int MT, int NT, bool TMA>
__global__ void __launch_bounds__(TMA ? kLoraThreads + 32 : kLoraThreads, MT == 128 ? 2 : 1) lora_down_kernel(const __grid_constant__ DownArgs<T> a) {
    constexpr int THREADS = kLoraThreads, PARTS = MT == kLoraSmallTile ? THREADS / 32 : 1;      // PARTS: warps that share a tile's sums
    constexpr int MS = MT == 128 ? 2 : 1, WARP_ROWS = 16 * MS;                                      // a warp's runs of 16 slots
    constexpr int ZS = THREADS / 8, ZR = (MT + ZS - 1) / ZS;                                        // rows that a copy of a word per thread takes
    extern __shared__ uint8_t down_smem_raw[];
    uint8_t* down_smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(down_smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ int32_t slots[MT];
    __shared__ __align__(8) uint64_t full[kDownStages];
    wait_for_prior_grid();
    let_next_grid_start();      // behind the wait, by every CTA: the second product comes up early and reads the order before its own wait
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
    if (TMA && tid == 0) {
        for (int i = 0; i < kDownStages; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
    }
    const LoraTile tile = find_tile<MT>(a.slots, b, slots);      // ends behind a barrier
    if (tile.n == 0) return;      // all of the cluster
    // whether this tile's rows of z are neighbours
    const bool run = TMA && a.tma[blockIdx.y] && job.div == 1 && slots[tile.n - 1] - slots[0] == tile.n - 1, w_tma = run && a.w_tma[blockIdx.y];
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
        z[i] = row < tile.n && tid < THREADS ? job.z + static_cast<int64_t>(slots[row] / job.div) * cols : nullptr;
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
            if (TMA && tid == THREADS && (run || w_tma)) {
                uint64_t* bar = &full[i % kDownStages];
                mbar_arrive_expect_tx(bar, (run ? MT * 128u : 0u) + (w_tma ? static_cast<uint32_t>(R) * 128u : 0u));
                if (run) tma_load_2d(zs, &a.zmap[blockIdx.y], col, slots[0], bar);
                if (w_tma) tma_load_2d(ws, &a.wmap[blockIdx.y], TRANS ? 0 : col, tile.adapter * (TRANS ? cols : R) + (TRANS ? col : 0), bar);
            }
            if (TMA && tid >= THREADS) return;
#pragma unroll
            for (int j = 0; j < ZR; ++j) {
                if (run) break;
                const bool there = col + part < cols && z[j] != nullptr;
                copy16(zs + (tid / 8 + ZS * j) * kDownCols + z_word, there ? z[j] + col + part : job.z, there);
            }
            const T* wc = w + static_cast<int64_t>(col) * (TRANS ? R : 1);
#pragma unroll
            for (int j = 0; j < WJ; ++j) {
                if (w_tma) break;
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
        bool ok = true;
        for (int32_t c = 0; c < n_chunks; ++c) {
            copies_wait<kDownStages - 2>();
            if (run || w_tma) ok = mbar_wait(&full[c % kDownStages], static_cast<uint32_t>(c / kDownStages & 1), a.err) && ok;
            if constexpr (TMA) {
                ok = __syncthreads_and(ok);
                if (!ok) {      // what is under way lands before the CTA's memory goes
                    for (int32_t q = c; (run || w_tma) && q < n_chunks && q < c + kDownStages - 1; ++q)
                        mbar_wait(&full[q % kDownStages], static_cast<uint32_t>(q / kDownStages & 1), a.err, kLastWaitNs);
                    break;
                }
            } else {
                __syncthreads();
            }
            if (c + kDownStages - 1 < n_chunks) load(c + kDownStages - 1);
            copies_commit();
            const T* zs = smem + c % kDownStages * stage_elems;
            const T* ws = zs + MT * kDownCols;
            if (TMA && tid >= THREADS) continue;
            uint32_t x[MS][KK][4];
#pragma unroll
            for (int m = 0; m < MS; ++m)
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) ldsm4(x[m][kk], zs + zat + m * 16 * kDownCols + zword[kk], false);
            constexpr int JU = NT >= 4 && MS == 1 ? 2 : 1;      // pairs of W's tiles at once: enough sums that none waits for itself
#pragma unroll
            for (int j0 = 0; j0 < NT / 2; j0 += JU) {
                if (2 * j0 >= nt) break;
                float sum[JU][MS][2][4] = {};
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) {
                    uint32_t b[JU][4];
#pragma unroll
                    for (int j = 0; j < JU; ++j) ldsm4(b[j], ws + wat[j0 + j] + wword[kk], TRANS);
#pragma unroll
                    for (int j = 0; j < JU; ++j)
#pragma unroll
                        for (int m = 0; m < MS; ++m) {      // behind the last tile: not looked at
                            mma16(sum[j][m][0], x[m][kk], b[j][0], b[j][1], T());
                            mma16(sum[j][m][1], x[m][kk], b[j][2], b[j][3], T());
                        }
                }
#pragma unroll
                for (int j = 0; j < JU; ++j)
#pragma unroll
                    for (int m = 0; m < MS; ++m)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            acc[m][2 * (j0 + j)][i] += sum[j][m][0][i];
                            acc[m][2 * (j0 + j) + 1][i] += sum[j][m][1][i];
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
        if (TMA && tid >= THREADS) break;
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
    const int32_t passes = part_passes(R), q4 = R / 4;
    const int64_t places = a.slots.n_slots;
    cluster_sync();
    for (int32_t i = static_cast<int32_t>(rank) * THREADS + tid; tid < THREADS && i < tile.n * q4; i += static_cast<int32_t>(size) * THREADS) {
        const int32_t s = i / q4, r = (i - s * q4) * 4;
        float4 x[8], v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
#pragma unroll
            for (uint32_t q = 0; q < 8; ++q)      // all asked for before the first is added
                if (q < size) x[q] = cluster_load4(sums + p * MT * R + i * 4, q);
#pragma unroll
            for (uint32_t q = 0; q < 8; ++q)
                if (q < size) v = make_float4(v.x + x[q].x, v.y + x[q].y, v.z + x[q].z, v.w + x[q].w);
        }
        if (job.u) *reinterpret_cast<float4*>(job.u + static_cast<int64_t>(slots[s]) * R + r) = v;
        if (job.parts) {
            uint32_t lo[3], hi[3];
            split_pair(v.x * scale, v.y * scale, lo);
            split_pair(v.z * scale, v.w * scale, hi);
            int32_t kind = 0;      // lines of the passes before
#pragma unroll
            for (int t = 0; t < 3; ++t) {
                if (t > 0 && part_pass(passes, t) != part_pass(passes, t - 1)) kind += part_lines(R, part_pass(passes, t - 1));
                const int32_t m = part_row(passes, R, t) + r;
                uint8_t* line = job.parts + ((kind + m / 64) * places + tile.first + s) * 128;
                *reinterpret_cast<uint2*>(line + (m % 64 / 8 ^ s % 8) * 16 + m % 8 * 2) = make_uint2(lo[t], hi[t]);
            }
        }
    }
    if (job.parts && passes == 2) {      // rows behind the third part's add to the second's: zeros
        const int32_t words = 8 - R / 8;
        for (int32_t i = static_cast<int32_t>(rank) * THREADS + tid; tid < THREADS && i < tile.n * words; i += static_cast<int32_t>(size) * THREADS) {
            const int32_t s = i / words, word = R / 8 + i - s * words;
            uint8_t* line = job.parts + (part_lines(R, 0) * places + tile.first + s) * 128;
            *reinterpret_cast<uint4*>(line + (word ^ s % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    cluster_sync();      // no CTA leaves while others read its sums
}

template <typename T, int MT, bool TMA>
int launch_down_typed(const DownArgs<T>& a, const LoraPlan& p, int jobs, cudaStream_t s) {
    size_t sm = static_cast<size_t>(kDownStages) * (MT * kDownCols + down_w_elems(a.rank)) * sizeof(T);
    const size_t sums = static_cast<size_t>(MT == kLoraSmallTile ? 4 * MT : MT) * a.rank * 4;
    if (sums > sm) sm = sums;
    sm += 1024;
    // As many CTAs as the GPU holds at once, with four stages of work or more each: a call of 8191 slots 58 us from a graph,
    // with half the cluster 60, with twice 63; 509 slots' gradients 32, 34, 32; 8192's 144, 165, 154.  By what a call can
    // have, not what it has: leaving out one product changes no bit of the other.
    const int64_t per_sm = static_cast<int64_t>(220 * 1024 / (sm + 1024)), fit = (per_sm < 8 ? per_sm : 8) * sm_count();
    unsigned cluster = 1;
    while (cluster < 8 && p.n_tiles * p.down_jobs * 2 * cluster <= fit * 5 / 4 && p.down_cols >= static_cast<int32_t>(2 * cluster) * 4 * kDownCols)
        cluster *= 2;
    const dim3 grid(static_cast<unsigned>(p.n_tiles * cluster), static_cast<unsigned>(jobs)), block(TMA ? kLoraThreads + 32 : kLoraThreads);
    auto go = [&](auto k) { return launch_with(k, "lora_down_kernel", grid, block, sm, true, cluster, s, a); };
    if (a.rank <= 16) return go(lora_down_kernel<T, MT, 2, TMA>);
    if (a.rank <= 32) return go(lora_down_kernel<T, MT, 4, TMA>);
    if constexpr (MT == 128) {      // tiles of 128 slots have a rank of 64 at most
        return go(lora_down_kernel<T, MT, 8, TMA>);
    } else {
        if (a.rank <= 64) return go(lora_down_kernel<T, MT, 8, TMA>);
        return go(lora_down_kernel<T, MT, 16, TMA>);
    }
}

template <typename T>
int launch_down(const LoraDown* jobs, int n_jobs, const LoraPlan& p, cudaStream_t s) {
    DownArgs<T> a{};
    const CUtensorMapDataType type = std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    for (int i = 0; i < n_jobs; ++i) {
        const LoraDown& j = jobs[i];
        a.job[i] = DownJob<T>{static_cast<const T*>(j.z), static_cast<const T*>(j.w), j.u, static_cast<uint8_t*>(j.parts), j.cols, j.div, j.trans};
        if (p.width == kLoraSmallTile) continue;
        const uint64_t cols = static_cast<uint64_t>(j.cols), bytes = cols * 2, rank = static_cast<uint64_t>(p.rank), L = static_cast<uint64_t>(p.n_adapters);
        a.tma[i] = j.div == 1 && j.cols >= kDownCols;
        if (a.tma[i])
            if (int st = encode_2d(&a.zmap[i], type, j.z, cols, static_cast<uint64_t>(p.n_slots), bytes, kDownCols, static_cast<uint32_t>(p.width),
                                   CU_TENSOR_MAP_SWIZZLE_128B, "rows of an adapter"))
                return st;
        // (turned, a box of the last columns would hold another adapter's rows, which may be no numbers)
        a.w_tma[i] = j.trans ? p.rank == kDownCols && j.cols % kDownCols == 0 : j.cols >= kDownCols;
        if (a.w_tma[i])
            if (int st = j.trans ? encode_2d(&a.wmap[i], type, j.w, rank, L * cols, rank * 2, kDownCols, kDownCols, CU_TENSOR_MAP_SWIZZLE_128B, "adapters")
                                 : encode_2d(&a.wmap[i], type, j.w, cols, L * rank, bytes, kDownCols, static_cast<uint32_t>(p.rank),
                                             CU_TENSOR_MAP_SWIZZLE_128B, "adapters"))
                return st;
    }
    a.slots = LoraSlots{p.ids, p.offsets, p.tiles, p.perm, p.n_slots, p.n_adapters, p.width};
    a.rank = p.rank;
    a.err = p.err;
    a.scales = p.scales;
    const bool tma = a.tma[0] || a.tma[n_jobs - 1];
    if (p.width == 128) return tma ? launch_down_typed<T, 128, true>(a, p, n_jobs, s) : launch_down_typed<T, 128, false>(a, p, n_jobs, s);
    if (p.width == 64) return tma ? launch_down_typed<T, 64, true>(a, p, n_jobs, s) : launch_down_typed<T, 64, false>(a, p, n_jobs, s);
    return launch_down_typed<T, kLoraSmallTile, false>(a, p, n_jobs, s);
}

}  // namespace

int launch_lora_down(const LoraDown* jobs, int n_jobs, const LoraPlan& p, int dtype, cudaStream_t s) {
    return dtype == FT_DTYPE_F16 ? launch_down<__half>(jobs, n_jobs, p, s) : launch_down<__nv_bfloat16>(jobs, n_jobs, p, s);
}

}  // namespace ft
