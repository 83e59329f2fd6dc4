// Load-balance loss of a router over packed sequences, and the experts' counts.
//
//   p_te    softmax(l)_e, or sigmoid(l)_e / max(sum, 1e-30), of row t
//   n_s     rows of sequence s with an expert that is not masked;  S' sequences with n_s > 0
//   c_se    slots of sequence s whose id is e;   P_se = sum of p_te over its rows
//   scale_s E / (top_k n_s^2 S'), 0 where n_s = 0
//   loss    sum_s scale_s sum_e c_se P_se
//
// Memory-bound: the logits are read once.  A CTA takes a run of rows, each by the lanes that hold its
// experts; P lies in the lanes' registers until the run or the sequence ends, where the CTA's lane groups
// are added up in order into a piece of the workspace, beside the counts.  A second launch adds the pieces of
// each sequence and expert up, and its last CTA to finish makes the loss; sums run in a fixed order, and only
// whole numbers are added by atomics.  CTA c's piece of sequence s is number c + s: both only rise along
// the rows, so that no two meet.  Batches of some rows and few sequences are one cluster's work, in one launch:
// its CTAs add up each other's shares through shared memory.
//
// 65536 rows of 128 fp32 in packed sequences: 12.9 us for the rows (34 MB, 2.6 TB/s: exponentials and sums, as much as the
// reads), 8.6 to join.  512 rows of 128 by one cluster: 8.8 us, a chain of loads, sums and meetings; by two launches
// that and the join's 8.  Four CTAs of an SM, one row of a lane group at work and one on its way: with two of each, three
// CTAs, 18 us.
#include <algorithm>
#include <type_traits>

#include "router_rows.cuh"
#include "ft_internal.h"
#include "launch.cuh"

namespace ft {

namespace {

constexpr int32_t kSingleRounds = 8, kSingleSeqs = 8;      // batches that one cluster works out: rounds of rows of a CTA, sequences
constexpr unsigned kSingleCtas = 8;
constexpr int32_t kLeastRounds = 2;                         // rounds of rows that a CTA takes at least
constexpr int kEarlyIds = 4;                                // ids of a thread asked for before the rows

struct Piece {
    float p;
    int32_t c;
};

struct BalanceArgs {
    const void* logits;
    const int32_t* ids;
    const int32_t* offsets;
    int64_t tokens, stride, rows_per_cta;
    int32_t n_experts, top_k, score, n_seqs;
    Piece* pieces;        // [ctas + n_seqs][n_experts]
    int32_t* piece_rows;  // [ctas + n_seqs]
    float* dots;          // [n_seqs][blocks of 8 experts]
    int32_t* seq_rows;    // [n_seqs]
    uint32_t* ticket;
    uint32_t* err;
    float* loss;
    int32_t* counts;
    float* seq_scale;
    bool wide, single;
};

// What a sequence of n rows has in the loss, of `full` sequences with rows.
__device__ __forceinline__ float seq_scale_of(const BalanceArgs& a, int32_t n, int32_t full) {
    const float rows = static_cast<float>(n);
    return n > 0 ? __fdiv_rn(static_cast<float>(a.n_experts), a.top_k * static_cast<float>(full) * rows * rows) : 0.0f;
}

// Sum over the CTA, in a fixed order, for every thread.
__device__ __forceinline__ float cta_sum(float v, float* part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31u) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < kRowThreads / 32; ++w) v += part[w];
    return v;
}

// seq_of for the whole CTA, which looks at 256 offsets at once.
__device__ __forceinline__ int32_t seq_of_cta(const int32_t* offsets, int32_t n, int64_t r) {
    if (n > 16 * kRowThreads) return seq_of(offsets, n, r);
    int32_t c = 0;
    for (int32_t s0 = 0; s0 < n; s0 += kRowThreads) {
        const int32_t s = s0 + static_cast<int32_t>(threadIdx.x);
        c += __syncthreads_count(s < n && __ldg(offsets + s) <= r);
    }
    return c > 0 ? c - 1 : 0;
}

template <typename T, int L, int STEPS>
__global__ void __launch_bounds__(kRowThreads, STEPS == 1 ? 4 : 2) balance_rows_kernel(const BalanceArgs a) {
    using G = RowGroup<L>;
    constexpr int WIDTH = 8 * L * STEPS;      // experts that the lanes have room for
    extern __shared__ __align__(16) uint8_t balance_smem[];
    float* part_sum = reinterpret_cast<float*>(balance_smem);                    // [8]
    float* part = part_sum + 8;                                                  // [8]
    int32_t* group_rows = reinterpret_cast<int32_t*>(part + 8);                // [rows at once]
    float* red = reinterpret_cast<float*>(group_rows + (G::kRows + 3) / 4 * 4);      // [rows at once][WIDTH]
    int32_t* hist = reinterpret_cast<int32_t*>(red + G::kRows * WIDTH);        // [E]
    float* share = reinterpret_cast<float*>(hist + a.n_experts);               // [E] P of this CTA (single)
    __shared__ float seq_dot[kSingleSeqs];                                     // of the experts that this CTA adds up
    __shared__ int32_t seq_n[kSingleSeqs];                                     // rows of this CTA
    let_next_grid_start();
    const G g{part};
    const int32_t E = a.n_experts, S = a.n_seqs, tid = threadIdx.x;
    const int64_t r0 = min(a.tokens, blockIdx.x * a.rows_per_cta);
    const int64_t r1 = r0 + a.rows_per_cta < a.tokens ? r0 + a.rows_per_cta : a.tokens;
    if (blockIdx.x == 0 && tid == 0 && !a.single) *a.ticket = 0;
    for (int32_t e = tid; e < E; e += kRowThreads) hist[e] = 0;
    __syncthreads();

    int64_t r = r0;
    for (int32_t s = a.single || !a.offsets ? 0 : seq_of_cta(a.offsets, S, r0); s < S && (a.single || r < r1); ++s) {
        const int64_t start = seq_start(a.offsets, s, a.tokens), end = seq_start(a.offsets, s + 1, a.tokens);
        const int64_t lo = start > r ? start : r, hi = end < r1 ? end : r1;
        if (lo >= hi && !a.single) continue;
        float acc[STEPS][8];
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
        int32_t rows = 0;
        // the first ids, and the next row: on their way while a row is worked on
        const int64_t id_end = hi * a.top_k;
        int64_t id_at = lo * a.top_k + tid;
        int32_t early[kEarlyIds];
#pragma unroll
        for (int i = 0; i < kEarlyIds; ++i) early[i] = id_at + i * kRowThreads < id_end ? __ldg(a.ids + id_at + i * kRowThreads) : -1;
        RowAhead<T, L, STEPS> ahead;
        auto row_of = [&](int64_t base) {
            const int64_t t = base + G::row();
            return static_cast<const T*>(a.logits) + (t < hi ? t : lo) * a.stride;
        };
        if (lo < hi) ahead.fetch(row_of(lo), E, a.wide);
        for (int64_t base = lo; base < hi; base += G::kRows) {      // whole groups: their lanes meet in shuffles
            float p[STEPS][8];
            ahead.take(row_of(base), E, a.wide, p);
            if (base + G::kRows < hi) ahead.fetch(row_of(base + G::kRows), E, a.wide);
            RowScale sc;
            float inv;
            if (a.score == FT_SCORE_SOFTMAX) {
                sc = row_softmax<L, STEPS>(g, p);
                inv = sc.inv;
            } else {
                float rest[STEPS][8];
                sc = row_sigmoid<L, STEPS>(g, p, rest);
                inv = __fdividef(1.0f, fmaxf(sc.sum, kScoreTiny));
            }
            if (base + G::row() < hi) {
                rows += sc.any ? 1 : 0;
#pragma unroll
                for (int i = 0; i < STEPS; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) acc[i][j] = fmaf(p[i][j], inv, acc[i][j]);
            }
        }
        auto count = [&](int32_t e) {
            if (e >= 0 && e < E) atomicAdd(&hist[e], 1);      // whole numbers: the order does not show
            else if (e != -1) atomicOr(a.err, FT_DEVERR_BAD_EXPERT_ID);
        };
#pragma unroll
        for (int i = 0; i < kEarlyIds; ++i) count(early[i]);
#pragma unroll 4
        for (id_at += kEarlyIds * kRowThreads; id_at < id_end; id_at += kRowThreads) count(__ldg(a.ids + id_at));
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            float4* to = reinterpret_cast<float4*>(red + G::row() * WIDTH + first_expert<L>(i));
            to[0] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
            to[1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
        }
        if (G::lane() == 0) group_rows[G::row()] = rows;
        __syncthreads();
        const int64_t piece = blockIdx.x + static_cast<int64_t>(s);
        for (int32_t e = tid; e < E; e += kRowThreads) {
            float p = 0.0f;
#pragma unroll 8
            for (int i = 0; i < G::kRows; ++i) p += red[i * WIDTH + e];
            if (a.single) {
                share[e] = p;
            } else {
                a.pieces[piece * E + e] = Piece{p, hist[e]};
                hist[e] = 0;
            }
        }
        if (tid == 0) {
            int32_t n = 0;
            for (int i = 0; i < G::kRows; ++i) n += group_rows[i];
            if (a.single) seq_n[s] = n;
            else a.piece_rows[piece] = n;
        }
        if (a.single) {
            cluster_sync();
            const uint32_t size = cluster_size(), rank = cluster_rank();
            float dot = 0.0f;
            for (int32_t e = tid * static_cast<int32_t>(size) + static_cast<int32_t>(rank); e < E; e += kRowThreads * static_cast<int32_t>(size)) {
                float p = 0.0f;
                int32_t c = 0;
                for (uint32_t q = 0; q < size; ++q) {
                    p += cluster_load(share + e, q);
                    c += __float_as_int(cluster_load(hist + e, q));
                }
                a.counts[static_cast<int64_t>(s) * E + e] = c;
                dot = fmaf(static_cast<float>(c), p, dot);
            }
            dot = cta_sum(dot, part_sum);
            if (tid == 0) seq_dot[s] = dot;
            cluster_sync();      // the others have read this CTA's shares
            for (int32_t e = tid; e < E; e += kRowThreads) hist[e] = 0;
        }
        __syncthreads();
        if (lo < hi) r = hi;
    }
    if (!a.single) return;
    if (cluster_rank() == 0 && tid < 32) {
        // lane q asks CTA q; every lane gets the sums
        int32_t n[kSingleSeqs], full = 0;
        float dot[kSingleSeqs], loss = 0.0f;
        const bool there = static_cast<uint32_t>(tid) < cluster_size();
#pragma unroll
        for (int s = 0; s < kSingleSeqs; ++s) {
            n[s] = there && s < S ? __float_as_int(cluster_load(seq_n + s, tid)) : 0;
            dot[s] = there && s < S ? cluster_load(seq_dot + s, tid) : 0.0f;
        }
#pragma unroll
        for (int s = 0; s < kSingleSeqs; ++s) {
#pragma unroll
            for (int o = static_cast<int>(kSingleCtas) / 2; o > 0; o >>= 1) {
                n[s] += __shfl_xor_sync(0xFFFFFFFFu, n[s], o);
                dot[s] += __shfl_xor_sync(0xFFFFFFFFu, dot[s], o);
            }
            full += n[s] > 0 ? 1 : 0;
        }
#pragma unroll
        for (int s = 0; s < kSingleSeqs; ++s) {
            const float scale = seq_scale_of(a, n[s], full);
            if (tid == 0 && s < S) a.seq_scale[s] = scale;
            loss = fmaf(scale, dot[s], loss);
        }
        if (tid == 0) *a.loss = loss;
    }
    cluster_sync();      // no CTA leaves while its sums are read
}

// Adds the pieces up: TASK threads per sequence and eight experts, a lane per expert in each of TASK / 8
// groups that share the pieces.
template <int TASK>
__global__ void __launch_bounds__(kRowThreads) balance_join_kernel(const BalanceArgs a) {
    __shared__ float part_sum[8];
    __shared__ Piece red[kRowThreads / 32][8];
    __shared__ int32_t red_rows[kRowThreads / 32];
    __shared__ bool last;
    wait_for_prior_grid();
    const int32_t E = a.n_experts, blocks = (E + 7) / 8;
    const int64_t tasks = static_cast<int64_t>(a.n_seqs) * blocks;
    const int64_t task = static_cast<int64_t>(blockIdx.x) * (kRowThreads / TASK) + threadIdx.x / TASK;
    const int32_t sub = threadIdx.x % TASK;
    const bool there = task < tasks;
    const int32_t s = !there ? 0 : tasks <= INT32_MAX ? static_cast<int32_t>(task) / blocks : static_cast<int32_t>(task / blocks);
    const int32_t b = there ? static_cast<int32_t>(task - static_cast<int64_t>(s) * blocks) : 0;
    const int32_t e = b * 8 + sub % 8;
    float p = 0.0f;
    int32_t c = 0, n = 0;
    if (there) {
        const int64_t lo = seq_start(a.offsets, s, a.tokens), hi = seq_start(a.offsets, s + 1, a.tokens);
        if (lo < hi) {
            const uint32_t per = static_cast<uint32_t>(a.rows_per_cta);      // tokens < 2^31
            const int64_t first = static_cast<uint32_t>(lo) / per, last_cta = static_cast<uint32_t>(hi - 1) / per;
#pragma unroll 8
            for (int64_t i = first + sub / 8; i <= last_cta; i += TASK / 8) {
                if (e < E) {
                    const int2 v = *reinterpret_cast<const int2*>(a.pieces + (i + s) * E + e);
                    p += __int_as_float(v.x);
                    c += v.y;
                }
                if (sub % 8 == 0 && b == 0) n += a.piece_rows[i + s];
            }
        }
    }
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
        p += __shfl_xor_sync(0xFFFFFFFFu, p, o);
        c += __shfl_xor_sync(0xFFFFFFFFu, c, o);
        n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
    }
    if constexpr (TASK == kRowThreads) {
        const uint32_t warp = threadIdx.x >> 5, lane = lane_id();
        if (lane < 8) red[warp][lane] = Piece{p, c};
        if (lane == 0) red_rows[warp] = n;
        __syncthreads();
        if (threadIdx.x < 8) {
            p = 0.0f;
            c = n = 0;
#pragma unroll
            for (int w = 0; w < kRowThreads / 32; ++w) {
                p += red[w][threadIdx.x].p;
                c += red[w][threadIdx.x].c;
                n += red_rows[w];
            }
        }
    }
    float dot = static_cast<float>(c) * p;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
    if (there && sub < 8) {
        if (e < E) a.counts[static_cast<int64_t>(s) * E + e] = c;
        if (sub == 0) {
            a.dots[task] = dot;
            if (b == 0) a.seq_rows[s] = n;
        }
    }
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(a.ticket, 1u) + 1 == gridDim.x;
    __syncthreads();
    if (!last) return;
    __threadfence();
    float full = 0.0f, loss = 0.0f;
    for (int32_t i = threadIdx.x; i < a.n_seqs; i += kRowThreads) full += __ldcg(a.seq_rows + i) > 0 ? 1.0f : 0.0f;
    const int32_t sequences = static_cast<int32_t>(cta_sum(full, part_sum));
    int32_t seq = static_cast<int32_t>(threadIdx.x) / blocks, rest = static_cast<int32_t>(threadIdx.x) % blocks;
    const int32_t seqs = kRowThreads / blocks, more = kRowThreads % blocks;
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < tasks; i += kRowThreads) {
        const float scale = seq_scale_of(a, __ldcg(a.seq_rows + seq), sequences);
        if (rest == 0) a.seq_scale[seq] = scale;
        loss = fmaf(scale, __ldcg(a.dots + i), loss);
        seq += seqs;
        rest += more;
        if (rest >= blocks) {
            rest -= blocks;
            ++seq;
        }
    }
    loss = cta_sum(loss, part_sum);
    if (threadIdx.x == 0) *a.loss = loss;
}

// Rows that a CTA takes at once.
int32_t rows_at_once(int32_t n_experts) {
    return with_row_lanes(n_experts, [](auto lanes, auto) { return kRowThreads / decltype(lanes)::value; });
}

int64_t balance_ctas(int64_t tokens, int32_t n_experts, int64_t most) {
    const int64_t rows = kLeastRounds * rows_at_once(n_experts), ctas = (tokens + rows - 1) / rows;
    return ctas < 1 ? 1 : ctas < most ? ctas : most;
}

bool balance_single(int64_t tokens, int32_t n_experts, int32_t n_seqs) {
    return n_seqs <= kSingleSeqs && tokens <= static_cast<int64_t>(kSingleCtas) * kSingleRounds * rows_at_once(n_experts);
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

// The CTAs depend on the device; the workspace has room for the most that there can be.
size_t balance_workspace(int64_t tokens, int32_t n_experts, int32_t n_seqs) {
    if (balance_single(tokens, n_experts, n_seqs)) return 0;
    const size_t S = static_cast<size_t>(n_seqs);
    const size_t pieces = static_cast<size_t>(balance_ctas(tokens, n_experts, kBalanceCtas)) + S;
    return 256 + up256(pieces * n_experts * sizeof(Piece)) + up256(pieces * 4) + up256(S * ((n_experts + 7) / 8) * 4) + up256(S * 4);
}

int launch_balance(const BalanceParams& p, const void* logits, int dtype, int64_t stride, const int32_t* ids,
                   const int32_t* offsets, float* loss, int32_t* counts, float* seq_scale, uint8_t* ws, uint32_t* err,
                   cudaStream_t s) {
    BalanceArgs a{};
    a.logits = logits;
    a.ids = ids;
    a.offsets = offsets;
    a.tokens = p.tokens;
    a.stride = stride;
    a.n_experts = p.n_experts;
    a.top_k = p.top_k;
    a.score = p.score;
    a.n_seqs = p.n_seqs;
    a.err = err;
    a.loss = loss;
    a.counts = counts;
    a.seq_scale = seq_scale;
    const int64_t rows = rows_at_once(p.n_experts);
    a.single = balance_single(p.tokens, p.n_experts, p.n_seqs);
    unsigned cluster = 1;
    while (a.single && cluster < kSingleCtas && p.tokens > static_cast<int64_t>(cluster) * kLeastRounds * rows) cluster *= 2;
    int64_t ctas = a.single ? cluster : balance_ctas(p.tokens, p.n_experts, std::min<int64_t>(4 * sm_count(), kBalanceCtas));
    a.rows_per_cta = p.tokens > 0 ? (p.tokens + ctas - 1) / ctas : 1;
    if (!a.single && p.tokens > 0) ctas = (p.tokens + a.rows_per_cta - 1) / a.rows_per_cta;
    const size_t pieces = static_cast<size_t>(ctas) + p.n_seqs, S = static_cast<size_t>(p.n_seqs);
    a.ticket = reinterpret_cast<uint32_t*>(ws);
    ws += 256;
    a.pieces = reinterpret_cast<Piece*>(ws);
    ws += up256(pieces * p.n_experts * sizeof(Piece));
    a.piece_rows = reinterpret_cast<int32_t*>(ws);
    ws += up256(pieces * 4);
    a.dots = reinterpret_cast<float*>(ws);
    ws += up256(S * ((p.n_experts + 7) / 8) * 4);
    a.seq_rows = reinterpret_cast<int32_t*>(ws);
    const int size = dtype == FT_DTYPE_F32 ? 4 : 2;
    a.wide = stride * size % 16 == 0 && reinterpret_cast<uintptr_t>(logits) % 16 == 0;
    const dim3 block(kRowThreads), grid(static_cast<unsigned>(ctas));
    const int st = with_row_lanes(p.n_experts, [&](auto lanes, auto steps) {
        constexpr int L = decltype(lanes)::value, N = decltype(steps)::value, ROWS = kRowThreads / L;
        const size_t sm = 64 + (ROWS + 3) / 4 * 16 + static_cast<size_t>(ROWS) * 8 * L * N * 4 + 8 * static_cast<size_t>(p.n_experts);
        if (dtype == FT_DTYPE_F32) return launch_with(balance_rows_kernel<float, L, N>, "balance_rows_kernel", grid, block, sm, false, cluster, s, a);
        if (dtype == FT_DTYPE_F16) return launch_with(balance_rows_kernel<__half, L, N>, "balance_rows_kernel", grid, block, sm, false, cluster, s, a);
        return launch_with(balance_rows_kernel<__nv_bfloat16, L, N>, "balance_rows_kernel", grid, block, sm, false, cluster, s, a);
    });
    if (st || a.single) return st;
    // a warp per eight experts of a sequence once the sequences are many and their pieces few
    const int64_t tasks = static_cast<int64_t>(p.n_seqs) * ((p.n_experts + 7) / 8);
    const bool wide_tasks = ctas / p.n_seqs >= 16;
    const int64_t join = wide_tasks ? tasks : (tasks + kRowThreads / 32 - 1) / (kRowThreads / 32);
    if (join > 0x7FFFFFFF) return fail(FT_ERR_SIZE, "too many sequences for one launch");
    const dim3 jgrid(static_cast<unsigned>(join));
    if (wide_tasks) return launch_with(balance_join_kernel<kRowThreads>, "balance_join_kernel", jgrid, block, 0, true, 1, s, a);
    return launch_with(balance_join_kernel<32>, "balance_join_kernel", jgrid, block, 0, true, 1, s, a);
}

}  // namespace ft
