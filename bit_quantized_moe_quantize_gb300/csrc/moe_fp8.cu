// Routed expert products in 8-bit floating point with a scale per block of 128:
//
//   out[s][r] = sum_b sa[row(s)][b] sw[e][r / 128][b] sum_{i in block b} w[e][r][i] a[row(s)][i]
//
// with e = topk_ids[s] and row(s) = s / act_div (act_div = top_k: one
// activation row per token; 1: one per slot), and the dense product (one
// matrix, slot s = row s).
//
// One tile: up to 256 slots of an expert x 256 of its weight rows, worked by a
// pair of CTAs with 2-CTA tcgen05 MMAs (kind::f8f6f4, M = 256 slots, N = the
// tile's weight rows rounded up to 32).  Each CTA loads its 128 slots' rows and
// half of the weight rows per block of 128 columns, so an operand byte in shared
// memory is read once for 256 x 256 products.  A block's products are summed by the tensor
// core in fp32 in tensor-memory accumulators (of 128 columns, two for each half of the tile, in
// turn); the scales change with the next block, so the drain takes each block's
// sums out of tensor memory and adds them, times sa * sw, to fp32 registers.
// Slots lie along the lanes, so that product is one number per thread: with the
// weight rows along the lanes a thread needs one scale per column, and reading
// those from shared memory for 32 rows at a time, or taking the accumulator out
// in 16-lane shapes to share them (half the rate: 514 cycles a block against 144),
// costs more than the MMAs of the block (512 cycles).
//
// Per CTA, warp-specialised:
//   8 drain warps  in two warpgroups, one per 128 weight rows (half) of the tile; warp w:
//                  TMEM lanes 32 (w % 4) .. + 31, one slot per thread
//   producer       TMA: the weight boxes, and the slots' rows in boxes of 32
//                  neighbouring rows, with 128-byte swizzle; columns past the
//                  row's end arrive as 0
//   MMA            (leader CTA) per block and half four MMAs of 32 columns, into
//                  one of the half's two accumulators of 128 columns
//
// An accumulator goes from the MMA to the drain warps of both CTAs and back, which
// takes about 1000 cycles on top of the MMAs (637 a block) and the drain: four
// accumulators of 128 columns in flight hide more of it than two of 256.
//
// Rows lie in router order: a TMA gather fetches four 128-byte rows per instruction
// and takes the unit about 85 cycles, so 128 slots a CTA would need 2700 a block.
//
// Bound by the drain beside the MMAs: a block takes some 920 cycles (dense 8192^3, all tiles
// full: 415 to 436 us, 2.5 to 2.65 PFLOP/s), where the MMAs alone take 512.  Routed, the tiles of 256 slots
// are not full: 8191 tokens, 8 of 128 experts, 1408 x 2816: 343 us with the order and the copies of
// the rows, 1.51 PFLOP/s.
#include <atomic>

#include "fp8_order.cuh"
#include "fp8_quant.cuh"
#include "fp8_tc.cuh"
#include "ft_internal.h"
#include "gemm_common.cuh"

namespace ft {

struct Pair {
    static constexpr int BM = 128;                 // slots per CTA
    static constexpr int BN = 256;                 // weight rows per tile
    static constexpr int STAGES = 4;
    static constexpr int A_BYTES = BM * kFp8Block;
    static constexpr int B_BYTES = BN / 2 * kFp8Block;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int BOX = 64;                 // weight rows per TMA box (half a half)
    static constexpr int ROW_BOX = 32;             // slots' rows per TMA box in router order
    static constexpr int N_DRAIN_WARPS = 8;
    static constexpr int WARP_PRODUCER = 8, WARP_MMA = 9, N_MMA_WARPS = 2, WARP_ZERO = 11;
    static constexpr int THREADS = 12 * 32;
    // registers: 384 threads are launched with LAUNCH_REGS each; the drain warps
    // take drain_regs, and the others give theirs down to other_regs
    static constexpr int LAUNCH_REGS = 168;
    static constexpr int drain_regs(bool gated) { return gated ? 216 : 200; }
    static constexpr int other_regs(bool gated) { return gated ? 72 : 104; }
    static_assert(216 * 256 + 72 * 128 <= LAUNCH_REGS * THREADS && 200 * 256 + 104 * 128 <= LAUNCH_REGS * THREADS,
                  "the split must fit the launch's registers");
    static constexpr int CW = BN / 2;              // columns of a half
    static constexpr int STAGE_ROW = 256 + 16;     // output staging: 256 bytes of a slot's row, and 16 so that
                                                   // eight lanes' 16-byte words fall in different banks
    static constexpr int OFF_OUT = STAGES * STAGE_BYTES;
    static constexpr int OFF_SCALE = OFF_OUT + N_DRAIN_WARPS * 32 * STAGE_ROW;
    static constexpr int SCALE_RING = 4;           // groups of four blocks' scales in flight
    static constexpr int OFF_BAR = OFF_SCALE + SCALE_RING * (N_DRAIN_WARPS * 32 + 2 * N_DRAIN_WARPS) * 16 + 4 * BM * 4;
    static constexpr int OFF_AMAX = OFF_BAR - 4 * BM * 4;       // [tile parity][half][slot], gated
    static constexpr int N_BARS = 2 * STAGES + 8 + 4;
    static constexpr int OFF_TMEM = OFF_BAR + N_BARS * 8;
    // offsets[E + 1] and tiles[E + 1] of up to MAX_E experts (a search in global memory waits for it at every step)
    static constexpr int MAX_E = 1024;
    static constexpr int OFF_ORDER = OFF_TMEM + 16;
    static constexpr int OFF_SLOT = OFF_ORDER + 2 * (MAX_E + 1) * 4;     // [tile parity][drain thread]
    static constexpr int SMEM_BYTES = OFF_SLOT + 2 * N_DRAIN_WARPS * 32 * 4 + 1024;    // + alignment slack
    static_assert(SMEM_BYTES <= 232448, "shared memory budget");
    static_assert(2 * BM == kWideTile, "slots per tile");
};

struct PairArgs {
    const int32_t* ids;          // [n_slots], nullptr: dense
    const int32_t* perm;         // router order -> slot (nullptr: dense)
    const int32_t* offsets;      // [n_experts + 1]
    const int32_t* tiles;        // [n_experts + 1] prefix of tiles of 256 slots
    const float* act_scales;
    const float* w_scales;
    uint32_t* err;
    int64_t n_slots, nrows;
    int32_t n_experts, nb, row_tiles, row_blocks;
    int32_t scale_pitch;         // act_scales: elements between rows
    bool scale_words;            // four neighbouring activation scales from a multiple of 4 on are a 16-byte word
    bool wide;                   // the rows of out are whole 16-byte words
    // gated: the weight rows are n_inter gate rows and n_inter up rows; a tile is 128 of
    // each, and the epilogue writes codes and scales of act(gate) * up in router order
    uint8_t* mid;
    float* mid_scales;
    int32_t n_inter, mid_pitch, act_kind;
};

struct PairTile {
    int32_t e, n, half, width;   // expert, valid slots, slots of CTA 0 (the rest are CTA 1's), MMA width
    int32_t p0, r0;              // first router position, first weight row
    // slots of CTA `rank`, and their first position
    __device__ int32_t mine(uint32_t rank) const { return rank ? n - half : half; }
    __device__ int32_t first(uint32_t rank) const { return p0 + (rank ? half : 0); }
    // MMA columns of half h (0, or past 0 where the tile has none)
    __device__ int32_t cols(int32_t h) const { return min(Pair::CW, width - h * Pair::CW); }
};

// A CTA pair's way through the tiles, `step` apart: row tile rt of slot tile st, of expert
// e.  The next one costs a few additions and a short walk over the experts; a division and a
// search per tile took the drain some 600 cycles.
struct PairWalk {
    int32_t st, rt, e, step_st, step_rt, row_tiles, slot_tiles;

    __device__ PairWalk(const PairArgs& a, const int32_t* tiles, int32_t first, int32_t step) {
        row_tiles = a.row_tiles;
        slot_tiles = tiles ? tiles[a.n_experts] : static_cast<int32_t>((a.n_slots + 2 * Pair::BM - 1) / (2 * Pair::BM));
        st = first / row_tiles;
        rt = first - st * row_tiles;
        step_st = step / row_tiles;
        step_rt = step - step_st * row_tiles;
        e = tiles && st < slot_tiles ? last_not_above(tiles, a.n_experts, st) : 0;
    }
    __device__ bool there() const { return st < slot_tiles; }
    __device__ void next(const int32_t* tiles) {
        st += step_st;
        rt += step_rt;
        if (rt >= row_tiles) {
            rt -= row_tiles;
            ++st;
        }
        if (tiles && st < slot_tiles)
            while (tiles[e + 1] <= st) ++e;      // tiles[n_experts] = slot_tiles > st ends it
    }
    __device__ PairTile tile(const PairArgs& a, const int32_t* tiles, const int32_t* offsets) const {
        PairTile t;
        t.e = e;
        t.r0 = rt * Pair::BN;
        t.width = (min(Pair::BN, static_cast<int32_t>(a.nrows) - t.r0) + 31) / 32 * 32;
        int32_t first = 0, count = static_cast<int32_t>(a.n_slots), j = st;
        if (tiles) {
            first = offsets[e];
            count = offsets[e + 1] - first;
            j = st - tiles[e];
        }
        t.p0 = first + j * (2 * Pair::BM);
        t.n = min(2 * Pair::BM, count - j * (2 * Pair::BM));
        t.half = min(t.n, (t.n + 63) / 64 * 32);        // whole warps, nearly even
        return t;
    }
};

// Two fp32 values in one 64-bit register, the operand of the packed FMA.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}

// The two as bf16, the first in the low half.
__device__ __forceinline__ uint32_t bf16x2(uint64_t v) {
    const float2 f = unpack2(v);
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(f.y), "f"(f.x));
    return r;
}

// acc += {lo, hi} * s
__device__ __forceinline__ void fma2(uint64_t& acc, uint32_t lo, uint32_t hi, uint64_t s) {
    asm("{\n\t.reg .b64 v;\n\tmov.b64 v, {%1, %2};\n\tfma.rn.f32x2 %0, v, %3, %0;\n\t}" : "+l"(acc) : "r"(lo), "r"(hi), "l"(s));
}

// The ring of scales: group g of four blocks lies in slot g % SCALE_RING.  A thread
// copies (asynchronously) and reads its own activation scales; the weight scales are
// its warp's.  A register would hold a load that the next block's code waits for
// even when an older one is wanted: with three blocks in flight in registers the
// products of a block waited 100 cycles.
template <int STEP>
__device__ __forceinline__ float4* ring_at(float4* ring, int32_t g) {
    return ring + g % Pair::SCALE_RING * STEP;
}

__device__ __forceinline__ void copy_async4(uint32_t dst, const void* src, int32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Starts the copies of group g (blocks past the row's end arrive as 0) and closes
// their group of asynchronous copies; groups past the last one close empty.
template <bool GATED>
__device__ __forceinline__ void copy_scales(const PairArgs& a, const float* sa, const float* sw, int32_t g, float4* ring_a,
                                            float4* ring_w) {
    const int32_t b = 4 * g;
    if (b < a.nb) {
        const uint32_t da = smem_u32(ring_at<256>(ring_a, g)), dw = smem_u32(ring_at<16>(ring_w, g));
        if (a.scale_words) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(da), "l"(sa + b) : "memory");
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) copy_async4(da + 4 * i, sa + min(b + i, a.nb - 1), b + i < a.nb ? 4 : 0);
        }
        const int32_t i = static_cast<int32_t>(lane_id());
        if (i < 4) copy_async4(dw + 4 * i, sw + min(b + i, a.nb - 1), b + i < a.nb ? 4 : 0);
        if constexpr (GATED) {      // the up rows' scales lie n_inter / 128 rows of blocks further
            if (i >= 4 && i < 8)
                copy_async4(dw + 8 * 16 + 4 * (i - 4), sw + static_cast<int64_t>(a.n_inter / kFp8Block) * a.nb + min(b + i - 4, a.nb - 1),
                            b + i - 4 < a.nb ? 4 : 0);
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// GATED: TO is unused.
template <typename TO, bool GATED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Pair::THREADS, 1)
    moe_fp8_pair_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                        const __grid_constant__ PairArgs a, TO* __restrict__ out) {
    using C = Pair;
    extern __shared__ uint8_t smem_raw[];
    // both CTAs round up by the same amount: their dynamic shared memory starts at the same offset
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* empty = full + C::STAGES;
    uint64_t* acc_full = empty + C::STAGES;      // [half][buffer]
    uint64_t* acc_empty = acc_full + 4;
    uint64_t* amax_bar = acc_empty + 4;          // gated: the two warps of 32 slots have stored their maxima
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_TMEM);

    const uint32_t warp = threadIdx.x >> 5, lane = lane_id(), rank = cluster_ctarank();
    const int32_t nb = a.nb;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], C::N_MMA_WARPS);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], C::N_DRAIN_WARPS);         // the leader's: a warpgroup of both CTAs
            mbar_init(&amax_bar[i], 2);
        }
        fence_mbar_init();
    }
    if (warp == C::WARP_MMA) tmem_alloc_pair(tmem_slot, 512);
    if (warp == C::WARP_PRODUCER && lane == 0) {
        prefetch_tmap(&wmap);
        prefetch_tmap(&xmap);
    }
    const int32_t *offsets = a.offsets, *tiles = a.tiles;
    if (tiles && a.n_experts <= C::MAX_E) {
        int32_t *o = reinterpret_cast<int32_t*>(smem + C::OFF_ORDER), *n = o + C::MAX_E + 1;
        for (int32_t e = static_cast<int32_t>(threadIdx.x); e <= a.n_experts; e += C::THREADS) {
            o[e] = offsets[e];
            n[e] = tiles[e];
        }
        offsets = o;
        tiles = n;
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    PairWalk walk(a, tiles, static_cast<int32_t>(blockIdx.x / 2), static_cast<int32_t>(gridDim.x / 2));

    if (warp >= C::N_DRAIN_WARPS) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::other_regs(GATED)));
        if (warp == C::WARP_PRODUCER) {
            // ------------------------------------------------------------ producer
            uint32_t it = 0;
            bool ok = true;
            for (; walk.there() && ok; walk.next(tiles)) {
                const PairTile t = walk.tile(a, tiles, offsets);
                const int32_t mine = t.mine(rank), other = t.mine(rank ^ 1u);
                constexpr int PER = C::ROW_BOX;      // lane l copies 32 of this CTA's slots
                const bool copies = static_cast<int32_t>(lane) * PER < mine;
                const int32_t y = t.first(rank) + static_cast<int32_t>(lane) * PER;
                // half h of the tile (weight rows 128 h ..): this CTA's part of its MMA's columns
                const int32_t halves = t.width > C::CW ? 2 : 1;
                const int64_t row0 = static_cast<int64_t>(t.e) * a.nrows + t.r0;
                // gated: columns 0 .. 63 of half h are gate rows 64 h .., columns 64 .. 127 the same up rows
                const int32_t wy = GATED ? static_cast<int32_t>(static_cast<int64_t>(t.e) * a.nrows + t.r0 / 2 + lane * C::BOX + rank * a.n_inter)
                                         : static_cast<int32_t>(row0 + lane * C::CW + rank * (t.cols(static_cast<int32_t>(lane)) / 2));
                const uint32_t bytes = 2 * halves * C::BOX * kFp8Block +
                                       ((mine + PER - 1) / PER + (other + PER - 1) / PER) * PER * kFp8Block;
                for (int32_t b = 0; b < nb; ++b, ++it) {
                    const uint32_t s = it % C::STAGES;
                    if (!mbar_wait_warp(&empty[s], ((it / C::STAGES) & 1u) ^ 1u, a.err)) { ok = false; break; }
                    const uint32_t bar = map_to_rank(smem_u32(&full[s]), 0);
                    const uint32_t dst = smem_u32(smem + s * C::STAGE_BYTES);
                    if (lane == 0 && rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
                    if (static_cast<int32_t>(lane) < halves)
                        tma_load_2d_pair(dst + C::A_BYTES + lane * (C::BOX * kFp8Block), &wmap, b * kFp8Block, wy, bar);
                    if (copies) tma_load_2d_pair(dst + lane * (PER * kFp8Block), &xmap, b * kFp8Block, y, bar);
                    __syncwarp();
                }
            }
            // the last fills: read by their MMAs, or at least arrived, before the CTA's memory goes
            for (uint32_t f = it - min(it, static_cast<uint32_t>(C::STAGES)); f != it; ++f) {
                const uint32_t s = f % C::STAGES, parity = (f / C::STAGES) & 1u;
                if (mbar_wait_warp(&empty[s], parity, a.err, ok ? kWaitLimitNs : kLastWaitNs)) continue;
                ok = false;
                if (rank == 0) mbar_wait_warp(&full[s], parity, a.err, kLastWaitNs);
            }
        } else if (warp < C::WARP_ZERO) {
            // ----------------------------------------------------------------- MMA
            // Warp h issues the MMAs of half h.  The whole warp runs the loop and one elected
            // lane issues: with the operands in uniform registers four MMAs and a commit take
            // 180 cycles to issue, from a single-lane branch 295, more than the 256 that they run.
            if (rank == 0) {
                const uint32_t h = warp - C::WARP_MMA;
                const bool elected = elect_one();
                const uint64_t desc0 = smem_desc_sw128(smem_u32(smem));
                const uint64_t bskip = (C::A_BYTES + h * (C::BOX * kFp8Block)) >> 4;
                uint32_t s = 0, phase = 0, done = 0;      // stage, its phase, blocks of this half
                bool ok = true;
                for (; walk.there() && ok; walk.next(tiles)) {
                    const PairTile t = walk.tile(a, tiles, offsets);
                    const int32_t cols = t.cols(static_cast<int32_t>(h));
                    const uint32_t idesc = idesc_e4m3_f32(2 * C::BM, max(cols, 0));
                    for (int32_t b = 0; b < nb; ++b) {
                        const uint32_t d = 2 * h + (done & 1u);
                        if (cols > 0) {
                            if (!mbar_wait2_warp(&full[s], phase, &acc_empty[d], ((done >> 1) & 1u) ^ 1u, a.err)) { ok = false; break; }
                            ++done;
                            tc_fence_after();
                            if (elected) {
                                const uint64_t adesc = desc0 + ((s * C::STAGE_BYTES) >> 4), bdesc = adesc + bskip;
#pragma unroll
                                for (int k = 0; k < 4; ++k) tc_mma_f8_pair(tmem + d * C::CW, adesc + 2 * k, bdesc + 2 * k, idesc, k);
                                tc_commit_pair(&acc_full[d]);
                                tc_commit_pair(&empty[s]);
                            }
                        } else {
                            if (!mbar_wait_warp(&full[s], phase, a.err)) { ok = false; break; }
                            if (elected) tc_commit_pair(&empty[s]);
                        }
                        if (++s == C::STAGES) {
                            s = 0;
                            phase ^= 1u;
                        }
                    }
                }
            }
            __syncwarp();
        } else if (!GATED && a.ids) {
            zero_unrouted<TO>(a.ids, a.n_slots, a.n_experts, a.nrows, a.err, out, blockIdx.x, gridDim.x);
        }
    } else {
        // --------------------------------------------------------------- drain
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::drain_regs(GATED)));
        const uint32_t lane0 = (warp & 3u) * 32u, h = warp >> 2;
        const uint32_t acc_empty0 = map_to_rank(smem_u32(acc_empty), 0);
        uint8_t* stage = smem + C::OFF_OUT + warp * (32 * C::STAGE_ROW);
        // this thread's word of the ring of activation scales, and its warp's of the ring of weight scales
        float4* ring_a = reinterpret_cast<float4*>(smem + C::OFF_SCALE) + threadIdx.x;
        float4* ring_w = reinterpret_cast<float4*>(smem + C::OFF_SCALE) + C::SCALE_RING * 256 + warp;     // + 8: the up rows'
        float* amax_of = reinterpret_cast<float*>(smem + C::OFF_AMAX);                                     // [tile parity][half][slot]
        uint32_t tiles_done = 0;         // gated: tiles that this warp had slots of
        uint32_t it = 0;                 // blocks of this half
        bool ok = true;
        // The tile to come: its place, this thread's slot in it and where its scales lie, looked
        // up after the last one's epilogue (before it, the lookup delays the rows that are
        // waiting: 207 us against 199 for 65536 slots x 2048 x 768).
        struct Next {
            int32_t r0, mine;
            const float *sa, *sw;
        } next;
        // this warp's rows of `out` (gated: of mid), of the current and the coming tile
        int32_t* rows_of = reinterpret_cast<int32_t*>(smem + C::OFF_SLOT) + warp * 32;
        uint32_t parity = 0;             // of the coming tile
        const int32_t m = static_cast<int32_t>(lane0 + lane);            // this thread's slot of the CTA
        auto look = [&]() {
            const PairTile t = walk.tile(a, tiles, offsets);
            next.r0 = GATED ? t.r0 / 2 : t.r0 + static_cast<int32_t>(h) * C::CW;      // first weight row of this half's scales
            next.mine = t.mine(rank);
            next.sa = a.act_scales;
            next.sw = a.w_scales + (static_cast<int64_t>(t.e) * a.row_blocks + min(next.r0 / kFp8Block, a.row_blocks - 1)) * nb;
            if (m < next.mine) {
                const int32_t p = t.first(rank) + m;
                int32_t* row = rows_of + parity * (C::N_DRAIN_WARPS * 32) + lane;
                // (a copy: a load would be waited for here, to be stored)
                if (GATED || !a.perm) *row = p;
                else copy_async4(smem_u32(row), a.perm + p, 4);
                next.sa += static_cast<int64_t>(p) * a.scale_pitch;
            }
            parity ^= 1u;
            // four blocks' scales at a time, through a ring in shared memory
            if (static_cast<int32_t>(lane0) < next.mine && (GATED || next.r0 < a.nrows)) {
#pragma unroll
                for (int i = 0; i < C::SCALE_RING - 1; ++i) copy_scales<GATED>(a, next.sa, next.sw, i, ring_a, ring_w);
            }
        };
        bool more = walk.there();
        if (more) look();
        while (more && ok) {
            const int32_t r0 = next.r0, mine = next.mine;
            const float *sa = next.sa, *sw = next.sw;
            if (!GATED && r0 >= a.nrows) {
                walk.next(tiles);
                more = walk.there();
                if (more) look();
                continue;
            }
            const bool busy = static_cast<int32_t>(lane0) < mine;        // the warp has a slot at all
            uint64_t acc[C::CW / 2];
#pragma unroll
            for (int i = 0; i < C::CW / 2; ++i) acc[i] = 0;
            const uint32_t tm = tmem + h * (2 * C::CW) + (lane0 << 16);     // buffer d of this half: + 128 d
            if (!busy) {
                for (int32_t b = 0; b < nb; ++b, ++it) {
                    if (!mbar_wait_warp(&acc_full[2 * h + (it & 1u)], (it >> 1) & 1u, a.err)) { ok = false; break; }
                    if (lane == 0) mbar_arrive_remote(acc_empty0 + (2 * h + (it & 1u)) * 8);
                }
                if (!ok) break;
                walk.next(tiles);
                more = walk.there();
                if (more) look();
                continue;
            }
            float sc[4] = {0.0f, 0.0f, 0.0f, 0.0f}, su[GATED ? 4 : 1] = {};      // gated: the up rows' beside the gate rows'
            // 16 columns are on their way from tensor memory while the 16 before them are added
            uint32_t v[2][16];
            if (!mbar_wait_warp(&acc_full[2 * h + (it & 1u)], (it >> 1) & 1u, a.err)) { ok = false; break; }
            tc_fence_after();
            tmem_ld_32x32b_x16(tm + (it & 1u) * C::CW, v[0]);
            for (int32_t b = 0; b < nb; ++b) {
                if ((b & 3) == 0) {
                    asm volatile("cp.async.wait_group %0;" ::"n"(C::SCALE_RING - 2) : "memory");
                    __syncwarp();
                    const float4 x = *ring_at<256>(ring_a, b >> 2), y = *ring_at<16>(ring_w, b >> 2);
                    sc[0] = x.x * y.x;
                    sc[1] = x.y * y.y;
                    sc[2] = x.z * y.z;
                    sc[3] = x.w * y.w;
                    if constexpr (GATED) {
                        const float4 z = *ring_at<16>(ring_w + 8, b >> 2);
                        su[0] = x.x * z.x;
                        su[1] = x.y * z.y;
                        su[2] = x.z * z.z;
                        su[3] = x.w * z.w;
                    }
                    __syncwarp();      // before the slot is filled again
                    copy_scales<GATED>(a, sa, sw, (b >> 2) + C::SCALE_RING - 1, ring_a, ring_w);
                }
                const float scale = sc[0];
                sc[0] = sc[1];
                sc[1] = sc[2];
                sc[2] = sc[3];
                const uint64_t s2 = pack2(scale, scale), u2 = GATED ? pack2(su[0], su[0]) : s2;
                if constexpr (GATED) {
                    su[0] = su[1];
                    su[1] = su[2];
                    su[2] = su[3];
                }
                const uint32_t nd = 2 * h + ((it + 1) & 1u), nph = ((it + 1) >> 1) & 1u;      // the next block's accumulator
                bool ready = false;
#pragma unroll
                for (int j = 0; j < C::CW / 16; ++j) {
                    tmem_wait_ld_regs(v[j & 1]);
                    if (j == C::CW / 16 - 3) ready = mbar_test(&acc_full[nd], nph);      // its latency passes under the sums
                    if (j < C::CW / 16 - 1) {
                        tmem_ld_32x32b_x16(tm + (it & 1u) * C::CW + 16 * (j + 1), v[(j + 1) & 1]);
                    } else {      // the block is in registers: its accumulator goes back, the next one's first columns come
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_remote(acc_empty0 + (2 * h + (it & 1u)) * 8);
                        ++it;
                        if (b + 1 < nb) {
                            if (!__all_sync(0xFFFFFFFFu, ready) && !mbar_wait_warp(&acc_full[nd], nph, a.err)) { ok = false; break; }
                            tc_fence_after();
                            tmem_ld_32x32b_x16(tm + (it & 1u) * C::CW, v[0]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) fma2(acc[8 * j + i], v[j & 1][2 * i], v[j & 1][2 * i + 1], j < C::CW / 32 ? s2 : u2);
                }
                if (!ok) break;
            }
            if (!ok) break;
            walk.next(tiles);
            more = walk.there();
            __syncwarp();      // every lane has read the last of this tile's scales

            // `parity` has moved on since this tile's rows were written
            const int32_t* rows = rows_of + (parity ^ 1u) * (C::N_DRAIN_WARPS * 32);
            if constexpr (GATED) {
                // this thread's 64 of the slot's 128 values; the other half's thread has the rest
                float amax = 0.0f;
#pragma unroll
                for (int i = 0; i < C::CW / 4; i += 4) {
                    uint64_t g[4], up[4], v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        g[j] = acc[i + j];
                        up[j] = acc[C::CW / 4 + i + j];
                    }
                    act_mul_pairs<4>(g, up, a.act_kind, v);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 x = split2(v[j]);
                        amax = max_nan(amax, fabsf(x.x), fabsf(x.y));
                        acc[i + j] = v[j];
                    }
                }
                float* both = amax_of + (tiles_done & 1u) * (2 * C::BM);
                both[h * C::BM + m] = amax;
                __syncwarp();
                if (lane == 0) mbar_arrive(&amax_bar[warp & 3u]);
                if (!mbar_wait_warp(&amax_bar[warp & 3u], tiles_done & 1u, a.err)) { ok = false; break; }
                amax = max_nan(amax, both[(h ^ 1u) * C::BM + m]);      // written again two tiles on, when the other warp has read it
                ++tiles_done;
                const float scale = __fdiv_rn(amax, kFp8Max), inv = rcp_approx(scale);      // as the quantizer's
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint2 q[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint64_t x[4] = {acc[8 * i + 4 * k], acc[8 * i + 4 * k + 1], acc[8 * i + 4 * k + 2], acc[8 * i + 4 * k + 3]};
                        q[k] = fp8_codes(x, scale, inv);
                    }
                    *reinterpret_cast<uint4*>(stage + lane * 80 + 16 * i) = make_uint4(q[0].x, q[0].y, q[1].x, q[1].y);
                }
                const int32_t p0 = rows[0], n = min(32, mine - static_cast<int32_t>(lane0));
                if (h == 0 && m < mine) a.mid_scales[static_cast<int64_t>(p0 + static_cast<int32_t>(lane)) * a.mid_pitch + r0 / kFp8Block] = scale;
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {      // eight rows at a time, 64 bytes of each
                    const int32_t r = 8 * i + static_cast<int32_t>(lane >> 2);
                    if (r < n)
                        *reinterpret_cast<uint4*>(a.mid + static_cast<int64_t>(p0 + r) * a.n_inter + r0 + h * 64 + (lane & 3u) * 16) =
                            *reinterpret_cast<const uint4*>(stage + r * 80 + (lane & 3u) * 16);
                }
                __syncwarp();
                if (more) look();
                continue;
            }
            // out: 256 bytes of each of the warp's rows at a time go through shared memory,
            // so that a row leaves in whole lines
            constexpr int PER = 16 / static_cast<int>(sizeof(TO)), PASS = 256 / static_cast<int>(sizeof(TO));
            const int32_t rows_here = min(32, mine - static_cast<int32_t>(lane0));
#pragma unroll
            for (int ps = 0; ps < C::CW / PASS; ++ps) {
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    uint4 o;
                    if constexpr (sizeof(TO) == 2) {
                        o = make_uint4(bf16x2(acc[4 * i]), bf16x2(acc[4 * i + 1]), bf16x2(acc[4 * i + 2]), bf16x2(acc[4 * i + 3]));
                    } else {
                        const float2 f = unpack2(acc[ps * (PASS / 2) + 2 * i]), g = unpack2(acc[ps * (PASS / 2) + 2 * i + 1]);
                        o = make_uint4(__float_as_uint(f.x), __float_as_uint(f.y), __float_as_uint(g.x), __float_as_uint(g.y));
                    }
                    *reinterpret_cast<uint4*>(stage + lane * C::STAGE_ROW + 16 * i) = o;
                }
                __syncwarp();
                const int32_t c0 = r0 + ps * PASS;
                const int32_t left = min(PASS, static_cast<int32_t>(a.nrows) - c0);
                if (a.wide) {
#pragma unroll 4
                    for (int k = 0; k < 16; ++k) {       // two rows at a time, 16 bytes a lane
                        const int32_t r = 2 * k + static_cast<int32_t>(lane >> 4), c = static_cast<int32_t>(lane & 15u) * PER;
                        if (r < rows_here && c < left)
                            *reinterpret_cast<uint4*>(out + static_cast<int64_t>(rows[r]) * a.nrows + c0 + c) =
                                *reinterpret_cast<const uint4*>(stage + r * C::STAGE_ROW + (lane & 15u) * 16);
                    }
                } else {
                    // single elements, four rows' at a time: one after the other waits for shared memory
                    // at each (8191 tokens, 1407 x 2816 of 128 experts: 459 us instead of 375)
                    constexpr int ROWS = 4;
                    for (int q = 0; q < rows_here; q += ROWS) {
                        TO x[ROWS][PASS / 32];
                        int32_t slot[ROWS];
#pragma unroll
                        for (int k = 0; k < ROWS; ++k) {
                            slot[k] = rows[min(q + k, 31)];
                            const TO* src = reinterpret_cast<const TO*>(stage + min(q + k, 31) * C::STAGE_ROW) + lane;
#pragma unroll
                            for (int i = 0; i < PASS / 32; ++i) x[k][i] = src[32 * i];
                        }
#pragma unroll
                        for (int k = 0; k < ROWS; ++k) {
                            TO* dst = out + static_cast<int64_t>(slot[k]) * a.nrows + c0 + lane;
#pragma unroll
                            for (int i = 0; i < PASS / 32; ++i)
                                if (q + k < rows_here && static_cast<int32_t>(lane) + 32 * i < left) dst[32 * i] = x[k][i];
                        }
                    }
                }
            }
            if (more) look();
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync_all();      // the peer's arrivals and operand reads are over
    if (warp == C::WARP_MMA) tmem_dealloc_pair(tmem, 512);
}

// Activation rows and scales in router order: a warp per position.  Rows of scales lie
// `pitch` apart (a multiple of 4, so that a drain thread takes four with one copy).
__global__ void __launch_bounds__(256)
    order_rows_kernel(const uint8_t* __restrict__ act, const float* __restrict__ scales, const int32_t* __restrict__ perm,
                      const int32_t* __restrict__ n_routed, int32_t act_div, int32_t row_words, int32_t nb, int32_t pitch,
                      uint4* __restrict__ act_out, float* __restrict__ scales_out) {
    const int64_t p = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (p >= *n_routed) return;
    const int64_t row = perm[p] / act_div;
    const uint4* src = reinterpret_cast<const uint4*>(act) + row * row_words;
    for (int32_t i = lane_id(); i < row_words; i += 32) act_out[p * row_words + i] = __ldg(src + i);
    for (int32_t i = lane_id(); i < nb; i += 32) scales_out[p * pitch + i] = __ldg(scales + row * nb + i);
}

// ------------------------------------------------------------------- host
namespace {

template <typename TO, bool GATED>
int launch_pair(const CUtensorMap& wmap, const CUtensorMap& xmap, const PairArgs& a, void* out, int grid, cudaStream_t s) {
    using C = Pair;
    const void* k = reinterpret_cast<const void*>(moe_fp8_pair_kernel<TO, GATED>);
    static std::atomic<int> known{0};     // registers of this instantiation: with fewer than LAUNCH_REGS the split of registers would never end
    int regs = known.load(std::memory_order_relaxed);
    if (regs == 0) {
        cudaFuncAttributes at{};
        const cudaError_t e = cudaFuncGetAttributes(&at, k);
        if (e != cudaSuccess) return fail(FT_ERR_CUDA, "cudaFuncGetAttributes: %s", cudaGetErrorString(e));
        known.store(regs = at.numRegs, std::memory_order_relaxed);
    }
    if (regs * C::THREADS < C::drain_regs(GATED) * 256 + C::other_regs(GATED) * 128)
        return fail(FT_ERR_LAUNCH, "moe_fp8_pair_kernel was compiled with %d registers, %d are needed", regs, C::LAUNCH_REGS);
    if (int st = set_smem_limit(k, C::SMEM_BYTES)) return st;
    moe_fp8_pair_kernel<TO, GATED><<<grid, C::THREADS, C::SMEM_BYTES, s>>>(wmap, xmap, a, static_cast<TO*>(out));
    return check_launch("moe_fp8_pair_kernel", dim3(grid), dim3(C::THREADS), C::SMEM_BYTES);
}

}  // namespace

int fp8_tile_width(int64_t n_slots, int32_t n_experts) {
    const double mean = static_cast<double>(n_slots) / n_experts;
    if (n_slots == 1 || mean <= kGemvMean) return 1;
    return mean <= kMean16 ? 16 : mean <= kMean32 ? 32 : kWideTile;
}

size_t fp8_order_layout(uint8_t* base, int64_t n_slots, int32_t n_experts, bool with_pos, Fp8Order* o) {
    size_t at = 0;
    auto take = [&at, base](size_t words) {
        int32_t* p = reinterpret_cast<int32_t*>(base + at);
        at = (at + 4 * words + 255) & ~size_t(255);
        return p;
    };
    const size_t E = static_cast<size_t>(n_experts), S = static_cast<size_t>(n_slots);
    const size_t hist = fp8_route_ok(n_slots, n_experts) ? fp8_route_scratch(n_slots, n_experts) / 4
                                                         : static_cast<size_t>(route_chunks(n_slots)) * E;
    o->offsets = take(E + 1);
    o->tiles = take(E + 1);
    o->perm = take(S);
    o->pos = with_pos ? take(S) : nullptr;
    o->hist = take(hist);
    o->counts = take(E);
    o->err = reinterpret_cast<uint32_t*>(take(1));
    return at;
}

int launch_fp8_order(const int32_t* ids, int64_t n_slots, int32_t n_experts, int tile, const Fp8Order& o, cudaStream_t s) {
    if (fp8_route_ok(n_slots, n_experts))
        return launch_fp8_route(ids, n_slots, n_experts, tile, o.hist, o.offsets, o.tiles, o.perm, o.pos, s);
    RouteBuffers rb{};
    rb.counts = o.counts;
    rb.offsets = o.offsets;
    rb.perm = o.perm;
    rb.hist = o.hist;
    rb.tiles_gemm = o.tiles;
    rb.err = o.err;
    if (int st = launch_route(ids, n_slots, n_experts, rb, tile, tile, nullptr, 0, s)) return st;
    return o.pos ? launch_fp8_invert(o.perm, o.offsets + n_experts, n_slots, o.pos, s) : FT_OK;
}

int launch_fp8_order_rows(Fp8Product* p, uint8_t* codes, float* scales, cudaStream_t s) {
    const int32_t pitch = fp8_scale_pitch(p->ncols), nb = static_cast<int32_t>(fp8_blocks(p->ncols));
    const dim3 grid(static_cast<unsigned>((p->n_slots + 7) / 8));
    order_rows_kernel<<<grid, 256, 0, s>>>(p->act, p->act_scales, p->order->perm, p->order->offsets + p->n_experts, p->act_div,
                                           static_cast<int32_t>(p->ncols / 16), nb, pitch, reinterpret_cast<uint4*>(codes), scales);
    p->act = codes;
    p->act_scales = scales;
    p->act_rows = p->n_slots;
    p->scale_pitch = pitch;
    p->ordered = true;
    return check_launch("order_rows_kernel", grid, dim3(256), 0);
}

int launch_fp8_product(const Fp8Product& p, int width, void* out, int out_dtype, uint32_t* err, cudaStream_t s) {
    using C = Pair;
    if (width == 1) return launch_fp8_gemv(p, out, out_dtype, err, s);
    if (width < 2 * C::BM) return launch_fp8_narrow(p, width, out, out_dtype, err, s);
    PairArgs a{};
    a.act_scales = p.act_scales;
    a.w_scales = p.w_scales;
    a.err = err;
    a.n_slots = p.n_slots;
    a.nrows = p.nrows;
    a.n_experts = p.n_experts;
    a.nb = static_cast<int32_t>(fp8_blocks(p.ncols));
    a.row_blocks = static_cast<int32_t>(fp8_blocks(p.nrows));
    a.row_tiles = static_cast<int32_t>((p.nrows + C::BN - 1) / C::BN);
    a.scale_pitch = p.scale_pitch;
    a.scale_words = p.scale_pitch % 4 == 0 && reinterpret_cast<uintptr_t>(p.act_scales) % 16 == 0;
    a.wide = p.nrows * (out_dtype == FT_DTYPE_F32 ? 4 : 2) % 16 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0;
    a.mid = p.mid;
    a.mid_scales = p.mid_scales;
    a.n_inter = static_cast<int32_t>(p.nrows / 2);
    a.mid_pitch = p.mid_pitch;
    a.act_kind = p.act_kind;
    if (p.ids) {
        a.ids = p.ids;
        a.perm = p.order->perm;
        a.offsets = p.order->offsets;
        a.tiles = p.order->tiles;
    }
    CUtensorMap wmap, xmap;
    if (int st = encode_2d(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.weights, p.ncols,
                           static_cast<uint64_t>(p.n_experts) * p.nrows, p.ncols, kFp8Block, C::BOX,
                           CU_TENSOR_MAP_SWIZZLE_128B, "FP8 weights"))
        return st;
    if (int st = encode_2d(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.act, p.ncols, p.act_rows, p.ncols, kFp8Block,
                           C::ROW_BOX, CU_TENSOR_MAP_SWIZZLE_128B, "FP8 activations"))
        return st;
    const int64_t slot_tiles = (p.n_slots + 2 * C::BM - 1) / (2 * C::BM) + (p.ids ? (p.n_experts < p.n_slots ? p.n_experts : p.n_slots) : 0);
    const int64_t pairs = slot_tiles * a.row_tiles, most = sm_count() / 2;
    const int grid = 2 * static_cast<int>(pairs < most ? pairs : most);
    if (p.mid) return launch_pair<float, true>(wmap, xmap, a, nullptr, grid, s);
    return out_dtype == FT_DTYPE_F32 ? launch_pair<float, false>(wmap, xmap, a, out, grid, s)
                                     : launch_pair<__nv_bfloat16, false>(wmap, xmap, a, out, grid, s);
}

}  // namespace ft
