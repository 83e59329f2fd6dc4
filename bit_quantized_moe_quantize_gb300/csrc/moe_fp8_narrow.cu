// The FP8 products for few slots per expert: what bounds them is
// reading the experts' matrices once.
//
// One tile: up to 128 weight rows of an expert x up to NW of its slots (16 or 32), one CTA,
// tcgen05 MMAs with M = 128 weight rows and N = the tile's slots rounded up to 16.  Here the
// weight rows lie along the tensor-memory lanes: with few slots the scales of a block are few,
// and a warp reads them from shared memory at a broadcast for its 32 rows.  Tiles of 128 rows also
// where a batch has too few of them to fill the GPU: of 64 or 32 rows, which it has more of, 21
// batches of 1 to 128 experts and 2 to 300 slots took up to 1.5 times as long (300 slots, 1024 x
// 4096 of 8: 39 us against 27; 16 slots, 1408 x 2816 of 8: 27.6 / 21.5) and none took less by more than 3 %.
//
// Blocks go through tensor memory in units of 64 columns (two blocks of 32 slots or four of 16),
// so that the drain waits once per unit and the MMAs of four units run ahead of it.  Two CTAs
// share an SM, so that one streams while the other starts or ends.
//
// Measured, 1536 x 2048 of 128 experts with cold caches: 64 tokens of 8 slots 85 us, 512 tokens
// 99 us (403 MB: 59 us at the copy's rate).  Where experts have more than 32 slots, what is left
// over the matrices' one reading is their next ones, from L2: 509 uneven tokens, 4 slots each,
// 1414 x 2000 of 60 experts: 56 us with the order, 45 without, for 170 MB (25 us).
//
// Up to 1024 slots are put in order by every CTA for itself, in shared memory (some 2 us
// less than a launch and the reads of its results); more come ordered.
//
// Per CTA: warps 0-3 drain (32 weight rows each), warp 4 TMA producer of the weight rows,
// warp 5 MMA, warp 6 scales (sa * sw of a unit's blocks and slots to a ring in shared memory),
// warp 7 copies the slots' rows and zeroes the rows of slots without an expert.
//
// The slots' rows lie anywhere, and are copied by cp.async, 16 bytes a lane, into the place that
// the 128-byte swizzle gives them.  A TMA gather fetches four rows and takes the unit about 85
// cycles: 32 slots in each of two CTAs kept it busy for most of a block's time.
#include "fp8_order.cuh"
#include "fp8_tc.cuh"
#include "ft_internal.h"
#include "gemm_common.cuh"

namespace ft {

template <int NW_>
struct Narrow {
    static constexpr int NW = NW_;
    static constexpr int BM = 128;                                  // lanes: weight rows of a tile
    static constexpr int G = 64 / NW;                               // blocks per unit
    static constexpr int UNIT = G * NW;                             // columns of a unit
    static constexpr int TMEM_COLS = 256;                           // two CTAs per SM
    static constexpr int UNITS = TMEM_COLS / UNIT;
    static constexpr int NSC = 4;                                   // units in the scale ring
    // a stage: NW slots' rows, then the weight rows
    static constexpr int STAGES = 4;
    static constexpr int ROW_BYTES = NW * kFp8Block, STAGE_BYTES = ROW_BYTES + BM * kFp8Block;
    static constexpr int OFF_SC = STAGES * STAGE_BYTES;
    static constexpr int OFF_BAR = OFF_SC + NSC * UNIT * 4;
    static constexpr int N_BARS = 2 * STAGES + 2 * UNITS + 2 * NSC;
    static constexpr int OFF_TMEM = OFF_BAR + N_BARS * 8;
    // in-CTA order: offsets[E + 1], tiles[E + 1], perm[1024]; the counts [8][E] lie in the ring
    static constexpr int MAX_E = 1024;
    static constexpr int OFF_ORDER = OFF_TMEM + 16;
    static constexpr int SMEM_BYTES = OFF_ORDER + (2 * (MAX_E + 1) + 1024 + 8) * 4 + 1024;
    static_assert(kChunkWarps * MAX_E * 4 <= OFF_SC, "counts");
    static constexpr int WARP_PRODUCER = 4, WARP_MMA = 5, WARP_SCALE = 6, WARP_ROWS = 7;
    static constexpr int THREADS = 256, N_DRAIN_WARPS = BM / 32;
    static_assert(2 * (SMEM_BYTES + 1024) <= 233472, "shared memory budget of two CTAs");
};

struct NarrowArgs {
    const int32_t* ids;
    const int32_t* perm;
    const int32_t* offsets;
    const int32_t* tiles;        // prefix of tiles of NW slots
    const uint8_t* act;
    const float* act_scales;
    const float* w_scales;
    uint32_t* err;
    int64_t n_slots, nrows, ncols;
    int32_t act_div, n_experts, nb, row_tiles, row_blocks, scale_pitch;
    bool ordered;                // activation rows lie in router order
    bool orders;                 // perm, offsets and tiles are worked out by the CTA
};

struct NarrowTile {
    int32_t e, p0, n, r0;        // expert, first position, slots, first weight row
};

template <int NW>
__device__ __forceinline__ NarrowTile narrow_tile(const NarrowArgs& a, const int32_t* tiles, const int32_t* offsets, int64_t w) {
    NarrowTile t;
    const int32_t st = static_cast<int32_t>(w / a.row_tiles);
    t.r0 = static_cast<int32_t>(w - static_cast<int64_t>(st) * a.row_tiles) * Narrow<NW>::BM;
    int32_t first = 0, count = static_cast<int32_t>(a.n_slots), j = st;
    t.e = 0;
    if (tiles) {
        t.e = last_not_above(tiles, a.n_experts, st);
        first = offsets[t.e];
        count = offsets[t.e + 1] - first;
        j = st - tiles[t.e];
    }
    t.p0 = first + j * NW;
    t.n = min(NW, count - j * NW);
    return t;
}

template <int NW, typename TO>
__global__ void __launch_bounds__(Narrow<NW>::THREADS, 2)
    moe_fp8_narrow_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ NarrowArgs a, TO* __restrict__ out) {
    using C = Narrow<NW>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* empty = full + C::STAGES;
    uint64_t* acc_full = empty + C::STAGES;
    uint64_t* acc_empty = acc_full + C::UNITS;
    uint64_t* sc_full = acc_empty + C::UNITS;
    uint64_t* sc_empty = sc_full + C::NSC;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_TMEM);
    float* sc_ring = reinterpret_cast<float*>(smem + C::OFF_SC);

    const uint32_t warp = threadIdx.x >> 5, lane = lane_id();
    const int32_t nb = a.nb;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&full[i], 1 + 32);      // the producer and the lanes that copy rows
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < C::UNITS; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], C::N_DRAIN_WARPS);
        }
        for (int i = 0; i < C::NSC; ++i) {
            mbar_init(&sc_full[i], 1);
            mbar_init(&sc_empty[i], C::N_DRAIN_WARPS);
        }
        fence_mbar_init();
    }
    if (warp == C::WARP_MMA) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    if (warp == C::WARP_PRODUCER && lane == 0) prefetch_tmap(&wmap);
    const int32_t *offsets = a.offsets, *tiles = a.tiles, *perm = a.perm;
    if (a.orders) {
        int32_t* o = reinterpret_cast<int32_t*>(smem + C::OFF_ORDER);
        int32_t *nt = o + C::MAX_E + 1, *pm = nt + C::MAX_E + 1, *part = pm + 1024;
        int32_t* mine = reinterpret_cast<int32_t*>(smem);
        const int32_t E = a.n_experts, n_slots = static_cast<int32_t>(a.n_slots);
        int32_t id[4], rank[4];
        const int32_t s0 = chunk_rank(a.ids, 0, n_slots, E, mine, id, rank);
        chunk_totals(mine, E, o);
        for (int32_t e = threadIdx.x; e < E; e += kChunkThreads) nt[e] = (o[e] + NW - 1) / NW;
        __syncthreads();
        const int32_t routed = chunk_scan(o, E, part), n_tiles = chunk_scan(nt, E, part);
        if (threadIdx.x == 0) {
            o[E] = routed;
            nt[E] = n_tiles;
        }
        chunk_starts(mine, E, o);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (id[i] >= 0) pm[mine[static_cast<int32_t>(warp) * E + id[i]] + rank[i]] = s0 + 32 * i;
        fence_proxy_async_smem();      // the copies that follow write where the counts lay
        perm = pm;
        offsets = o;
        tiles = nt;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const int64_t slot_tiles = tiles ? tiles[a.n_experts] : (a.n_slots + NW - 1) / NW;
    const int64_t total = slot_tiles * a.row_tiles;

    if (warp == C::WARP_PRODUCER) {
        // ------------------------------------------------------------ producer
        uint32_t s = 0, phase = 1, it = 0;
        bool ok = true;
        for (int64_t w = blockIdx.x; w < total && ok; w += gridDim.x) {
            const NarrowTile t = narrow_tile<NW>(a, tiles, offsets, w);
            const int32_t wy = static_cast<int32_t>(static_cast<int64_t>(t.e) * a.nrows + t.r0);
            for (int32_t b = 0; b < nb; ++b, ++it) {
                if (!mbar_wait_warp(&empty[s], phase, a.err)) { ok = false; break; }
                if (lane == 0) {
                    mbar_arrive_expect_tx(&full[s], C::STAGE_BYTES - C::ROW_BYTES);
                    tma_load_2d(smem + s * C::STAGE_BYTES + C::ROW_BYTES, &wmap, b * kFp8Block, wy, &full[s]);
                }
                __syncwarp();
                if (++s == C::STAGES) {
                    s = 0;
                    phase ^= 1u;
                }
            }
        }
        // the last fills: read by their MMAs, or at least arrived, before the CTA's memory goes
        for (uint32_t f = it - min(it, static_cast<uint32_t>(C::STAGES)); f != it; ++f) {
            const uint32_t last = f % C::STAGES, parity = (f / C::STAGES) & 1u;
            if (mbar_wait_warp(&empty[last], parity, a.err, ok ? kWaitLimitNs : kLastWaitNs)) continue;
            ok = false;
            mbar_wait_warp(&full[last], parity, a.err, kLastWaitNs);
        }
    } else if (warp == C::WARP_MMA) {
        // ----------------------------------------------------------------- MMA
        const bool elected = elect_one();
        const uint64_t desc0 = smem_desc_sw128(smem_u32(smem));
        uint32_t s = 0, phase = 0, unit = 0;
        bool ok = true;
        for (int64_t w = blockIdx.x; w < total && ok; w += gridDim.x) {
            const NarrowTile t = narrow_tile<NW>(a, tiles, offsets, w);
            const uint32_t idesc = idesc_e4m3_f32(C::BM, (t.n + 15) / 16 * 16);
            for (int32_t b0 = 0; b0 < nb && ok; b0 += C::G, ++unit) {
                const uint32_t u = unit % C::UNITS;
                if (!mbar_wait_warp(&acc_empty[u], ((unit / C::UNITS) & 1u) ^ 1u, a.err)) { ok = false; break; }
                const int32_t n = min(C::G, nb - b0);
                for (int32_t g = 0; g < n; ++g) {
                    if (!mbar_wait_warp(&full[s], phase, a.err)) { ok = false; break; }
                    fence_proxy_async_smem();      // the copied rows are ordinary writes
                    tc_fence_after();
                    if (elected) {
                        const uint64_t bdesc = desc0 + ((s * C::STAGE_BYTES) >> 4), adesc = bdesc + (C::ROW_BYTES >> 4);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            tc_mma_f8(tmem + u * C::UNIT + static_cast<uint32_t>(g) * NW, adesc + 2 * k, bdesc + 2 * k, idesc, k);
                        tc_commit(&empty[s]);
                        if (g == n - 1) tc_commit(&acc_full[u]);
                    }
                    if (++s == C::STAGES) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == C::WARP_SCALE) {
        // -------------------------------------------------------------- scales
        uint32_t unit = 0;
        bool ok = true;
        for (int64_t w = blockIdx.x; w < total && ok; w += gridDim.x) {
            const NarrowTile t = narrow_tile<NW>(a, tiles, offsets, w);
            const float* sa = nullptr;                   // of slot `lane`
            if (static_cast<int32_t>(lane) < t.n) {
                const int32_t p = t.p0 + static_cast<int32_t>(lane);
                sa = a.act_scales + static_cast<int64_t>(a.ordered ? p : perm[p] / a.act_div) * a.scale_pitch;
            }
            const float* sw = a.w_scales + (static_cast<int64_t>(t.e) * a.row_blocks + t.r0 / kFp8Block) * nb;
            // a load takes longer than a unit: those of four units are in flight
            constexpr int AHEAD = 4;
            float v[AHEAD][C::G], x[AHEAD][C::G];
            auto load = [&](int q, int32_t b0) {
#pragma unroll
                for (int g = 0; g < C::G; ++g) {
                    x[q][g] = b0 + g < nb ? __ldg(sw + b0 + g) : 0.0f;
                    v[q][g] = sa && b0 + g < nb ? __ldg(sa + b0 + g) : 0.0f;
                }
            };
#pragma unroll
            for (int q = 0; q < AHEAD; ++q) load(q, q * C::G);
            for (int32_t b0 = 0; b0 < nb && ok; b0 += AHEAD * C::G) {
#pragma unroll
                for (int q = 0; q < AHEAD; ++q) {
                    if (b0 + q * C::G < nb && ok) {
                        const uint32_t r = unit % C::NSC;
                        if (!mbar_wait_warp(&sc_empty[r], ((unit / C::NSC) & 1u) ^ 1u, a.err)) {
                            ok = false;
                        } else {
#pragma unroll
                            for (int g = 0; g < C::G; ++g)
                                if (lane < static_cast<uint32_t>(NW)) sc_ring[r * C::UNIT + g * NW + lane] = v[q][g] * x[q][g];
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&sc_full[r]);
                            ++unit;
                            load(q, b0 + (q + AHEAD) * C::G);
                        }
                    }
                }
            }
        }
    } else if (warp < C::N_DRAIN_WARPS) {
        // --------------------------------------------------------------- drain
        uint32_t unit = 0;
        bool ok = true;
        for (int64_t w = blockIdx.x; w < total && ok; w += gridDim.x) {
            const NarrowTile t = narrow_tile<NW>(a, tiles, offsets, w);
            float acc[NW];
#pragma unroll
            for (int i = 0; i < NW; ++i) acc[i] = 0.0f;
            const int32_t pl = t.p0 + min(static_cast<int32_t>(lane), t.n - 1), slot_of = perm ? perm[pl] : pl;      // of slot `lane`
            for (int32_t b0 = 0; b0 < nb; b0 += C::G, ++unit) {
                const uint32_t u = unit % C::UNITS, r = unit % C::NSC;
                if (!mbar_wait2_warp(&sc_full[r], (unit / C::NSC) & 1u, &acc_full[u], (unit / C::UNITS) & 1u, a.err)) { ok = false; break; }
                tc_fence_after();
                const float4* sc = reinterpret_cast<const float4*>(sc_ring + r * C::UNIT);
#pragma unroll
                for (int j = 0; j < C::UNIT / 16; ++j) {      // 16 columns: slots 16 j % NW .. of block 16 j / NW
                    if (b0 + 16 * j / NW < nb && 16 * j % NW < t.n) {
                        uint32_t v[16];
                        tmem_ld_32x32b_x16(tmem + u * C::UNIT + ((warp * 32u) << 16) + 16 * j, v);
                        float4 c[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) c[i] = sc[4 * j + i];
                        tmem_wait_ld_regs(v);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float* o = acc + 16 * j % NW + 4 * i;
                            o[0] = fmaf(__uint_as_float(v[4 * i]), c[i].x, o[0]);
                            o[1] = fmaf(__uint_as_float(v[4 * i + 1]), c[i].y, o[1]);
                            o[2] = fmaf(__uint_as_float(v[4 * i + 2]), c[i].z, o[2]);
                            o[3] = fmaf(__uint_as_float(v[4 * i + 3]), c[i].w, o[3]);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&acc_empty[u]);
                    mbar_arrive(&sc_empty[r]);
                }
            }
            if (!ok) break;
            const int32_t row = t.r0 + static_cast<int32_t>(threadIdx.x);
#pragma unroll
            for (int c = 0; c < NW; ++c) {
                if (c < t.n) {
                    const int32_t slot = __shfl_sync(0xFFFFFFFFu, slot_of, c);
                    if (row < a.nrows) out[static_cast<int64_t>(slot) * a.nrows + row] = from_f32<TO>(acc[c]);
                }
            }
        }
    } else if (warp == C::WARP_ROWS) {
        // ---------------------------------------------------------------- rows
        // lane: 16-byte word `word` of rows first, first + 4, ..
        const uint32_t word = lane & 7u, first = lane >> 3;
        uint32_t s = 0, phase = 1;
        bool ok = true;
        for (int64_t w = blockIdx.x; w < total && ok; w += gridDim.x) {
            const NarrowTile t = narrow_tile<NW>(a, tiles, offsets, w);
            const uint8_t* src[NW / 4];
#pragma unroll
            for (int i = 0; i < NW / 4; ++i) {
                const int32_t p = t.p0 + min(static_cast<int32_t>(first) + 4 * i, t.n - 1);
                src[i] = a.act + static_cast<int64_t>(a.ordered ? p : perm[p] / a.act_div) * a.ncols + 16 * word;
            }
            int64_t left = a.ncols - 16 * word;      // columns from this lane's word to the rows' end
            for (int32_t b = 0; b < nb; ++b, left -= kFp8Block) {
                if (!mbar_wait_warp(&empty[s], phase, a.err)) { ok = false; break; }
                const uint32_t dst = smem_u32(smem + s * C::STAGE_BYTES);
#pragma unroll
                for (int i = 0; i < NW / 4; ++i) {
                    const uint32_t r = first + 4 * i;
                    if (static_cast<int32_t>(r) < t.n)      // (words past the rows' end arrive as 0)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + r * kFp8Block + ((word ^ (r & 7u)) << 4)),
                                     "l"(left > 0 ? src[i] : a.act), "r"(left > 0 ? 16 : 0)
                                     : "memory");
                    src[i] += kFp8Block;
                }
                // arrives when this lane's copies have
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&full[s])) : "memory");
                if (++s == C::STAGES) {
                    s = 0;
                    phase ^= 1u;
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (a.ids) zero_unrouted<TO>(a.ids, a.n_slots, a.n_experts, a.nrows, a.err, out, blockIdx.x, gridDim.x);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == C::WARP_MMA) tmem_dealloc(tmem, C::TMEM_COLS);
}

// ------------------------------------------------------------------- host
namespace {

template <int NW, typename TO>
int launch_narrow(const CUtensorMap& wmap, const NarrowArgs& a, void* out, int64_t tiles, cudaStream_t s) {
    using C = Narrow<NW>;
    const void* k = reinterpret_cast<const void*>(moe_fp8_narrow_kernel<NW, TO>);
    if (int st = set_smem_limit(k, C::SMEM_BYTES)) return st;
    const int64_t ctas = 2 * sm_count();
    const dim3 grid(static_cast<unsigned>(tiles < ctas ? tiles : ctas));
    moe_fp8_narrow_kernel<NW, TO><<<grid, C::THREADS, C::SMEM_BYTES, s>>>(wmap, a, static_cast<TO*>(out));
    return check_launch("moe_fp8_narrow_kernel", grid, dim3(C::THREADS), C::SMEM_BYTES);
}

}  // namespace

// (us, ordered by the product's CTAs / by a launch before it: 512 and 1024 slots of 128 experts,
// 1536 x 2048, 90.1 / 92.3 and 90.6 / 92.5; 1024 of 60, 1414 x 2000, 53.1 / 55.5; 1024 of 512, 512 x 1024,
// 60.8 / 62.7.  One chunk is what the CTAs' arrays hold.)
bool fp8_orders_itself(int64_t n_slots, int32_t n_experts, int width) {
    return width == 1 || (width <= 32 && n_slots <= kChunk && n_experts <= Narrow<16>::MAX_E);
}

// width: slots per tile (16 or 32), that of p.order's tiles
int launch_fp8_narrow(const Fp8Product& p, int width, void* out, int out_dtype, uint32_t* err, cudaStream_t s) {
    NarrowArgs a{};
    a.act = p.act;
    a.act_scales = p.act_scales;
    a.w_scales = p.w_scales;
    a.err = err;
    a.n_slots = p.n_slots;
    a.nrows = p.nrows;
    a.ncols = p.ncols;
    a.act_div = p.act_div;
    a.n_experts = p.n_experts;
    a.nb = static_cast<int32_t>(fp8_blocks(p.ncols));
    a.row_blocks = static_cast<int32_t>(fp8_blocks(p.nrows));
    a.scale_pitch = p.scale_pitch;
    a.ordered = p.ordered || !p.ids;
    if (p.ids) {
        a.ids = p.ids;
        a.orders = fp8_orders_itself(p.n_slots, p.n_experts, width);
        a.perm = p.order->perm;
        a.offsets = p.order->offsets;
        a.tiles = p.order->tiles;
    }
    const int64_t most_tiles = (p.n_slots + width - 1) / width + (p.ids ? (p.n_experts < p.n_slots ? p.n_experts : p.n_slots) : 0);
    a.row_tiles = static_cast<int32_t>((p.nrows + Narrow<16>::BM - 1) / Narrow<16>::BM);
    CUtensorMap wmap;
    if (int st = encode_2d(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.weights, p.ncols,
                           static_cast<uint64_t>(p.n_experts) * p.nrows, p.ncols, kFp8Block, Narrow<16>::BM,
                           CU_TENSOR_MAP_SWIZZLE_128B, "FP8 weights"))
        return st;
    const int64_t tiles = most_tiles * a.row_tiles;
    const bool f32 = out_dtype == FT_DTYPE_F32;
    if (width == 16)
        return f32 ? launch_narrow<16, float>(wmap, a, out, tiles, s) : launch_narrow<16, __nv_bfloat16>(wmap, a, out, tiles, s);
    return f32 ? launch_narrow<32, float>(wmap, a, out, tiles, s) : launch_narrow<32, __nv_bfloat16>(wmap, a, out, tiles, s);
}

}  // namespace ft
