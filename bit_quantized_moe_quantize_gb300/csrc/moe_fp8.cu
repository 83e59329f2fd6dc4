// Routed expert products in 8-bit floating point with a scale per block of 128:
//
//   out[s][r] = sum_b sa[row(s)][b] sw[e][r / 128][b] sum_{i in block b} w[e][r][i] a[row(s)][i]
//
// with e = topk_ids[s] and row(s) = s / act_div (act_div = top_k: one
// activation row per token; 1: one per slot), and the dense product (one
// matrix, slot s = row s).
//
// One tile: 256 weight rows of an expert x up to 256 of its slots, worked by a
// pair of CTAs with 2-CTA tcgen05 MMAs (kind::f8f6f4, M = 256, N = the tile's
// slots rounded up to 32).  Each CTA loads its 128 weight rows and half of the
// slots' rows per block of 128 columns, so an operand byte in shared memory is
// read once for 256 x 256 products.  A block's products are summed by the tensor core in
// fp32 in a tensor-memory accumulator (two of them, 256 columns each, in turn);
// the scales change with the next block, so the drain takes each block's sums
// out of tensor memory and adds them, times sa * sw, to fp32 registers.
//
// Per CTA, warp-specialised:
//   8 drain warps  warp w: TMEM lanes 32 (w % 4) .. + 31, columns 128 (w / 4) .. + 127,
//                  loaded with the 16x256b shape: a thread holds 4 rows x 32
//                  columns, one shared load of four scales serves 16 of them
//   producer       TMA: the 128 x 128-byte weight box, and the slots' rows four
//                  at a time by index (gather), or in boxes of 16 neighbouring
//                  rows where slots lie in order, both with 128-byte swizzle;
//                  columns past the row's end arrive as 0
//   MMA            (leader CTA) four MMAs of 32 columns per block
//   2 scale warps  sa * sw of each block's slots to a ring in shared memory
//
// Slots of an expert are dealt to tiles of nearly equal width, so an expert
// with 257 slots gets two tiles of 160 and 97 rather than 256 and 1.
#include "fp8_tc.cuh"
#include "ft_internal.h"
#include "gemm_common.cuh"

namespace ft {

struct Pair {
    static constexpr int BM = 128;                 // weight rows per CTA
    static constexpr int BN = 256;                 // slots per tile at most
    static constexpr int STAGES = 5;
    static constexpr int A_BYTES = BM * kFp8Block;
    static constexpr int B_BYTES = BN / 2 * kFp8Block;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int N_DRAIN_WARPS = 8;
    static constexpr int WARP_PRODUCER = 8, WARP_MMA = 9, WARP_SCALE = 10, N_SCALE_WARPS = 2;
    static constexpr int THREADS = 12 * 32;
    static constexpr int CW = BN / 2;              // columns per drain warp
    static constexpr int QP = CW / 4 + 4;          // da_index pitch
    static constexpr int SC_FLOATS = 2 * 4 * QP;   // scales of one block
    static constexpr int NSC = 8;                  // scale ring depth (blocks)
    static constexpr int OFF_SC = STAGES * STAGE_BYTES;
    static constexpr int OFF_BAR = OFF_SC + NSC * SC_FLOATS * 4;
    static constexpr int N_BARS = 2 * STAGES + 4 + 2 * NSC;
    static constexpr int OFF_TMEM = OFF_BAR + N_BARS * 8;
    static constexpr int SMEM_BYTES = OFF_TMEM + 16 + 1024;    // + alignment slack
    // registers: 384 threads are launched with LAUNCH_REGS each; the drain warps
    // take DRAIN_REGS and the others give theirs down to OTHER_REGS
    static constexpr int LAUNCH_REGS = 168, DRAIN_REGS = 208, OTHER_REGS = 88;
    static_assert(DRAIN_REGS * 256 + OTHER_REGS * 128 <= LAUNCH_REGS * THREADS, "the split must fit the launch's registers");
    static_assert(SMEM_BYTES <= 232448, "shared memory budget");
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
    int32_t act_div, n_experts, nb, row_tiles, row_blocks;
};

struct PairTile {
    int32_t e, n, width;         // expert, valid slots, MMA width (a multiple of 32)
    int64_t p0, m0;              // first router position, first weight row
};

// Work item w: row tile w % row_tiles of slot tile w / row_tiles.
__device__ __forceinline__ PairTile pair_tile(const PairArgs& a, int64_t w) {
    PairTile t;
    const int64_t st = w / a.row_tiles;
    t.m0 = (w - st * a.row_tiles) * (2 * Pair::BM);
    int64_t first = 0, count = a.n_slots, nt = (a.n_slots + Pair::BN - 1) / Pair::BN, j = st;
    t.e = 0;
    if (a.tiles) {
        int32_t lo = 0, hi = a.n_experts - 1;
        while (lo < hi) {
            const int32_t mid = (lo + hi + 1) >> 1;
            if (a.tiles[mid] <= st) lo = mid;
            else hi = mid - 1;
        }
        t.e = lo;
        first = a.offsets[lo];
        count = a.offsets[lo + 1] - first;
        nt = a.tiles[lo + 1] - a.tiles[lo];
        j = st - a.tiles[lo];
    }
    // nearly equal widths; from 5 tiles on the rounding could leave the last one empty
    const int64_t per = nt > 4 ? Pair::BN : ((count + nt - 1) / nt + 31) / 32 * 32;
    t.p0 = first + j * per;
    t.n = static_cast<int32_t>(min(per, count - j * per));
    t.width = (t.n + 31) / 32 * 32;
    return t;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(r)
        : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)),
          "l"(*reinterpret_cast<uint64_t*>(&c)));
    return *reinterpret_cast<float2*>(&r);
}

// Rows of slots without an expert are 0; ids that are neither -1 nor an expert raise the flag.
template <typename TO>
__device__ __forceinline__ void zero_unrouted(const PairArgs& a, TO* out, int64_t warp, int64_t n_warps) {
    for (int64_t s0 = warp * 32; s0 < a.n_slots; s0 += n_warps * 32) {
        const int64_t s = s0 + lane_id();
        const int32_t id = s < a.n_slots ? a.ids[s] : 0;
        const bool none = id < 0 || id >= a.n_experts;
        if (none && id != -1) atomicOr(a.err, FT_DEVERR_BAD_EXPERT_ID);
        uint32_t left = __ballot_sync(0xFFFFFFFFu, none);
        while (left) {
            const int64_t row = s0 + __ffs(left) - 1;
            left &= left - 1;
            for (int64_t r = lane_id(); r < a.nrows; r += 32) out[row * a.nrows + r] = from_f32<TO>(0.0f);
        }
    }
}

template <typename TO, bool GATHER>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Pair::THREADS, 1)
    moe_fp8_pair_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                        const PairArgs a, TO* __restrict__ out) {
    using C = Pair;
    extern __shared__ uint8_t smem_raw[];
    // both CTAs round up by the same amount: their dynamic shared memory starts at the same offset
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* empty = full + C::STAGES;
    uint64_t* acc_full = empty + C::STAGES;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* sc_full = acc_empty + 2;
    uint64_t* sc_empty = sc_full + C::NSC;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_TMEM);
    float* sc_ring = reinterpret_cast<float*>(smem + C::OFF_SC);

    const uint32_t warp = threadIdx.x >> 5, lane = lane_id(), rank = cluster_ctarank();
    const int32_t nb = a.nb;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 2 * C::N_DRAIN_WARPS);     // the leader's: drain warps of both CTAs
        }
        for (int i = 0; i < C::NSC; ++i) {
            mbar_init(&sc_full[i], C::N_SCALE_WARPS);
            mbar_init(&sc_empty[i], C::N_DRAIN_WARPS);
        }
        fence_mbar_init();
    }
    if (warp == C::WARP_MMA) tmem_alloc_pair(tmem_slot, 512);
    if (warp == C::WARP_PRODUCER && lane == 0) {
        prefetch_tmap(&wmap);
        prefetch_tmap(&xmap);
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const int64_t slot_tiles = a.tiles ? a.tiles[a.n_experts] : (a.n_slots + C::BN - 1) / C::BN;
    const int64_t total = slot_tiles * a.row_tiles;
    const int64_t w0 = blockIdx.x / 2, dw = gridDim.x / 2;

    if (warp >= C::N_DRAIN_WARPS) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::OTHER_REGS));
        if (warp == C::WARP_PRODUCER) {
            // -------------------------------------------------------- producer
            uint32_t it = 0;
            bool ok = true;
            for (int64_t w = w0; w < total && ok; w += dw) {
                const PairTile t = pair_tile(a, w);
                const int32_t half = t.width / 2;
                const int64_t wy = static_cast<int64_t>(t.e) * a.nrows + t.m0 + rank * C::BM;
                // this CTA's slots: positions p0 + rank * half ..; lane l copies 4 (gather) or 16 of them
                const int32_t mine = max(0, min(half, t.n - static_cast<int32_t>(rank) * half));
                const int32_t other = max(0, min(half, t.n - static_cast<int32_t>(1 - rank) * half));
                constexpr int PER = GATHER ? 4 : 16;
                const bool copies = static_cast<int32_t>(lane) * PER < mine;
                int32_t y[4] = {0, 0, 0, 0};
                if (copies) {
                    const int64_t p = t.p0 + rank * half + lane * PER;
                    if constexpr (GATHER) {
                        const int64_t last = t.p0 + t.n - 1;      // the last rows of a part group repeat it
#pragma unroll
                        for (int i = 0; i < 4; ++i) y[i] = a.perm[min(p + i, last)] / a.act_div;
                    } else {
                        y[0] = static_cast<int32_t>(p);
                    }
                }
                const uint32_t bytes = 2 * C::A_BYTES + ((mine + PER - 1) / PER + (other + PER - 1) / PER) * PER * kFp8Block;
                for (int32_t b = 0; b < nb; ++b, ++it) {
                    const uint32_t s = it % C::STAGES;
                    if (!mbar_wait_warp(&empty[s], ((it / C::STAGES) & 1u) ^ 1u, a.err)) { ok = false; break; }
                    const uint32_t bar = map_to_rank(smem_u32(&full[s]), 0);
                    const uint32_t dst = smem_u32(smem + s * C::STAGE_BYTES);
                    if (lane == 0) {
                        if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
                        tma_load_2d_pair(dst, &wmap, b * kFp8Block, static_cast<int32_t>(wy), bar);
                    }
                    if (copies) {
                        const uint32_t d = dst + C::A_BYTES + lane * (PER * kFp8Block);
                        if constexpr (GATHER) tma_gather4_pair(d, &xmap, b * kFp8Block, y, bar);
                        else tma_load_2d_pair(d, &xmap, b * kFp8Block, y[0], bar);
                    }
                    __syncwarp();
                }
            }
        } else if (warp == C::WARP_MMA) {
            // ------------------------------------------------------------- MMA
            if (rank == 0 && lane == 0) {
                uint32_t it = 0;
                bool ok = true;
                for (int64_t w = w0; w < total && ok; w += dw) {
                    const PairTile t = pair_tile(a, w);
                    const uint32_t idesc = idesc_e4m3_f32(2 * C::BM, t.width);
                    for (int32_t b = 0; b < nb; ++b, ++it) {
                        const uint32_t s = it % C::STAGES, d = it & 1u;
                        if (!mbar_wait_cluster(&acc_empty[d], ((it >> 1) & 1u) ^ 1u, a.err)) { ok = false; break; }
                        if (!mbar_wait_cluster(&full[s], (it / C::STAGES) & 1u, a.err)) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t abase = smem_u32(smem + s * C::STAGE_BYTES), bbase = abase + C::A_BYTES;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            tc_mma_f8_pair(tmem + d * C::BN, smem_desc_sw128(abase + 32 * k),
                                           smem_desc_sw128(bbase + 32 * k), idesc, k);
                        tc_commit_pair(&empty[s]);
                        tc_commit_pair(&acc_full[d]);
                    }
                }
            }
            __syncwarp();
        } else {
            // ---------------------------------------------------------- scales
            constexpr int PER = C::BN / (32 * C::N_SCALE_WARPS);        // slots per thread
            const uint32_t u = (warp - C::WARP_SCALE) * 32 + lane;
            uint32_t it = 0;
            bool ok = true;
            for (int64_t w = w0; w < total && ok; w += dw) {
                const PairTile t = pair_tile(a, w);
                const float* sa[PER];
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int32_t c = static_cast<int32_t>(u) + i * 32 * C::N_SCALE_WARPS;
                    int64_t row = -1;
                    if (c < t.n) {
                        row = t.p0 + c;
                        if (a.perm) row = a.perm[row] / a.act_div;
                    }
                    sa[i] = row < 0 ? nullptr : a.act_scales + row * nb;
                }
                const int64_t rb = t.m0 / kFp8Block + rank;
                const float* sw = a.w_scales + (static_cast<int64_t>(t.e) * a.row_blocks + min(rb, static_cast<int64_t>(a.row_blocks - 1))) * nb;
                for (int32_t b0 = 0; b0 < nb && ok; b0 += 4) {
                    const int32_t n = min(4, nb - b0);
                    float v[PER][4], g[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        g[j] = j < n ? __ldg(sw + b0 + j) : 0.0f;
#pragma unroll
                        for (int i = 0; i < PER; ++i) v[i][j] = j < n && sa[i] ? __ldg(sa[i] + b0 + j) : 0.0f;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (j < n && ok) {
                            const uint32_t r = it % C::NSC;
                            if (!mbar_wait_warp(&sc_empty[r], ((it / C::NSC) & 1u) ^ 1u, a.err)) ok = false;
                            if (ok) {
                                float* ring = sc_ring + r * C::SC_FLOATS;
#pragma unroll
                                for (int i = 0; i < PER; ++i)
                                    ring[da_index<C::CW>(u + i * 32 * C::N_SCALE_WARPS)] = v[i][j] * g[j];
                                __syncwarp();
                                if (lane == 0) mbar_arrive(&sc_full[r]);
                                ++it;
                            }
                        }
                    }
                }
            }
        }
    } else {
        // --------------------------------------------------------------- drain
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::DRAIN_REGS));
        if (a.ids) zero_unrouted<TO>(a, out, static_cast<int64_t>(blockIdx.x) * C::N_DRAIN_WARPS + warp,
                                     static_cast<int64_t>(gridDim.x) * C::N_DRAIN_WARPS);
        const uint32_t lane0 = (warp & 3u) * 32u, col0 = (warp >> 2) * static_cast<uint32_t>(C::CW), q = lane & 3u;
        const uint32_t acc_empty0 = map_to_rank(smem_u32(acc_empty), 0);
        uint32_t it = 0;
        bool ok = true;
        for (int64_t w = w0; w < total && ok; w += dw) {
            const PairTile t = pair_tile(a, w);
            float2 acc[2][2][16];        // [16-lane half][row, row + 8][column pair]
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[h][r][i] = make_float2(0.0f, 0.0f);
            for (int32_t b = 0; b < nb; ++b, ++it) {
                const uint32_t d = it & 1u, r = it % C::NSC;
                if (!mbar_wait_warp(&sc_full[r], (it / C::NSC) & 1u, a.err)) { ok = false; break; }
                if (!mbar_wait_warp(&acc_full[d], (it >> 1) & 1u, a.err)) { ok = false; break; }
                tc_fence_after();
                const float4* sc = reinterpret_cast<const float4*>(sc_ring + r * C::SC_FLOATS + (col0 / C::CW) * 4 * C::QP + q * C::QP);
#pragma unroll
                for (int ch = 0; ch < 2; ++ch) {
                    if (static_cast<int32_t>(col0) + 64 * ch < t.width) {
                        float4 c[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) c[i] = sc[4 * ch + i];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t v[32];
                            tmem_ld_16x256b_x8(tmem + d * C::BN + ((lane0 + 16 * h) << 16) + col0 + 64 * ch, v);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float2 s2 = (i & 1) ? make_float2(c[i >> 1].z, c[i >> 1].w) : make_float2(c[i >> 1].x, c[i >> 1].y);
#pragma unroll
                                for (int rr = 0; rr < 2; ++rr)
                                    acc[h][rr][8 * ch + i] =
                                        fma2(make_float2(__uint_as_float(v[4 * i + 2 * rr]), __uint_as_float(v[4 * i + 2 * rr + 1])),
                                             s2, acc[h][rr][8 * ch + i]);
                            }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive_remote(acc_empty0 + d * 8);
                    mbar_arrive(&sc_empty[r]);
                }
            }
            if (!ok) break;
            // rows m0 + 128 rank + lane0 + 16 h + 8 rr + lane / 4, slots p0 + col0 + 8 i + 2 q + e
            const int64_t row0 = t.m0 + rank * C::BM + lane0 + (lane >> 2);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int32_t n = static_cast<int32_t>(col0) + 8 * i + 2 * static_cast<int32_t>(q) + e;
                    if (n < t.n) {
                        const int64_t p = t.p0 + n, slot = a.perm ? a.perm[p] : p;
                        TO* o = out + slot * a.nrows;
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int rr = 0; rr < 2; ++rr) {
                                const int64_t row = row0 + 16 * h + 8 * rr;
                                if (row < a.nrows) o[row] = from_f32<TO>(e ? acc[h][rr][i].y : acc[h][rr][i].x);
                            }
                    }
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync_all();      // the peer's arrivals and operand reads are over
    if (warp == C::WARP_MMA) tmem_dealloc_pair(tmem, 512);
}

// ------------------------------------------------------------------- host
namespace {

struct ProductWs {
    size_t counts, offsets, perm, tiles, hist, err, total;
};

ProductWs product_ws(int64_t n_slots, int32_t n_experts) {
    ProductWs L{};
    size_t o = 0;
    auto take = [&o](size_t bytes) {
        const size_t at = o;
        o = (o + bytes + 255) & ~size_t(255);
        return at;
    };
    const size_t E = static_cast<size_t>(n_experts), S = static_cast<size_t>(n_slots);
    L.counts = take(4 * E);
    L.offsets = take(4 * (E + 1));
    L.perm = take(4 * S);
    L.tiles = take(4 * (E + 1));
    L.hist = take(4 * static_cast<size_t>(route_chunks(n_slots)) * E);
    L.err = take(4);       // the router's own flags: ids of -1 are no error here
    L.total = o;
    return L;
}

template <typename TO, bool GATHER>
int launch_pair(const CUtensorMap& wmap, const CUtensorMap& xmap, const PairArgs& a, TO* out, int grid, cudaStream_t s) {
    using C = Pair;
    const void* k = reinterpret_cast<const void*>(moe_fp8_pair_kernel<TO, GATHER>);
    static int regs = 0;     // of this instantiation; the split of registers must fit what it launches with
    if (regs == 0) {
        cudaFuncAttributes at{};
        const cudaError_t e = cudaFuncGetAttributes(&at, k);
        if (e != cudaSuccess) return fail(FT_ERR_CUDA, "cudaFuncGetAttributes: %s", cudaGetErrorString(e));
        regs = at.numRegs;
    }
    if (regs * C::THREADS < C::DRAIN_REGS * 256 + C::OTHER_REGS * 128)
        return fail(FT_ERR_LAUNCH, "moe_fp8_pair_kernel was compiled with %d registers, %d are needed", regs, C::LAUNCH_REGS);
    if (int st = set_smem_limit(k, C::SMEM_BYTES)) return st;
    moe_fp8_pair_kernel<TO, GATHER><<<grid, C::THREADS, C::SMEM_BYTES, s>>>(wmap, xmap, a, out);
    return check_launch("moe_fp8_pair_kernel", dim3(grid), dim3(C::THREADS), C::SMEM_BYTES);
}

}  // namespace

size_t fp8_product_workspace(int64_t n_slots, int32_t n_experts) { return product_ws(n_slots, n_experts).total; }

int launch_fp8_product(const Fp8Product& p, void* out, int out_dtype, void* workspace, uint32_t* err, cudaStream_t s) {
    using C = Pair;
    const ProductWs L = product_ws(p.n_slots, p.n_experts);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    PairArgs a{};
    a.act_scales = p.act_scales;
    a.w_scales = p.w_scales;
    a.err = err;
    a.n_slots = p.n_slots;
    a.nrows = p.nrows;
    a.act_div = p.act_div;
    a.n_experts = p.n_experts;
    a.nb = static_cast<int32_t>(fp8_blocks(p.ncols));
    a.row_blocks = static_cast<int32_t>(fp8_blocks(p.nrows));
    a.row_tiles = static_cast<int32_t>((p.nrows + 2 * C::BM - 1) / (2 * C::BM));
    if (p.ids) {
        RouteBuffers rb{};
        rb.counts = reinterpret_cast<int32_t*>(ws + L.counts);
        rb.offsets = reinterpret_cast<int32_t*>(ws + L.offsets);
        rb.perm = reinterpret_cast<int32_t*>(ws + L.perm);
        rb.hist = reinterpret_cast<int32_t*>(ws + L.hist);
        rb.tiles_gemm = reinterpret_cast<int32_t*>(ws + L.tiles);
        rb.err = reinterpret_cast<uint32_t*>(ws + L.err);
        if (int st = launch_route(p.ids, p.n_slots, p.n_experts, rb, C::BN, C::BN, nullptr, 0, s)) return st;
        a.ids = p.ids;
        a.perm = rb.perm;
        a.offsets = rb.offsets;
        a.tiles = rb.tiles_gemm;
    }
    CUtensorMap wmap, xmap;
    if (int st = encode_2d(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.weights, p.ncols,
                           static_cast<uint64_t>(p.n_experts) * p.nrows, p.ncols, kFp8Block, C::BM,
                           CU_TENSOR_MAP_SWIZZLE_128B, "FP8 weights"))
        return st;
    if (int st = encode_2d(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.act, p.ncols, p.act_rows, p.ncols, kFp8Block,
                           p.ids ? 1 : 16, CU_TENSOR_MAP_SWIZZLE_128B, "FP8 activations"))
        return st;
    const int64_t slot_tiles = (p.n_slots + C::BN - 1) / C::BN + (p.ids ? (p.n_experts < p.n_slots ? p.n_experts : p.n_slots) : 0);
    const int64_t pairs = slot_tiles * a.row_tiles, most = sm_count() / 2;
    const int grid = 2 * static_cast<int>(pairs < most ? pairs : most);
    if (out_dtype == FT_DTYPE_F32) {
        float* o = static_cast<float*>(out);
        return p.ids ? launch_pair<float, true>(wmap, xmap, a, o, grid, s) : launch_pair<float, false>(wmap, xmap, a, o, grid, s);
    }
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out);
    return p.ids ? launch_pair<__nv_bfloat16, true>(wmap, xmap, a, o, grid, s)
                 : launch_pair<__nv_bfloat16, false>(wmap, xmap, a, o, grid, s);
}

}  // namespace ft
