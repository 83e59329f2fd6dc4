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
// core in fp32 in a tensor-memory accumulator (two of them, 256 columns each, in
// turn); the scales change with the next block, so the drain takes each block's
// sums out of tensor memory and adds them, times sa * sw, to fp32 registers.
// Slots lie along the lanes, so that product is one number per thread: with the
// weight rows along the lanes a thread needs one scale per column, and reading
// those from shared memory for 32 rows at a time, or taking the accumulator out
// in 16-lane shapes to share them (half the rate: 514 cycles a block against 144),
// costs more than the MMAs of the block (512 cycles).
//
// Per CTA, warp-specialised:
//   8 drain warps  warp w: TMEM lanes 32 (w % 4) .. + 31 (one slot per thread),
//                  columns 128 (w / 4) .. + 127
//   producer       TMA: the weight boxes, and the slots' rows four at a time by
//                  index (gather), or in boxes of 16 neighbouring rows where
//                  slots lie in order, both with 128-byte swizzle; columns past
//                  the row's end arrive as 0
//   MMA            (leader CTA) four MMAs of 32 columns per block
#include "fp8_tc.cuh"
#include "ft_internal.h"
#include "gemm_common.cuh"

namespace ft {

struct Pair {
    static constexpr int BM = 128;                 // slots per CTA
    static constexpr int BN = 256;                 // weight rows per tile
    static constexpr int STAGES = 5;
    static constexpr int A_BYTES = BM * kFp8Block;
    static constexpr int B_BYTES = BN / 2 * kFp8Block;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int BOX = 64;                 // weight rows per TMA box
    static constexpr int N_DRAIN_WARPS = 8;
    static constexpr int WARP_PRODUCER = 8, WARP_MMA = 9;
    static constexpr int THREADS = 12 * 32;        // warps 10 and 11 complete the third warpgroup and zero rows
    // registers: 384 threads are launched with LAUNCH_REGS each; the drain warps
    // take DRAIN_REGS, and the others give theirs down to OTHER_REGS
    static constexpr int LAUNCH_REGS = 168, DRAIN_REGS = 216, OTHER_REGS = 72;
    static_assert(DRAIN_REGS * 256 + OTHER_REGS * 128 <= LAUNCH_REGS * THREADS, "the split must fit the launch's registers");
    static constexpr int CW = BN / 2;              // columns per drain warp
    static constexpr int OFF_BAR = STAGES * STAGE_BYTES;
    static constexpr int N_BARS = 2 * STAGES + 4;
    static constexpr int OFF_TMEM = OFF_BAR + N_BARS * 8;
    static constexpr int SMEM_BYTES = OFF_TMEM + 16 + 1024;    // + alignment slack
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
    bool wide;                   // the rows of out are whole 16-byte words
};

struct PairTile {
    int32_t e, n, half, width;   // expert, valid slots, slots of CTA 0 (the rest are CTA 1's), MMA width
    int64_t p0, r0;              // first router position, first weight row
    // slots of CTA `rank`, and their first position
    __device__ int32_t mine(uint32_t rank) const { return rank ? n - half : half; }
    __device__ int64_t first(uint32_t rank) const { return p0 + (rank ? half : 0); }
};

// Work item w: row tile w % row_tiles of slot tile w / row_tiles.
__device__ __forceinline__ PairTile pair_tile(const PairArgs& a, int64_t w) {
    PairTile t;
    const int64_t st = w / a.row_tiles;
    t.r0 = (w - st * a.row_tiles) * Pair::BN;
    t.width = static_cast<int32_t>(min(static_cast<int64_t>(Pair::BN), (a.nrows - t.r0 + 31) / 32 * 32));
    int64_t first = 0, count = a.n_slots, j = st;
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
        j = st - a.tiles[lo];
    }
    t.p0 = first + j * (2 * Pair::BM);
    t.n = static_cast<int32_t>(min(static_cast<int64_t>(2 * Pair::BM), count - j * (2 * Pair::BM)));
    t.half = min(t.n, (t.n + 63) / 64 * 32);        // whole warps, nearly even
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
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_TMEM);

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

    const int64_t slot_tiles = a.tiles ? a.tiles[a.n_experts] : (a.n_slots + 2 * C::BM - 1) / (2 * C::BM);
    const int64_t total = slot_tiles * a.row_tiles;
    const int64_t w0 = blockIdx.x / 2, dw = gridDim.x / 2;

    if (warp >= C::N_DRAIN_WARPS) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::OTHER_REGS));
    if (warp == C::WARP_PRODUCER) {
        // ------------------------------------------------------------ producer
        uint32_t it = 0;
        bool ok = true;
        for (int64_t w = w0; w < total && ok; w += dw) {
            const PairTile t = pair_tile(a, w);
            const int32_t mine = t.mine(rank), other = t.mine(rank ^ 1u);
            // lane l copies 4 (gather) or 16 of this CTA's slots
            constexpr int PER = GATHER ? 4 : 16;
            const bool copies = static_cast<int32_t>(lane) * PER < mine;
            int32_t y[4] = {0, 0, 0, 0};
            if (copies) {
                const int64_t p = t.first(rank) + lane * PER;
                if constexpr (GATHER) {
                    const int64_t last = t.first(rank) + mine - 1;      // the last rows of a part group repeat it
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = a.perm[min(p + i, last)] / a.act_div;
                } else {
                    y[0] = static_cast<int32_t>(p);
                }
            }
            // weight rows of this CTA's half of the tile: one box or two
            const int32_t boxes = t.width > 2 * C::BOX ? 2 : 1;
            const int32_t wy = static_cast<int32_t>(static_cast<int64_t>(t.e) * a.nrows + t.r0 + rank * (t.width / 2));
            const uint32_t bytes = 2 * boxes * C::BOX * kFp8Block +
                                   ((mine + PER - 1) / PER + (other + PER - 1) / PER) * PER * kFp8Block;
            for (int32_t b = 0; b < nb; ++b, ++it) {
                const uint32_t s = it % C::STAGES;
                if (!mbar_wait_warp(&empty[s], ((it / C::STAGES) & 1u) ^ 1u, a.err)) { ok = false; break; }
                const uint32_t bar = map_to_rank(smem_u32(&full[s]), 0);
                const uint32_t dst = smem_u32(smem + s * C::STAGE_BYTES);
                if (lane == 0 && rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
                if (static_cast<int32_t>(lane) < boxes)
                    tma_load_2d_pair(dst + C::A_BYTES + lane * (C::BOX * kFp8Block), &wmap, b * kFp8Block,
                                     wy + static_cast<int32_t>(lane) * C::BOX, bar);
                if (copies) {
                    const uint32_t d = dst + lane * (PER * kFp8Block);
                    if constexpr (GATHER) tma_gather4_pair(d, &xmap, b * kFp8Block, y, bar);
                    else tma_load_2d_pair(d, &xmap, b * kFp8Block, y[0], bar);
                }
                __syncwarp();
            }
        }
    } else if (warp == C::WARP_MMA) {
        // ----------------------------------------------------------------- MMA
        if (rank == 0 && lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int64_t w = w0; w < total && ok; w += dw) {
                const PairTile t = pair_tile(a, w);
                const uint32_t idesc = idesc_e4m3_f32(2 * C::BM, t.width);
                for (int32_t b = 0; b < nb; ++b, ++it) {
                    const uint32_t s = it % C::STAGES, d = it & 1u;
                    if (!mbar_wait(&acc_empty[d], ((it >> 1) & 1u) ^ 1u, a.err)) { ok = false; break; }
                    if (!mbar_wait(&full[s], (it / C::STAGES) & 1u, a.err)) { ok = false; break; }
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
    } else if (warp > C::WARP_MMA) {
        if (a.ids) zero_unrouted<TO>(a, out, static_cast<int64_t>(blockIdx.x) * 2 + (warp & 1u),
                                     static_cast<int64_t>(gridDim.x) * 2);
    }
    } else {
        // --------------------------------------------------------------- drain
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::DRAIN_REGS));
        const uint32_t lane0 = (warp & 3u) * 32u, col0 = (warp >> 2) * static_cast<uint32_t>(C::CW);
        const uint32_t acc_empty0 = map_to_rank(smem_u32(acc_empty), 0);
        uint32_t it = 0;
        bool ok = true;
        for (int64_t w = w0; w < total && ok; w += dw) {
            const PairTile t = pair_tile(a, w);
            const int32_t mine = t.mine(rank);
            const int32_t m = static_cast<int32_t>(lane0 + lane);        // this thread's slot of the CTA
            const bool has = m < mine;
            // nothing to do for warps without a slot or past the weight rows
            const bool busy = static_cast<int32_t>(lane0) < mine && static_cast<int32_t>(col0) < t.width;
            int64_t slot = 0;
            const float* sa = a.act_scales;
            if (has) {
                slot = t.first(rank) + m;
                if (a.perm) slot = a.perm[slot];
                sa += slot / a.act_div * nb;
            }
            const int64_t rb = min((t.r0 + col0) / kFp8Block, static_cast<int64_t>(a.row_blocks - 1));
            const float* sw = a.w_scales + (static_cast<int64_t>(t.e) * a.row_blocks + rb) * nb;
            float2 acc[C::CW / 2];
#pragma unroll
            for (int i = 0; i < C::CW / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
            float next = __ldg(sa) * __ldg(sw);
            for (int32_t b = 0; b < nb; ++b, ++it) {
                const uint32_t d = it & 1u;
                const float2 sc = make_float2(next, next);
                if (b + 1 < nb) next = __ldg(sa + b + 1) * __ldg(sw + b + 1);
                if (!mbar_wait_warp(&acc_full[d], (it >> 1) & 1u, a.err)) { ok = false; break; }
                tc_fence_after();
                if (busy) {
#pragma unroll
                    for (int j = 0; j < C::CW / 32; ++j) {
                        uint32_t v[32];
                        tmem_ld_32x32b_x32(tmem + d * C::BN + (lane0 << 16) + col0 + 32 * j, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            acc[16 * j + i] = fma2(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), sc,
                                                   acc[16 * j + i]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(acc_empty0 + d * 8);
            }
            if (!ok) break;
            if (busy && has) {
                TO* o = out + slot * a.nrows + t.r0 + col0;
                const int32_t left = static_cast<int32_t>(min(static_cast<int64_t>(C::CW), a.nrows - t.r0 - col0));
                constexpr int PER = 16 / static_cast<int>(sizeof(TO));
                const float* f = reinterpret_cast<const float*>(acc);
                if (a.wide) {
#pragma unroll
                    for (int i = 0; i < C::CW / PER; ++i) {
                        if (PER * i < left) {
                            __align__(16) TO v[PER];
#pragma unroll
                            for (int k = 0; k < PER; ++k) v[k] = from_f32<TO>(f[PER * i + k]);
                            *reinterpret_cast<uint4*>(o + PER * i) = *reinterpret_cast<const uint4*>(v);
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < C::CW; ++i)
                        if (i < left) o[i] = from_f32<TO>(f[i]);
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
    static int regs = 0;     // of this instantiation: with fewer than LAUNCH_REGS the split of registers would never end
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
    a.row_tiles = static_cast<int32_t>((p.nrows + C::BN - 1) / C::BN);
    const int out_bytes = out_dtype == FT_DTYPE_F32 ? 4 : 2;
    a.wide = p.nrows * out_bytes % 16 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0;
    if (p.ids) {
        RouteBuffers rb{};
        rb.counts = reinterpret_cast<int32_t*>(ws + L.counts);
        rb.offsets = reinterpret_cast<int32_t*>(ws + L.offsets);
        rb.perm = reinterpret_cast<int32_t*>(ws + L.perm);
        rb.hist = reinterpret_cast<int32_t*>(ws + L.hist);
        rb.tiles_gemm = reinterpret_cast<int32_t*>(ws + L.tiles);
        rb.err = reinterpret_cast<uint32_t*>(ws + L.err);
        if (int st = launch_route(p.ids, p.n_slots, p.n_experts, rb, 2 * C::BM, 2 * C::BM, nullptr, 0, s)) return st;
        a.ids = p.ids;
        a.perm = rb.perm;
        a.offsets = rb.offsets;
        a.tiles = rb.tiles_gemm;
    }
    CUtensorMap wmap, xmap;
    if (int st = encode_2d(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.weights, p.ncols,
                           static_cast<uint64_t>(p.n_experts) * p.nrows, p.ncols, kFp8Block, C::BOX,
                           CU_TENSOR_MAP_SWIZZLE_128B, "FP8 weights"))
        return st;
    if (int st = encode_2d(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.act, p.ncols, p.act_rows, p.ncols, kFp8Block,
                           p.ids ? 1 : 16, CU_TENSOR_MAP_SWIZZLE_128B, "FP8 activations"))
        return st;
    const int64_t slot_tiles = (p.n_slots + 2 * C::BM - 1) / (2 * C::BM) + (p.ids ? (p.n_experts < p.n_slots ? p.n_experts : p.n_slots) : 0);
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
