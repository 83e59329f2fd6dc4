// Slots by adapter for batches of up to 131072 slots and 512 adapters, in one launch of one cluster: a stable counting
// sort.  Each warp takes a run of slots, in rounds of 32 whose equal ids rank by lane, and counts them in a row of its own;
// prefixes over the warps, over the cluster's CTAs and over the adapters make the slots' places, so that no order depends
// on timing.  Equal ids are found by a vote for each of their bits: __match_any_sync takes a turn for every different id of a
// warp (16384 slots of 128 adapters in one CTA: 28 us with it, 15 with votes; by eight CTAs 8).  Larger batches go through the FP8
// products' router (fp8_route.cu), whose outputs these are.
//
//   offsets[e]  first place of adapter e, offsets[L] = slots that have one
//   tiles[e]    prefix over adapters of ceil(count / width)
//   perm[p]     slot at place p, ascending within an adapter
#include "fp8_common.cuh"
#include "ft_internal.h"
#include "launch.cuh"

namespace ft {

namespace {

constexpr int kOrderThreads = 1024, kOrderWarps = 32, kOrderRounds = 16;
constexpr int32_t kOrderAdapters = 512;
constexpr unsigned kOrderCtas = 8;

__global__ void __launch_bounds__(kOrderThreads)
    lora_order_kernel(const int32_t* __restrict__ ids, int32_t n_slots, int32_t L, int32_t bits, int32_t width, int32_t* __restrict__ offsets,
                      int32_t* __restrict__ tiles, int32_t* __restrict__ perm) {
    extern __shared__ int32_t order_smem[];
    let_next_grid_start();
    __shared__ int2 part[kOrderWarps];
    int32_t* hist = order_smem;                     // [warps][L] counts, then first places
    int32_t* start = hist + kOrderWarps * L;        // [L] this CTA's slots, then its first places
    const int32_t tid = static_cast<int32_t>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    const uint32_t size = cluster_size(), cta = cluster_rank();
    const int32_t per_round = kOrderThreads * static_cast<int32_t>(size), rounds = (n_slots + per_round - 1) / per_round;
    const int32_t first = (static_cast<int32_t>(cta) * kOrderWarps + warp) * rounds * 32 + lane;
    int32_t id[kOrderRounds], rank[kOrderRounds];
#pragma unroll
    for (int i = 0; i < kOrderRounds; ++i) {
        const int32_t s = first + i * 32, e = i < rounds && s < n_slots ? __ldg(ids + s) : -1;
        id[i] = e >= 0 && e < L ? e : -1;
    }
    for (int32_t i = tid; i < kOrderWarps * L; i += kOrderThreads) hist[i] = 0;
    __syncthreads();
    int32_t* count = hist + warp * L;
    const uint32_t below = (1u << lane) - 1u;
#pragma unroll
    for (int i = 0; i < kOrderRounds; ++i) {
        if (i >= rounds) break;
        uint32_t same = __ballot_sync(0xFFFFFFFFu, id[i] >= 0);
        for (int b = 0; b < bits; ++b) {
            const uint32_t set = __ballot_sync(0xFFFFFFFFu, id[i] >> b & 1);
            same &= id[i] >> b & 1 ? set : ~set;
        }
        rank[i] = id[i] >= 0 ? count[id[i]] + __popc(same & below) : 0;
        __syncwarp();
        if (id[i] >= 0 && (same & below) == 0) count[id[i]] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    // one thread per adapter: its slots of the warps and of the CTAs before, and all of them
    int32_t n = 0, earlier = 0;
    if (tid < L) {
#pragma unroll 8
        for (int w = 0; w < kOrderWarps; ++w) {
            const int32_t c = hist[w * L + tid];
            hist[w * L + tid] = n;
            n += c;
        }
        start[tid] = n;
    }
    cluster_sync();
    if (tid < L) {
        n = 0;
        for (uint32_t q = 0; q < size; ++q) {
            const int32_t c = __float_as_int(cluster_load(start + tid, q));
            earlier += q < cta ? c : 0;
            n += c;
        }
    }
    cluster_sync();      // all have read
    const int32_t t = (n + width - 1) / width;
    int2 inc = make_int2(n, t);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t x = __shfl_up_sync(0xFFFFFFFFu, inc.x, o), y = __shfl_up_sync(0xFFFFFFFFu, inc.y, o);
        if (lane >= o) inc = make_int2(inc.x + x, inc.y + y);
    }
    if (lane == 31) part[warp] = inc;
    __syncthreads();
    int2 before = make_int2(0, 0);
    for (int w = 0; w < warp; ++w) before = make_int2(before.x + part[w].x, before.y + part[w].y);
    if (tid < L) {
        start[tid] = before.x + inc.x - n + earlier;
        if (cta == 0) {
            offsets[tid] = before.x + inc.x - n;
            tiles[tid] = before.y + inc.y - t;
            if (tid == L - 1) {
                offsets[L] = before.x + inc.x;
                tiles[L] = before.y + inc.y;
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kOrderRounds; ++i)
        if (i < rounds && id[i] >= 0) perm[start[id[i]] + count[id[i]] + rank[i]] = first + i * 32;
}

}  // namespace

int launch_lora_order(const int32_t* ids, int64_t n_slots, int32_t n_adapters, int width, const Fp8Order& o, cudaStream_t s) {
    if (n_slots > static_cast<int64_t>(kOrderCtas) * kOrderThreads * kOrderRounds || n_adapters > kOrderAdapters)
        return launch_fp8_order(ids, n_slots, n_adapters, width, o, s);
    int32_t bits = 0;
    while ((1 << bits) < n_adapters) ++bits;
    unsigned cluster = 1;
    while (cluster < kOrderCtas && static_cast<int64_t>(cluster) * kOrderThreads < n_slots) cluster *= 2;
    const size_t sm = 4 * static_cast<size_t>(kOrderWarps + 1) * n_adapters;
    return launch_with(lora_order_kernel, "lora_order_kernel", dim3(cluster), dim3(kOrderThreads), sm, false, cluster, s, ids,
                       static_cast<int32_t>(n_slots), n_adapters, bits, static_cast<int32_t>(width), o.offsets, o.tiles, o.perm);
}

}  // namespace ft
