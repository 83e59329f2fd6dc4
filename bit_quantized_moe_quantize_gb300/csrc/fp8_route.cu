// Router order for the FP8 products: a stable counting sort of the slots by
// expert, in one launch (up to 1024 slots) or two.
//
//   offsets[e]  first position of expert e; offsets[n_experts] = routed slots
//   perm[p]     slot at position p, ascending within an expert
//   pos[s]      position of slot s, -1 where it has no expert (may be null)
//   tiles[e]    prefix over experts of ceil(count / tile)
//
// A chunk of 1024 slots belongs to one CTA.  The first launch counts each
// chunk's experts.  In the second every CTA adds up the chunks before its own
// (and all of them, for the offsets) by itself, which for up to 256 chunks is
// less work than another launch, and places its slots: each of its eight warps
// counts 128 of them, and equal ids in a step of 32 rank by lane, so that the
// order never depends on timing.
//
// 65536 slots, 128 experts: 5 us and 17 us; bound by the place kernel's chain of barriers.
//
// Past kFastRouteSlots or kMostRouteExperts the GGUF path's router: the prefixes over chunks take
// chunks^2 times experts reads in all, and somewhere past both bounds that is the longer way.
// A product of short rows on this router / on that one (us): 262152 slots of 128 experts 119 / 127,
// 524288 212 / 221, 2 million 1085 / 778; 8192 slots of 1100 experts 39 / 48, 65536 of 2048 166 / 180,
// 262144 of 4096 1862 / 1231.
#include "fp8_order.cuh"
#include "ft_internal.h"

namespace ft {

constexpr int32_t kMostRouteExperts = 1024;

bool fp8_route_ok(int64_t n_slots, int32_t n_experts) {
    return n_slots <= kFastRouteSlots && n_experts <= kMostRouteExperts;
}

size_t fp8_route_scratch(int64_t n_slots, int32_t n_experts) {
    return 4 * static_cast<size_t>((n_slots + kChunk - 1) / kChunk) * static_cast<size_t>(n_experts);
}

__global__ void __launch_bounds__(kChunkThreads)
    fp8_count_kernel(const int32_t* __restrict__ ids, int32_t n_slots, int32_t n_experts, int32_t* __restrict__ hist) {
    extern __shared__ int32_t count[];
    for (int32_t e = threadIdx.x; e < n_experts; e += kChunkThreads) count[e] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kChunk / kChunkThreads; ++i) {
        const int32_t s = static_cast<int32_t>(blockIdx.x) * kChunk + i * kChunkThreads + static_cast<int32_t>(threadIdx.x);
        const int32_t e = s < n_slots ? ids[s] : -1;
        if (e >= 0 && e < n_experts) atomicAdd(&count[e], 1);      // a count: the order of the additions does not show
    }
    __syncthreads();
    for (int32_t e = threadIdx.x; e < n_experts; e += kChunkThreads)
        hist[static_cast<int64_t>(blockIdx.x) * n_experts + e] = count[e];
}

// hist == nullptr: one chunk, whose counts are the totals.
__global__ void __launch_bounds__(kChunkThreads)
    fp8_place_kernel(const int32_t* __restrict__ ids, int32_t n_slots, int32_t n_experts, const int32_t* __restrict__ hist,
                     int32_t n_chunks, int32_t tile, int32_t* __restrict__ offsets, int32_t* __restrict__ tiles,
                     int32_t* __restrict__ perm, int32_t* __restrict__ pos) {
    extern __shared__ int32_t sh[];
    int32_t* mine = sh;                                  // [warps][E] counts, then first positions
    int32_t* before = mine + kChunkWarps * n_experts;    // [E] slots of the chunks before this one
    int32_t* total = before + n_experts;                 // [E] slots, then offsets
    int32_t* nt = total + n_experts;                     // [E] tiles
    int32_t* part = nt + n_experts;                      // [8]
    const int32_t E = n_experts, chunk = static_cast<int32_t>(blockIdx.x);
    int32_t id[4], rank[4];
    const int32_t s0 = chunk_rank(ids, chunk * kChunk, n_slots, E, mine, id, rank);
    const int32_t* count = mine + static_cast<int32_t>(threadIdx.x >> 5) * E;
    if (hist) {
        // the chunks are shared out between the threads that E experts leave
        const int32_t parts = E < kChunkThreads ? kChunkThreads / E : 1;
        for (int32_t e = threadIdx.x; e < E; e += kChunkThreads) before[e] = total[e] = 0;
        __syncthreads();
        for (int32_t i = threadIdx.x; i < parts * E; i += kChunkThreads) {
            const int32_t e = i % E, part = i / E;
            int32_t b = 0, t = 0;
#pragma unroll 16
            for (int32_t c = part; c < n_chunks; c += parts) {
                const int32_t x = __ldg(hist + static_cast<int64_t>(c) * E + e);
                t += x;
                b += c < chunk ? x : 0;
            }
            atomicAdd(&before[e], b);      // whole numbers: the order of the additions does not show
            atomicAdd(&total[e], t);
        }
        __syncthreads();
    } else {
        chunk_totals(mine, E, total);
        for (int32_t e = threadIdx.x; e < E; e += kChunkThreads) before[e] = 0;
        __syncthreads();
    }
    for (int32_t e = threadIdx.x; e < E; e += kChunkThreads) nt[e] = (total[e] + tile - 1) / tile;
    __syncthreads();
    const int32_t routed = chunk_scan(total, E, part);
    if (chunk == 0) {
        const int32_t n_tiles = chunk_scan(nt, E, part);
        for (int32_t e = threadIdx.x; e < E; e += kChunkThreads) {
            offsets[e] = total[e];
            tiles[e] = nt[e];
        }
        if (threadIdx.x == 0) {
            offsets[E] = routed;
            tiles[E] = n_tiles;
        }
    }
    for (int32_t e = threadIdx.x; e < E; e += kChunkThreads) total[e] += before[e];
    __syncthreads();
    chunk_starts(mine, E, total);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int32_t s = s0 + 32 * i;
        if (s < n_slots) {
            const int32_t p = id[i] >= 0 ? count[id[i]] + rank[i] : -1;
            if (p >= 0) perm[p] = s;
            if (pos) pos[s] = p;
        }
    }
}

__global__ void __launch_bounds__(256)
    invert_kernel(const int32_t* __restrict__ perm, const int32_t* __restrict__ n_routed, int64_t n_slots,
                  int32_t* __restrict__ pos, bool clear) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n_slots) return;
    if (clear) pos[i] = -1;
    else if (i < *n_routed) pos[perm[i]] = static_cast<int32_t>(i);
}

int launch_fp8_route(const int32_t* ids, int64_t n_slots, int32_t n_experts, int32_t tile, int32_t* hist, int32_t* offsets,
                     int32_t* tiles, int32_t* perm, int32_t* pos, cudaStream_t s) {
    const int32_t chunks = static_cast<int32_t>((n_slots + kChunk - 1) / kChunk);
    const size_t sm = (static_cast<size_t>(kChunkWarps + 3) * n_experts + 8) * 4;
    if (int st = set_smem_limit(reinterpret_cast<const void*>(fp8_place_kernel), static_cast<int>(sm))) return st;
    const dim3 grid(chunks), block(kChunkThreads);
    if (chunks > 1) {
        fp8_count_kernel<<<grid, block, 4 * static_cast<size_t>(n_experts), s>>>(ids, static_cast<int32_t>(n_slots), n_experts, hist);
        if (int st = check_launch("fp8_count_kernel", grid, block, 4 * static_cast<size_t>(n_experts))) return st;
    }
    fp8_place_kernel<<<grid, block, sm, s>>>(ids, static_cast<int32_t>(n_slots), n_experts, chunks > 1 ? hist : nullptr, chunks,
                                             tile, offsets, tiles, perm, pos);
    return check_launch("fp8_place_kernel", grid, block, sm);
}

int launch_fp8_invert(const int32_t* perm, const int32_t* n_routed, int64_t n_slots, int32_t* pos, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>((n_slots + 255) / 256));
    for (int i = 0; i < 2; ++i) {
        invert_kernel<<<grid, 256, 0, s>>>(perm, n_routed, n_slots, pos, i == 0);
        if (int st = check_launch("invert_kernel", grid, dim3(256), 0)) return st;
    }
    return FT_OK;
}

}  // namespace ft
