// Pieces of the router order that a CTA of 256 threads works out for a chunk of up to
// 1024 slots: the ranks of its slots, the experts' totals, prefixes.
#pragma once

#include "fp8_common.cuh"

namespace ft {

constexpr int kChunk = 1024, kChunkThreads = 256, kChunkWarps = kChunkThreads / 32;

// Exclusive prefix of v[0 .. n) in shared memory by the whole CTA; returns the total.  part: 8 words.
__device__ __forceinline__ int32_t chunk_scan(int32_t* v, int32_t n, int32_t* part) {
    const int32_t tid = threadIdx.x, per = (n + kChunkThreads - 1) / kChunkThreads;
    const int32_t lo = min(n, tid * per), hi = min(n, lo + per);
    const uint32_t lane = lane_id(), warp = threadIdx.x >> 5;
    int32_t sum = 0;
    for (int32_t i = lo; i < hi; ++i) sum += v[i];
    int32_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= static_cast<uint32_t>(o)) inc += y;
    }
    if (lane == 31) part[warp] = inc;
    __syncthreads();
    int32_t before = 0, total = 0;
    for (int w = 0; w < kChunkWarps; ++w) {
        if (w < static_cast<int>(warp)) before += part[w];
        total += part[w];
    }
    int32_t run = before + inc - sum;
    for (int32_t i = lo; i < hi; ++i) {
        const int32_t x = v[i];
        v[i] = run;
        run += x;
    }
    __syncthreads();
    return total;
}

// Counts the experts of the slots from `first` on, warp by warp (mine[warp][E]: 128 slots
// each): id[i] is the expert of slot s0 + 32 i (-1: none), s0 the returned value, and rank[i] how
// many slots of the warp before it have the same.  Ends without a barrier.
__device__ __forceinline__ int32_t chunk_rank(const int32_t* __restrict__ ids, int32_t first, int32_t n_slots, int32_t E,
                                              int32_t* mine, int32_t (&id)[4], int32_t (&rank)[4]) {
    const uint32_t warp = threadIdx.x >> 5, lane = lane_id();
    for (int32_t i = threadIdx.x; i < kChunkWarps * E; i += kChunkThreads) mine[i] = 0;
    __syncthreads();
    int32_t* count = mine + static_cast<int32_t>(warp) * E;
    const int32_t s0 = first + static_cast<int32_t>(warp) * 128 + static_cast<int32_t>(lane);
    uint32_t below;
    asm("mov.u32 %0, %%lanemask_lt;" : "=r"(below));
#pragma unroll
    for (int i = 0; i < 4; ++i) {      // all four on their way before the first is used
        const int32_t s = s0 + 32 * i, e = s < n_slots ? ids[s] : -1;
        id[i] = e >= 0 && e < E ? e : -1;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, id[i]);
        rank[i] = id[i] >= 0 ? count[id[i]] + __popc(same & below) : 0;
        __syncwarp();
        if (id[i] >= 0 && (same & below) == 0) count[id[i]] += __popc(same);
        __syncwarp();
    }
    return s0;
}

// total[e]: the chunk's slots of expert e.  Barriers before and after.
__device__ __forceinline__ void chunk_totals(const int32_t* mine, int32_t E, int32_t* total) {
    __syncthreads();
    for (int32_t e = threadIdx.x; e < E; e += kChunkThreads) {
        int32_t t = 0;
        for (int w = 0; w < kChunkWarps; ++w) t += mine[w * E + e];
        total[e] = t;
    }
    __syncthreads();
}

// mine[warp][e] := first position of the warp's slots of expert e, the chunk's first being start[e].
__device__ __forceinline__ void chunk_starts(int32_t* mine, int32_t E, const int32_t* start) {
    for (int32_t e = threadIdx.x; e < E; e += kChunkThreads) {
        int32_t at = start[e];
        for (int w = 0; w < kChunkWarps; ++w) {
            const int32_t n = mine[w * E + e];
            mine[w * E + e] = at;
            at += n;
        }
    }
    __syncthreads();
}

// Number of the last of v[0 .. n) that is <= x (v ascending, v[0] <= x).
__device__ __forceinline__ int32_t last_not_above(const int32_t* v, int32_t n, int32_t x) {
    int32_t lo = 0, hi = n - 1;
    while (lo < hi) {
        const int32_t mid = (lo + hi + 1) >> 1;
        if (v[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

}  // namespace ft
