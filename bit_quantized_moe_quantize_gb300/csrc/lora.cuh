// Pieces of the low-rank adapters' kernels: tiles of slots that share an adapter, asynchronous copies, and
// products of fp32 values with 16-bit ones on the tensor cores (mma.sync).
//
// The products here have one side of rank 8 to 128 and are bound by memory: reading a row of x of K values and
// writing one of N takes 2 K + 2 N or 2 K + 4 N bytes for 2 R (K + N) operations, R / 2 to R operations a byte, where
// the card has 280 for a byte.  Registers as accumulators, which the next step needs anyway, cost less
// there than a trip through tensor memory.
#pragma once

#include "fp8_common.cuh"

namespace ft {

constexpr int kLoraSmallTile = 16;      // slots of a tile: 16, 64 or 128
constexpr int kLoraThreads = 128;

// Slots by adapter: in order (perm, by lora_order.cu), or perm == nullptr: found by each CTA (lora_few.cuh).
struct LoraSlots {
    const int32_t *ids, *offsets, *tiles, *perm;
    int32_t n_slots, n_adapters, width;      // width: of the order's tiles
};

struct LoraTile {
    int32_t adapter;      // -1: slot `first` has none
    int32_t n;            // slots, 0: nothing to do
    int32_t first;        // in order; without one the slot itself
};

// Tile b of width MT (with an order: part b % (width / MT) of the order's tile b / (width / MT)); its slots go to slots[0 .. n).
// By all threads of the CTA; ends behind a barrier.
// Without an order, b is a slot, and stands for itself and those behind it that share its adapter where the number
// of such slots before it is a multiple of MT.
template <int MT>
__device__ __forceinline__ LoraTile find_tile(const LoraSlots& s, int32_t b, int32_t* slots) {
    constexpr int32_t threads = kLoraThreads;
    const int32_t tid = static_cast<int32_t>(threadIdx.x), L = s.n_adapters;
    if (s.perm) {
        __shared__ LoraTile found;
        if (tid == 0) found = LoraTile{0, 0, 0};
        __syncthreads();
        const int32_t parts = s.width / MT, tile = b / parts, skip = (b - tile * parts) * MT;
        for (int32_t e = tid; e < L; e += threads) {      // all that is needed asked for at once
            const int32_t t0 = __ldg(s.tiles + e), t1 = __ldg(s.tiles + e + 1), o0 = __ldg(s.offsets + e), o1 = __ldg(s.offsets + e + 1);
            const int32_t first = o0 + (tile - t0) * s.width + skip;
            if (t0 <= tile && tile < t1) found = LoraTile{e, max(0, min(MT, o1 - first)), first};
        }
        __syncthreads();
        const LoraTile t = found;
        if (tid < t.n) slots[tid] = __ldg(s.perm + t.first + tid);
        __syncthreads();
        return t;
    }
    const int32_t a = __ldg(s.ids + b);
    if (a < 0 || a >= L) return LoraTile{-1, 0, b};
    int32_t before = 0;
    for (int32_t s0 = 0; s0 < b; s0 += threads) before += __syncthreads_count(s0 + tid < b && __ldg(s.ids + s0 + tid) == a);
    if (before % MT != 0) return LoraTile{a, 0, b};
    int32_t n = 0;
    __shared__ int32_t warp_n[threads / 32];
    for (int32_t s0 = b; s0 < s.n_slots && n < MT; s0 += threads) {
        const bool mine = s0 + tid < s.n_slots && __ldg(s.ids + s0 + tid) == a;
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, mine);
        if (lane_id() == 0) warp_n[tid >> 5] = __popc(mask);
        __syncthreads();
        int32_t at = n + __popc(mask & ((1u << lane_id()) - 1u));
        for (int32_t w = 0; w < threads / 32; ++w) {
            if (w < tid >> 5) at += warp_n[w];
            n += warp_n[w];
        }
        if (mine && at < MT) slots[at] = s0 + tid;
        __syncthreads();
    }
    return LoraTile{a, min(n, MT), b};
}

// ----------------------------------------------------------- asynchronous copies
// 16 bytes to shared memory, zeros where not `there` (src is not read then).
__device__ __forceinline__ void copy16_at(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy16(void* dst, const void* src, bool there) { copy16_at(smem_u32(dst), src, there); }
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// ------------------------------------------------------------------- matrices
// Four 8 x 8 matrices of 16-bit values; lane l gives the address of row l % 8 of matrix l / 8.
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const void* row, bool trans) {
    if (trans)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(smem_u32(row)) : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(smem_u32(row)) : "memory");
}

// d += a b over 16 values; a 16 x 16 (rows of the tile), b 16 x 8.
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __nv_bfloat16) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __half) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma8_tf32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t tf32_of(float v) {
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// A pair of fp32 values as the sums of three bf16 parts, which hold their 24 bits.
__device__ __forceinline__ void split_pair(float lo, float hi, uint32_t (&part)[3]) {
#pragma unroll
    for (int t = 0; t < 3; ++t) {
        part[t] = bf16_pair(lo, hi);
        lo -= __uint_as_float(part[t] << 16);
        hi -= __uint_as_float(part[t] & 0xFFFF0000u);
    }
}

// A 16 x 16 operand of fp32 values, to be multiplied with 16-bit ones: v[2 i], v[2 i + 1] are neighbours in the
// place that mma's 16-bit operand register i has.  With bf16 as sums of three bf16 parts; with fp16, whose values
// and products have no such range, as two tf32 parts of 11 bits against fp16 turned to tf32, which is exact.  Fewer parts would
// not do where results have 16 bits either: products of ranks that cancel each other leave what the parts dropped.
template <typename T>
struct Wide16;

template <>
struct Wide16<__nv_bfloat16> {
    uint32_t part[3][4];
    __device__ __forceinline__ void set(const float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t p[3];
            split_pair(v[2 * i], v[2 * i + 1], p);
#pragma unroll
            for (int t = 0; t < 3; ++t) part[t][i] = p[t];
        }
    }
    template <int N>
    __device__ __forceinline__ void mul(float (&d)[N][4], const uint32_t (&b)[N][2]) const {
#pragma unroll
        for (int t = 2; t >= 0; --t)
#pragma unroll
            for (int j = 0; j < N; ++j) mma16(d[j], part[t], b[j][0], b[j][1], __nv_bfloat16());
    }
};

template <>
struct Wide16<__half> {
    float v[8];
    __device__ __forceinline__ void set(const float (&x)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = x[i];
    }
    template <int N>
    __device__ __forceinline__ void mul(float (&d)[N][4], const uint32_t (&b)[N][2]) const {
#pragma unroll
        for (int h = 0; h < 2; ++h) {      // the pairs' first and second eight
            uint32_t hi[4], lo[4];         // mma's rows and its first and second four: here the pairs' first and second
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = v[2 * ((i & 1) + 2 * h) + (i >> 1)];
                hi[i] = tf32_of(x);
                lo[i] = tf32_of(x - __uint_as_float(hi[i]));
            }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&b[j][h]));
                const uint32_t b0 = __float_as_uint(f.x), b1 = __float_as_uint(f.y);
                mma8_tf32(d[j], lo[0], lo[1], lo[2], lo[3], b0, b1);
                mma8_tf32(d[j], hi[0], hi[1], hi[2], hi[3], b0, b1);
            }
        }
    }
};

// A slot's fp32 sums as three bf16 parts, as the matrices' gradients take them (lora_grad_tc.cu): rows of an MMA of 128, one for all
// parts up to rank 40 (parts one after the other), one for the first two and one for the third up to rank 64, one for each
// above.  64 rows make a line of 128 bytes, whose 16-byte words are exchanged by word ^ slot % 8, slots counted within
// their adapter; lines of one kind lie in the order of the slots: [kinds][places][128 bytes].
__host__ __device__ inline int32_t part_passes(int32_t rank) { return 3 * rank <= 128 ? 1 : 2 * rank <= 128 ? 2 : 3; }
// Lines of a pass's slot; of the passes before.
__host__ __device__ inline int32_t part_lines(int32_t rank, int32_t pass) {
    const int32_t passes = part_passes(rank), rows = passes == 1 ? 3 * rank : passes == 2 && pass == 0 ? 2 * rank : rank;
    return (rows + 63) / 64;
}
__host__ __device__ inline int32_t part_kinds(int32_t rank) {
    int32_t n = 0;
    for (int32_t p = 0; p < part_passes(rank); ++p) n += part_lines(rank, p);
    return n;
}
// The pass of part t, and its first row there.
__host__ __device__ inline int32_t part_pass(int32_t passes, int32_t t) { return passes == 3 ? t : passes == 2 ? t / 2 : 0; }
__host__ __device__ inline int32_t part_row(int32_t passes, int32_t rank, int32_t t) { return passes == 3 || (passes == 2 && t == 2) ? 0 : t * rank; }

// Elements between rows of `n` 16-bit values in shared memory: whole 16-byte words, an odd number of them, so that
// eight rows' words at one column lie in different banks.
inline __host__ __device__ int32_t odd_pitch(int32_t n) { return ((n + 7) / 8 | 1) * 8; }

// Neighbouring threads hold columns 2 q and 2 q + 1 of each of four tiles of eight: of 32 columns, eight a thread.  Columns are
// put where that makes whole 16-byte words side by side for neighbours: column 8 q + 2 j + i goes to place 8 j + 2 q + i, and with
// fp32 results, which are two words a thread, column 16 (j / 2) + 4 q + 2 (j % 2) + i does.
template <bool FP32>
__device__ __forceinline__ int32_t spread_col(int32_t c) {
    if (FP32) return (c & ~31) | (c >> 4 & 1) << 4 | (c >> 1 & 1) << 3 | (c >> 2 & 3) << 1 | (c & 1);
    return (c & ~31) | (c >> 1 & 3) << 3 | (c >> 3 & 3) << 1 | (c & 1);
}

}  // namespace ft
