// Rows of router logits in registers, for the kernels that need every expert's score: a group of L lanes
// holds a row of up to 8 * L * STEPS experts, eight neighbouring ones per lane and step.
#pragma once

#include "fp8_common.cuh"

namespace ft {

constexpr int kRowThreads = 256;      // of a CTA
constexpr float kScoreTiny = 1e-30f;  // smallest sum that scores are divided by

// Lanes that share a row: up to 32 neighbouring ones of a warp, or the whole CTA.
template <int L>
struct RowGroup {
    static_assert(L <= 32 || L == kRowThreads, "lanes of a warp, or the CTA");
    static constexpr int kRows = kRowThreads / L;      // rows of a CTA at once
    float* part;      // one word per warp in shared memory (used where L is the CTA)

    __device__ __forceinline__ static uint32_t lane() { return threadIdx.x % L; }
    __device__ __forceinline__ static uint32_t row() { return threadIdx.x / L; }
    __device__ __forceinline__ void sync() const {
        if constexpr (L <= 32) __syncwarp();
        else __syncthreads();
    }
    template <typename F>
    __device__ __forceinline__ float reduce(float v, const F& f) const {
#pragma unroll
        for (int o = (L < 32 ? L : 32) / 2; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
        if constexpr (L > 32) {
            __syncthreads();
            if ((threadIdx.x & 31u) == 0) part[threadIdx.x >> 5] = v;
            __syncthreads();
            v = part[0];
#pragma unroll
            for (int w = 1; w < L / 32; ++w) v = f(v, part[w]);
        }
        return v;
    }
    __device__ __forceinline__ float max(float v) const {
        return reduce(v, [](float a, float b) { return fmaxf(a, b); });
    }
    __device__ __forceinline__ float sum(float v) const {
        return reduce(v, [](float a, float b) { return a + b; });
    }
};

// The first expert of a lane's step.
template <int L>
__device__ __forceinline__ int32_t first_expert(int step) {
    return (step * L + static_cast<int32_t>(RowGroup<L>::lane())) * 8;
}

// A lane's logits of a row on their way: words as they come, made logits when they are wanted.
// wide: rows start at whole 16-byte words.
template <typename T, int L, int STEPS>
struct RowAhead {
    static constexpr int WORDS = static_cast<int>(sizeof(T)) * 8 / 16;
    uint4 word[STEPS][WORDS];
    __device__ __forceinline__ void fetch(const T* row, int32_t E, bool wide) {
        if (!wide) return;
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
            for (int w = 0; w < WORDS; ++w)
                if (first_expert<L>(s) + 8 <= E) word[s][w] = __ldg(reinterpret_cast<const uint4*>(row + first_expert<L>(s)) + w);
    }
    // Masked experts (-inf, NaN) and those past the last are -inf.
    __device__ __forceinline__ void take(const T* row, int32_t E, bool wide, float (&l)[STEPS][8]) const {
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int32_t e0 = first_expert<L>(s);
            const T* v = reinterpret_cast<const T*>(word[s]);
            if (wide && e0 + 8 <= E) {
#pragma unroll
                for (int i = 0; i < 8; ++i) l[s][i] = fmaxf(to_f32<T>(v[i]), -INFINITY);      // the operand that is no NaN
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) l[s][i] = e0 + i < E ? fmaxf(to_f32<T>(row[e0 + i]), -INFINITY) : -INFINITY;
            }
        }
    }
};

// e^x for x <= 0, off by (1.5 |x| + 4) 2^-24 of itself: the argument times log2(e) rounded, log2(e) itself, two units
// in the power; below 2^-126 it is 0.  With the quotients by __fdividef, two units more, fp32 gradients of a sigmoid router are
// 1.3 10^-7 off (777 x 256), a plain fp32 form 1.0 10^-7.
__device__ __forceinline__ float row_exp(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
    return r;
}

// sigmoid(l) and 1 - sigmoid(l), neither by a difference.
__device__ __forceinline__ void sigmoid_pair(float l, float& s, float& rest) {
    const float e = row_exp(-fabsf(l)), r = __fdividef(1.0f, 1.0f + e), small = e * r;
    s = l >= 0.0f ? r : small;
    rest = l >= 0.0f ? small : r;
}

// What a row's scores need beside its logits.
struct RowScale {
    float top, inv;      // softmax: the largest logit, the reciprocal of the sum of exponentials (0 where no expert is there)
    float sum;           // sigmoid: of the scores
    bool any;            // some expert is there
};

// exp(l - top) of an expert that is there; experts at +inf share the softmax.
__device__ __forceinline__ float soft_exp(float l, float top) { return l == top ? 1.0f : row_exp(l - top); }

// In place: logits -> exp(l - top), 0 where masked; times RowScale::inv, the softmax.
template <int L, int STEPS>
__device__ __forceinline__ RowScale row_softmax(const RowGroup<L>& g, float (&l)[STEPS][8]) {
    float top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, l[s][i]);
    top = g.max(top);
    const bool any = top > -INFINITY;
    float base = any ? top : 0.0f;
    if (top == INFINITY) {
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
            for (int i = 0; i < 8; ++i) l[s][i] = l[s][i] == INFINITY ? 0.0f : -INFINITY;
        base = 0.0f;
    }
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            l[s][i] = row_exp(l[s][i] - base);
            sum += l[s][i];
        }
    sum = g.sum(sum);
    return RowScale{top, any ? __fdividef(1.0f, sum) : 0.0f, 0.0f, any};      // the largest logit alone makes the sum 1 or more
}

// In place: logits -> sigmoid scores, 0 where masked; rest: 1 - score there.
template <int L, int STEPS>
__device__ __forceinline__ RowScale row_sigmoid(const RowGroup<L>& g, float (&l)[STEPS][8], float (&rest)[STEPS][8]) {
    float sum = 0.0f, there = 0.0f;
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool ok = l[s][i] > -INFINITY;
            float v;
            sigmoid_pair(l[s][i], v, rest[s][i]);
            l[s][i] = ok ? v : 0.0f;
            rest[s][i] = ok ? rest[s][i] : 0.0f;
            there = ok ? 1.0f : there;
            sum += l[s][i];
        }
    sum = g.sum(sum);
    return RowScale{0.0f, 0.0f, sum, g.max(there) > 0.0f};
}

// Sequences of packed rows: offsets[0 .. n] ascending, or null: one sequence of all rows.  Whatever the
// offsets hold, what comes back lies in [0, rows].
__device__ __forceinline__ int64_t seq_start(const int32_t* offsets, int32_t s, int64_t rows) {
    if (!offsets) return s == 0 ? 0 : rows;
    const int64_t o = __ldg(offsets + s);
    return o < 0 ? 0 : o < rows ? o : rows;
}

// The last sequence that starts at or before row r (0 if none does).
__device__ __forceinline__ int32_t seq_of(const int32_t* offsets, int32_t n, int64_t r) {
    int32_t lo = 0, hi = n - 1;
    while (lo < hi) {
        const int32_t mid = (lo + hi + 1) >> 1;
        if (__ldg(offsets + mid) <= r) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Calls f with the lanes per row and the steps that E experts take; FEW: half the lanes where that can be.
template <bool FEW = false, typename F>
int with_row_lanes(int32_t E, const F& f) {
    if constexpr (FEW) {
        if (E > 32 && E <= 64) return f(std::integral_constant<int, 4>{}, std::integral_constant<int, 2>{});
        if (E > 64 && E <= 128) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 2>{});
        if (E > 128 && E <= 256) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 2>{});
    }
    if (E <= 32) return f(std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{});
    if (E <= 64) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
    if (E <= 128) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
    if (E <= 256) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 1>{});
    if (E <= 512) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, kRowThreads>{}, std::integral_constant<int, 2>{});
}

}  // namespace ft
