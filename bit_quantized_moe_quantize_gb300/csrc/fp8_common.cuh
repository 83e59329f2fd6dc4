// Device helpers of the FP8 expert-layer operators: e4m3 conversions, typed
// element loads and stores, and the order-preserving integer form of a float.
//
// Format: e4m3 values (4 exponent bits, 3 mantissa bits, no infinities,
// largest finite value 448) with one fp32 scale per 128 consecutive values of
// an activation row and per 128 x 128 block of a weight matrix.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ft_common.cuh"

namespace ft {

constexpr int kFp8Block = 128;        // values per scale
constexpr float kFp8Max = 448.0f;     // largest finite e4m3 value

inline __host__ __device__ int64_t fp8_blocks(int64_t n) { return (n + kFp8Block - 1) / kFp8Block; }

// Two fp32 values -> two e4m3 codes (round to nearest even, saturating; NaN
// stays NaN), `lo` in the low byte.
__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    return static_cast<uint32_t>(e4m3x2(a, b)) | (static_cast<uint32_t>(e4m3x2(c, d)) << 16);
}

// Loads of one element of a FT_DTYPE_* type as fp32 (exact).
template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// fp32 -> T, round to nearest even.
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// N consecutive elements, whole 16-byte words of them, as fp32; p must be 16-byte aligned.
template <typename T, int N>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[N]) {
    constexpr int PER = 16 / static_cast<int>(sizeof(T));
    static_assert(N % PER == 0, "whole words");
#pragma unroll
    for (int i = 0; i < N / PER; ++i) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(p) + i);
        const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
        for (int j = 0; j < PER; ++j) v[i * PER + j] = to_f32<T>(e[j]);
    }
}

// The same by ordinary loads, for data that another kernel may have written while this one
// was already running.
template <int N>
__device__ __forceinline__ void load_vec_plain(const float* p, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        const float4 w = reinterpret_cast<const float4*>(p)[i];
        v[4 * i] = w.x;
        v[4 * i + 1] = w.y;
        v[4 * i + 2] = w.z;
        v[4 * i + 3] = w.w;
    }
}

// Unsigned integer that orders like the float (-0 and +0 stay equal: the sum
// with +0 turns -0 into +0); larger is larger, -inf maps above 0.
__device__ __forceinline__ uint32_t float_order(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}

}  // namespace ft
