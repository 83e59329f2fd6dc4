// Dot products of e4m3 codes on the CUDA cores: 16 codes of a weight row by 16 of an
// activation row per lane.
//
// Codes become fp16 pairs (exact); the activations' also times 2^-4 (exact), which keeps
// every product inside fp16's range of exact ones (448 * 448 / 16 < 65504, the smallest
// 2^-22).  Products are added in fp32 by mixed FMAs.
#pragma once

#include "fp8_common.cuh"

namespace ft {

constexpr float kActDown = 0.0625f, kActUp = 16.0f;      // 2^-4, and what undoes it

__device__ __forceinline__ void e4m3x4_to_f16(uint32_t q, uint32_t (&h)[2]) {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[0]) : "h"(static_cast<uint16_t>(q & 0xFFFFu)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[1]) : "h"(static_cast<uint16_t>(q >> 16)));
}

// acc += a * b, fp16 operands, fp32 sum.
__device__ __forceinline__ float fma_f16(uint16_t a, uint16_t b, float acc) {
    float r;
    asm("fma.rn.f32.f16 %0, %1, %2, %3;" : "=f"(r) : "h"(a), "h"(b), "f"(acc));
    return r;
}

// 16 activation codes -> eight fp16 pairs, times 2^-4.
__device__ __forceinline__ void act_to_f16(uint4 x, uint32_t (&a)[8]) {
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t h[2];
        e4m3x4_to_f16(xs[j], h);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const __half2 d = __hmul2(*reinterpret_cast<__half2*>(&h[k]), __floats2half2_rn(kActDown, kActDown));
            a[2 * j + k] = *reinterpret_cast<const uint32_t*>(&d);
        }
    }
}

// 2^-4 times the dot product of 16 weight codes with them.
__device__ __forceinline__ float dot16(uint4 w, const uint32_t (&a)[8]) {
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
    float even = 0.0f, odd = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t h[2];
        e4m3x4_to_f16(ws[j], h);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            even = fma_f16(static_cast<uint16_t>(h[k] & 0xFFFFu), static_cast<uint16_t>(a[2 * j + k] & 0xFFFFu), even);
            odd = fma_f16(static_cast<uint16_t>(h[k] >> 16), static_cast<uint16_t>(a[2 * j + k] >> 16), odd);
        }
    }
    return even + odd;
}

}  // namespace ft
