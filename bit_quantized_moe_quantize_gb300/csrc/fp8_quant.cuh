// The arithmetic of the FP8 quantizer, shared by every kernel that forms codes from fp32
// values with IEEE quotients: the gated activation, the codes of eight values, and the
// scale of a block held by half a warp.
#pragma once

#include "fp8_common.cuh"

namespace ft {

__device__ __forceinline__ float rcp_approx(float x) {      // within one unit in the last place; 0 for infinity
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The gated activation of one value: act(g) * up with act(g) = g / (1 + exp(-z)), z = g for
// SiLU and 2 sqrt(2/pi) (g + 0.044715 g^3) for the tanh form of GELU.  exp(-z) = 2^(-z log2 e)
// is off by the rounding of its argument, 2^-24 |z| of itself, and two units in the last place:
// some 2^-20 where act(g) has a size to speak of, beside the 2^-4 that a code rounds off
// (expf's exact reduction of the argument takes four more instructions of some twenty).
__device__ __forceinline__ float act_mul_f32(float g, float up, int kind) {
    const float cube = __fmul_rn(__fmul_rn(__fmul_rn(0.044715f, g), g), g);
    const float z = kind == FT_ACT_SILU ? g : __fmul_rn(1.5957691216057308f, __fadd_rn(g, cube));
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
    return g * rcp_approx(1.0f + e) * up;
}

// Two fp32 values in a 64-bit register, and their packed product.
__device__ __forceinline__ uint64_t pair2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint32_t e4m3x4(uint64_t a, uint64_t b) {
    float2 x, y;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x.x), "=f"(x.y) : "l"(a));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(y.x), "=f"(y.y) : "l"(b));
    return e4m3x4(x.x, x.y, y.x, y.y);
}

// Codes of v / scale for eight values; inv: rcp_approx(scale).  y = v * inv lies within
// 2^-22 |v / scale| of the IEEE quotient (2^-23 of the reciprocal, 2^-24 of the product and of
// the quotient), so both round to the same code unless y (1 - 2^-21) and y (1 + 2^-21) do not;
// only then, or where 1 / scale could overflow, are the quotients formed.
__device__ __forceinline__ uint2 fp8_codes(const float (&v)[8], float scale, float inv) {
    const uint64_t inv2 = pair2(inv, inv), down = pair2(1.0f - 0x1p-21f, 1.0f - 0x1p-21f), up = pair2(1.0f + 0x1p-21f, 1.0f + 0x1p-21f);
    uint32_t lo[2], hi[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint64_t a = mul2(pair2(v[4 * h], v[4 * h + 1]), inv2), b = mul2(pair2(v[4 * h + 2], v[4 * h + 3]), inv2);
        lo[h] = e4m3x4(mul2(a, down), mul2(b, down));
        hi[h] = e4m3x4(mul2(a, up), mul2(b, up));
    }
    if (lo[0] != hi[0] || lo[1] != hi[1] || !(scale > 1.0e-36f)) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            lo[h] = scale == 0.0f ? 0u
                                  : e4m3x4(__fdiv_rn(v[4 * h], scale), __fdiv_rn(v[4 * h + 1], scale),
                                           __fdiv_rn(v[4 * h + 2], scale), __fdiv_rn(v[4 * h + 3], scale));
    }
    return make_uint2(lo[0], lo[1]);
}

// The largest of two or three values, NaN if one of them is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Scale of a block of 128 values, eight in each of 16 neighbouring lanes or 16 in each of 8.
template <int N>
__device__ __forceinline__ float fp8_block_scale(const float (&v)[N][8]) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 8; j += 2) top = max_nan(top, fabsf(v[i][j]), fabsf(v[i][j + 1]));
#pragma unroll
    for (int o = 8 / N; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    return __fdiv_rn(top, kFp8Max);
}

}  // namespace ft
