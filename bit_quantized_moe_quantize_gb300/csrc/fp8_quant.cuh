// The arithmetic of the FP8 quantizer, shared by every kernel that forms codes from fp32
// values with IEEE quotients: the gated activation, the codes of eight values, and the
// scale of a block held by half a warp.
#pragma once

#include "fp8_common.cuh"

namespace ft {

// The gated activation of one value: act(g) * up with act(g) = g / (1 + exp(-z)), z = g for
// SiLU and 2 sqrt(2/pi) (g + 0.044715 g^3) for the tanh form of GELU.  The quotient is
// within two units in the last place.
__device__ __forceinline__ float act_mul_f32(float g, float up, int kind) {
    const float cube = __fmul_rn(__fmul_rn(__fmul_rn(0.044715f, g), g), g);
    const float z = kind == FT_ACT_SILU ? g : __fmul_rn(1.5957691216057308f, __fadd_rn(g, cube));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + expf(-z)));      // 0 for an infinite sum
    return g * r * up;
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

// Codes of v / scale for eight values.  y = v * (1 / scale) lies within 2^-22 |v / scale| of
// the IEEE quotient (two roundings of half a unit against one), so both round to the same
// code unless y (1 - 2^-21) and y (1 + 2^-21) do not; only then, or where 1 / scale could
// overflow, are the quotients formed.
__device__ __forceinline__ uint2 fp8_codes(const float (&v)[8], float scale) {
    const float inv = __frcp_rn(scale);
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

// The larger of two values, NaN if one of them is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Scale of a block of 128 values, eight in each lane of half a warp.
__device__ __forceinline__ float fp8_block_scale(const float (&v)[8]) {
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max_nan(top, fabsf(v[j]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    return __fdiv_rn(top, kFp8Max);
}

}  // namespace ft
