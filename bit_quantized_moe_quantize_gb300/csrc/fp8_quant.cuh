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

// Two fp32 values in a 64-bit register, and packed operations on them.
__device__ __forceinline__ uint64_t pair2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}

__device__ __forceinline__ float2 split2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint64_t mad2(uint64_t a, uint64_t b, uint64_t c) {      // a * b + c, rounded once
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint64_t same2(float x) { return pair2(x, x); }

__device__ __forceinline__ float ex2_approx(float x) {      // within 2^-22 of 2^x; 0 below 2^-126
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
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

// The gated activation of one value: act(g) * up with act(g) = g / (1 + exp(-z)), z = g for
// SiLU and 2 sqrt(2/pi) (g + 0.044715 g^3) for the tanh form of GELU.  Every operation is the
// IEEE one, and expf, so that codes and scales are the formula's in fp32 bit for bit.
__device__ __forceinline__ float act_mul_f32(float g, float up, int kind) {
    const float cube = __fmul_rn(__fmul_rn(__fmul_rn(0.044715f, g), g), g);
    const float z = kind == FT_ACT_SILU ? g : __fmul_rn(1.5957691216057308f, __fadd_rn(g, cube));
    return __fmul_rn(__fdiv_rn(g, __fadd_rn(1.0f, expf(-z))), up);
}

// The same of 2 N values within some 10 * 2^-24 of their size, for the epilogue of the wide
// products, whose drain warps have the tensor cores wait: with act_mul_f32 a layer of 8192 tokens
// takes 105 us more than its 538, and to write the product's rows and read them again some 70 more.
//
// exp(-z) = 2^-t exp(-c) with t the rounded z log2(e) and c = z - t ln 2 what that rounding left
// out (ln 2 in two parts), at most 2^-17 while 2^-t is finite, so that 1 - c stands for exp(-c).
// Without c the exponential is off by 2^-24 |z| of itself.  A quarter of 1 + exp(-z) keeps
// its reciprocal a normal number as long as exp(-z) is finite; past that act(g) is 0.
template <int N>
__device__ __forceinline__ void act_mul_pairs(const uint64_t (&g)[N], const uint64_t (&up)[N], int kind, uint64_t (&out)[N]) {
    uint64_t z[N];
    float far = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        z[i] = g[i];
        if (kind != FT_ACT_SILU) {
            const uint64_t cube = mul2(mul2(mul2(same2(0.044715f), g[i]), g[i]), g[i]);
            z[i] = mul2(same2(1.5957691216057308f), add2(g[i], cube));
        }
        const float2 a = split2(z[i]);
        far = max_nan(far, fabsf(a.x), fabsf(a.y));
    }
    if (!(far < 0x1p20f)) {      // (as far out nothing changes any more, but products overflow)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float2 a = split2(z[i]);
            z[i] = pair2(fminf(fmaxf(a.x, -128.0f), 128.0f), fminf(fmaxf(a.y, -128.0f), 128.0f));
        }
    }
    constexpr float kLn2Hi = 0.693147182f, kLn2Lo = -1.90465421e-9f;      // ln 2 = kLn2Hi + kLn2Lo
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint64_t t = mul2(z[i], same2(1.4426950408889634f));
        const uint64_t c = mad2(t, same2(-kLn2Lo), mad2(t, same2(-kLn2Hi), z[i]));
        const float2 ts = split2(t);
        const uint64_t e = pair2(ex2_approx(-ts.x), ex2_approx(-ts.y));
        const float2 d = split2(mad2(e, mad2(c, same2(-0.25f), same2(0.25f)), same2(0.25f)));
        out[i] = mul2(mul2(mul2(g[i], same2(0.25f)), pair2(rcp_approx(d.x), rcp_approx(d.y))), up[i]);
    }
}

__device__ __forceinline__ uint32_t e4m3x4(uint64_t a, uint64_t b) {
    const float2 x = split2(a), y = split2(b);
    return e4m3x4(x.x, x.y, y.x, y.y);
}

// Codes of v / scale for eight values; inv: rcp_approx(scale).  y = v * inv lies within
// 2^-22 |v / scale| of the IEEE quotient (2^-23 of the reciprocal, 2^-24 of the product and of
// the quotient), so both round to the same code unless y (1 - 2^-21) and y (1 + 2^-21) do not;
// only then, or where 1 / scale could overflow, are the quotients formed.
__device__ __forceinline__ uint2 fp8_codes(const uint64_t (&v)[4], float scale, float inv) {
    const uint64_t inv2 = same2(inv), down = same2(1.0f - 0x1p-21f), up = same2(1.0f + 0x1p-21f);
    uint32_t lo[2], hi[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint64_t a = mul2(v[2 * h], inv2), b = mul2(v[2 * h + 1], inv2);
        lo[h] = e4m3x4(mul2(a, down), mul2(b, down));
        hi[h] = e4m3x4(mul2(a, up), mul2(b, up));
    }
    if (lo[0] != hi[0] || lo[1] != hi[1] || !(scale > 1.0e-36f)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float2 x = split2(v[2 * h]), y = split2(v[2 * h + 1]);
            lo[h] = scale == 0.0f ? 0u
                                  : e4m3x4(__fdiv_rn(x.x, scale), __fdiv_rn(x.y, scale), __fdiv_rn(y.x, scale), __fdiv_rn(y.y, scale));
        }
    }
    return make_uint2(lo[0], lo[1]);
}

__device__ __forceinline__ uint2 fp8_codes(const float (&v)[8], float scale, float inv) {
    const uint64_t p[4] = {pair2(v[0], v[1]), pair2(v[2], v[3]), pair2(v[4], v[5]), pair2(v[6], v[7])};
    return fp8_codes(p, scale, inv);
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
