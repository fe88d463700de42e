// Scales and codes of the 8-bit blocks and of the NVFP4 rows, shared by the quantisers.
#pragma once

#include "common.cuh"

namespace nvfp4 {

namespace {

constexpr float kE4m3Max = 448.0f;

// Below this amax 448 / amax could overflow: the block is first brought up by 2^64, exactly.
constexpr float kTinyAmax = 0x1p-100f;

__device__ __forceinline__ float block_scale(uint32_t amax_bits) {
    return amax_bits == 0u ? 1.0f : __uint_as_float(amax_bits) / kE4m3Max;
}
// 448 / amax, of a tiny block 448 / (2^64 amax).
__device__ __forceinline__ float block_inverse(uint32_t amax_bits) {
    const float a = __uint_as_float(amax_bits);
    return amax_bits == 0u ? 1.0f : kE4m3Max / (a < kTinyAmax ? a * 0x1p64f : a);
}

// p rounded to 16 significant bits. In a block with infinities or NaN nothing is added (half 0), so
// that the quotient's NaN does not wrap into a number.
__device__ __forceinline__ float snap16(float p, uint32_t half) {
    return __uint_as_float((__float_as_uint(p) + half) & 0xFFFFFF00u);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// ---------------------------------------------------------------- NVFP4 rows
// Row scale of a row with this largest magnitude (fp32 bits): the smallest power of two >= a / 2688, at least
// 2^-126; 1 for zeros, NaN for a row that is not finite. A bf16 a / 2688 is a power of two exactly or at least
// 1/168 away from one, so the rounded quotient is on the right side.
__device__ __forceinline__ float row_scale(uint32_t amax_bits) {
    if (amax_bits == 0u) return 1.0f;
    if (amax_bits >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
    const uint32_t q = __float_as_uint(__fdiv_rn(__uint_as_float(amax_bits), 2688.0f));
    return __uint_as_float(max((q + 0x007FFFFFu) & 0x7F800000u, 0x00800000u));
}
// 1 / s of a power of two 2^-126 .. 2^126.
__device__ __forceinline__ float inverse_pow2(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }

// 1 / x within 2^-23.
__device__ __forceinline__ float fast_rcp(float x) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// E4M3 code of a block whose largest magnitude is b row scales, and the reciprocal of its value within 2^-23 (0 for code
// 0). EXACT: b is bf16, so that b / 6 is on a rounding point of E4M3 or off it by over 2^-13: the product with 1 / 6,
// within 2^-22 of it, goes back on the point when it is rounded to 16 bits.
template <bool EXACT>
__device__ __forceinline__ uint32_t nvfp4_block_scale(float b, float* inv) {
    const float q = b * (1.0f / 6.0f);
    const uint32_t e = e4m3x2(EXACT ? snap16(q, 0x80u) : q, 0.f) & 0xFFu;
    *inv = e == 0u ? 0.f : fast_rcp(e4m3_to_f32(e));
    return e;
}

// (a, b) *= s, each product rounded: the packed fp32 pipe.
__device__ __forceinline__ void mul2(float& a, float& b, float s) {
    asm("{\n .reg .b64 v, s;\n mov.b64 v, {%0, %1};\n mov.b64 s, {%2, %2};\n mul.rn.f32x2 v, v, s;\n"
        " mov.b64 {%0, %1}, v;\n}" : "+f"(a), "+f"(b) : "f"(s));
}

// Eight values of a block times 1 / (block scale * row scale) -> eight codes, the first in the low four bits. EXACT: the
// values are bf16, so that v / e (8 bits by at most 4) is on a rounding point of E2M1 or off it by over 2^-8: p, within
// 2^-22 of the quotient, goes back on the point when it is rounded to 16 bits.
template <bool EXACT>
__device__ __forceinline__ uint32_t nvfp4_codes8(float (&p)[8], float inv) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) mul2(p[i], p[i + 1], inv);
    if (EXACT)
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = snap16(p[i], 0x80u);
    uint32_t r;
    asm("{\n .reg .b8 a, b, c, d;\n"
        " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        " mov.b32 %0, {a, b, c, d};\n}"
        : "=r"(r) : "f"(p[0]), "f"(p[1]), "f"(p[2]), "f"(p[3]), "f"(p[4]), "f"(p[5]), "f"(p[6]), "f"(p[7]));
    return inv == 0.f ? 0u : r;
}

}  // namespace

}  // namespace nvfp4
