// fp4.cuh - microscaled 4-bit floating point: elements of e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6
// and their negatives, two to a byte, the even element in the low nibble) that share a
// scale in blocks along the contraction.
//   mx: blocks of 32, scale 2^(c - 127) (ue8m0, c = 255: NaN). 2^(floor(log2 amax) - 2).
//   nv: blocks of 16, scale ue4m3, amax / (6 g) to the nearest; the values are
//       element * scale * g with g one fp32 number for a whole matrix.
// Scales lie as the block-scaled tcgen05 instructions take them: tiles of 128 rows x 4
// blocks, 512 bytes each, the tiles of a 128-row group in order of their blocks; in a tile
// row r's four bytes are at 16 (r % 32) + 4 (r / 32).
#pragma once

#include <stdint.h>

#include "ep_device.cuh"

namespace ep {

constexpr int kFp4Mx = 0, kFp4Nv = 1;

namespace {

template <int FMT>
struct Fp4 {
    static constexpr int kBlock = FMT == kFp4Mx ? 32 : 16;
};

// Offset of the scales of row `row` and blocks [4 kt, 4 kt + 4); tiles: tiles in a row.
__device__ __forceinline__ int64_t fp4_scale_at(int64_t row, int64_t kt, int64_t tiles)
{
    return ((row >> 7) * tiles + kt) * 512 + ((row & 31) << 4) + (((row >> 5) & 3) << 2);
}

// Two fp32 to two e2m1 in a byte (lo in the low nibble), nearest even, at most 6.
__device__ __forceinline__ uint32_t cvt_e2m1x2(float lo, float hi)
{
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\t"
        "cvt.u32.u8 %0, t;\n\t}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}

// Eight fp32 to the word of their e2m1.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float* v)
{
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// 1 / v within an ulp or two (rcp.approx), which is all that quotients for rounding need.
__device__ __forceinline__ float rcp_near(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// The two values of the byte's two e2m1, as two fp16 (the low nibble's in the low half).
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t byte)
{
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\t"
        "cvt.u8.u32 t, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, t;\n\t}"
        : "=r"(r)
        : "r"(byte));
    return r;
}

// The eight of a word.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t word, uint32_t (&h2)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h2[0]), "=r"(h2[1]), "=r"(h2[2]), "=r"(h2[3])
        : "r"(word));
}

__device__ __forceinline__ float f16_lo(uint32_t h2)
{
    float f;
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, a;\n\t}" : "=f"(f) : "r"(h2));
    return f;
}

__device__ __forceinline__ float f16_hi(uint32_t h2)
{
    float f;
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, b;\n\t}" : "=f"(f) : "r"(h2));
    return f;
}

// ue4m3 of a non-negative number (nearest even, at most 448), and its value.
__device__ __forceinline__ uint32_t cvt_ue4m3(float v)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
    return r & 0xFFu;
}

__device__ __forceinline__ float ue4m3_value(uint32_t c)
{
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)c));
    return f16_lo(h2);
}

__device__ __forceinline__ float ue8m0_value(uint32_t c)
{
    return __uint_as_float(c == 0u ? 0x00400000u : c == 255u ? 0x7FC00000u : c << 23);
}

constexpr uint32_t kNanMx = 0xFFu, kNanNv = 0x7Fu, kLargestNv = 0x7Eu;

// x / (d g) near enough to round it to a format of few bits: what an fp32 product with the
// reciprocal gives, except next to a number of at most BITS fraction bits (the borders
// between the format's numbers are such), where the remainder x - q d g decides, whose sign
// one fma gives exactly: the quotient then lies on the border or on the right side of it.
// d: few bits (a scale, or 6), so that q d is exact. rinv: 1 / (d g), off by 2^-22 at most, so that
// x rinv is within 2^-21 and a number within 2^-20 of a border is looked at.
template <int BITS>
__device__ __forceinline__ float quotient_for_rounding(float x, float d, float g, float rinv)
{
    const float q0 = x * rinv;
    const float qr = __uint_as_float((__float_as_uint(q0) + 8u) & ~15u);
    const bool border = (__float_as_uint(qr) & ((1u << (23 - BITS)) - 1u)) == 0u;
    const float rest = __fmaf_rn(-(qr * d), g, x);
    // 2^10 times the remainder: out of reach of the sum's own rounding, and still within
    // 2^-9 of the border.
    return border ? __fmaf_rn(rest, rinv * 1024.0f, qr) : q0;
}

// Numbers below and above a quotient that an fp32 product with a reciprocal off by 2^-22 gives: if
// both round to the same code, so does the quotient itself, and only else has it to be looked at.
constexpr float kBelow = 1.0f - 0x1p-20f, kAbove = 1.0f + 0x1p-20f;

// The block's scale code from the largest magnitude in it (not NaN: then, and for an
// infinity, the code is the NaN). g: the matrix's scale, 1 without one.
template <int FMT>
__device__ __forceinline__ uint32_t fp4_scale_code(float amax, float g)
{
    if (FMT == kFp4Mx) {
        const uint32_t e = __float_as_uint(amax) >> 23;
        return e == 255u ? kNanMx : e < 2u ? 0u : e - 2u;
    }
    if (!(amax < __uint_as_float(0x7F800000u))) return kNanNv;
    if (amax == 0.0f) return 0u;   // g may be 0 for a matrix of zeros
    const float rinv = rcp_near(6.0f * g);
    uint16_t both;   // what lies a little below the quotient and a little above it round to
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(both)
        : "f"(amax * (rinv * kAbove)), "f"(amax * (rinv * kBelow)));
    if ((both >> 8) == (both & 0xFF)) return both & 0xFFu;
    return cvt_ue4m3(quotient_for_rounding<4>(amax, 6.0f, g, rinv));
}

// (a, b) * (m, m) in one instruction.
__device__ __forceinline__ void mul2(float a, float b, float m, float& x, float& y)
{
    asm("{\n\t.reg .b64 p, q;\n\t"
        "mov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %4};\n\t"
        "mul.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "=f"(x), "=f"(y)
        : "f"(a), "f"(b), "f"(m));
}

// Codes of 16 elements in a block with scale code c.
template <int FMT, bool TENSOR_SCALE>
__device__ __forceinline__ uint2 fp4_codes16(const float (&v)[16], uint32_t c, float g)
{
    float q[16];
    if (FMT == kFp4Mx) {
        if (c == kNanMx) return make_uint2(0u, 0u);
        const float inv = __uint_as_float((254u - c) << 23);   // 2^(127 - c), c <= 252
#pragma unroll
        for (int i = 0; i < 16; i += 2) mul2(v[i], v[i + 1], inv, q[i], q[i + 1]);
        return make_uint2(cvt_e2m1x8(q), cvt_e2m1x8(q + 8));
    }
    if (c == kNanNv || c == 0u) return make_uint2(0u, 0u);
    const float s = ue4m3_value(c);
    const float rinv = rcp_near(s * g);
    if (TENSOR_SCALE) {
        const float lo = rinv * kBelow, hi = rinv * kAbove;
        uint32_t w[2], differ = 0u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float below[8], above[8];
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                mul2(v[8 * h + i], v[8 * h + i + 1], lo, below[i], below[i + 1]);
                mul2(v[8 * h + i], v[8 * h + i + 1], hi, above[i], above[i + 1]);
            }
            w[h] = cvt_e2m1x8(below);
            differ |= w[h] ^ cvt_e2m1x8(above);
        }
        if (differ == 0u) return make_uint2(w[0], w[1]);
        // Some element lies next to a border. In a block whose scale is the largest there is, elements
        // may be anything above the grid, up to quotients that overflow and leave no sign.
        float near[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) near[i] = v[i];
        if (c == kLargestNv) {
            const float far = 1024.0f * s * g;
#pragma unroll
            for (int i = 0; i < 16; ++i) near[i] = fminf(fmaxf(v[i], -far), far);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) q[i] = quotient_for_rounding<2>(near[i], s, g, rinv);
    } else {
        // x has 8 bits and s 4: the quotient is on a border or 2^-12 away from it, and its last
        // bits are the reciprocal's.
#pragma unroll
        for (int i = 0; i < 16; i += 2) mul2(v[i], v[i + 1], rinv, q[i], q[i + 1]);
#pragma unroll
        for (int i = 0; i < 16; ++i) q[i] = __uint_as_float((__float_as_uint(q[i]) + 8u) & ~15u);
    }
    return make_uint2(cvt_e2m1x8(q), cvt_e2m1x8(q + 8));
}

// 16 bf16 (32 bytes) as fp32.
__device__ __forceinline__ void bf16x16(const int4& a, const int4& b, float (&v)[16])
{
    const uint32_t q[8] = {(uint32_t)a.x, (uint32_t)a.y, (uint32_t)a.z, (uint32_t)a.w,
                           (uint32_t)b.x, (uint32_t)b.y, (uint32_t)b.z, (uint32_t)b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[2 * i] = __uint_as_float(q[i] << 16);
        v[2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u);
    }
}

// Largest magnitude of 8 or 16 bf16, as they lie: as integers, in which NaN is above infinity.
__device__ __forceinline__ float amax8(const int4& a)
{
    const uint32_t m =
        __vmaxu2(__vmaxu2((uint32_t)a.x & 0x7FFF7FFFu, (uint32_t)a.y & 0x7FFF7FFFu),
                 __vmaxu2((uint32_t)a.z & 0x7FFF7FFFu, (uint32_t)a.w & 0x7FFF7FFFu));
    return __uint_as_float(max(m << 16, m & 0xFFFF0000u));
}

__device__ __forceinline__ float amax16(const int4& a, const int4& b)
{
    return __uint_as_float(max(__float_as_uint(amax8(a)), __float_as_uint(amax8(b))));
}

// The same of 16 fp32.
__device__ __forceinline__ float amax16(const float (&v)[16])
{
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    return __uint_as_float(m);
}

}  // namespace
}  // namespace ep
