// Numbers of a microscaled 4-bit matrix: e2m1 codes, and scales as biased exponents of two.
#pragma once
#include <cuda_fp16.h>
#include <cstdint>

#include "ptx.cuh"

namespace sdv2 {

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// The largest of three magnitudes; NaN if one is.
__device__ __forceinline__ float max_size(float a, float b, float c)
{
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The scale's byte of a block whose largest magnitude has the bits `amax` (as fp32): the least e with
// amax <= 7 * 2^e, plus 127.  With amax = 1.m * 2^(E - 127) that is E - 2, and one more where 1.m > 1.75, which a carry out
// of the mantissa gives; infinities and NaN (whose bits compare above all others) give 255.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t amax)
{
    const int e = static_cast<int>((amax + 0x1FFFFFu) >> 23) - 2;
    return amax >= 0x7F800000u ? 255u : static_cast<uint32_t>(e > 0 ? e : 0);
}

// 2^-e of a scale's byte, by which the block's numbers are multiplied (exactly; 0 for NaN, whose codes do not matter).
__device__ __forceinline__ float mx4_inverse(uint32_t byte) { return __uint_as_float(byte == 255u ? 0u : (254u - byte) << 23); }

// 2^e of a scale's byte.
__device__ __forceinline__ float mx4_scale(uint32_t byte)
{
    return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255u ? 0x7FC00000u : byte << 23);
}

// Eight numbers to their nearest codes, the first in the lowest bits; middles go to even codes, sizes above 6 to 6.
__device__ __forceinline__ uint32_t mx4_codes(const float (&x)[8])
{
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

// The eight numbers of four bytes of codes, without their scale.
__device__ __forceinline__ void mx4_numbers(uint32_t codes, __half2 (&x)[4])
{
    uint32_t r[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(codes));
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<__half2*>(&r[i]);
}

// y/2 * (1 + tanh(u)), u = sqrt(2/pi) * (y + 0.044715 y^3), as y / (1 + exp(-2u)), of two numbers.  One reciprocal serves both:
// that of the product of the two divisors, which stays below 2^112 because y is taken to be at least -7.2 (the result there,
// -2^-52, stands for all smaller ones).  Two exponentials and a reciprocal leave the MUFU pipe 1.5 operations a number.
__device__ __forceinline__ uint64_t gelu2(uint64_t y)
{
    constexpr float k = -2.0f * 0.7978845608028654f * 1.4426950408889634f;
    float a, b;
    f32x2_unpack(y, a, b);
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(-7.2f));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(b) : "f"(-7.2f));
    y = f32x2_pack(a, b);
    const uint64_t z = mul2(y, ffma2(mul2(y, y), f32x2_pack(k * 0.044715f, k * 0.044715f), f32x2_pack(k, k)));
    f32x2_unpack(z, a, b);
    a = fmaxf(1.0f + ex2_approx(a), 1.0f);           // (1 for NaN, which then reaches its own result only)
    b = fmaxf(1.0f + ex2_approx(b), 1.0f);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a * b));
    return mul2(y, mul2(f32x2_pack(r, r), f32x2_pack(b, a)));
}

__device__ __forceinline__ float gelu(float y)
{
    float a, b;
    f32x2_unpack(gelu2(f32x2_pack(y, 0.0f)), a, b);
    return a;
}

}  // namespace sdv2
