// Numbers of a microscaled 4-bit matrix: e2m1 codes, and scales as biased exponents of two.
#pragma once
#include <cuda_fp16.h>
#include <cstdint>

namespace sdv2 {

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

// y/2 * (1 + tanh(u)), u = sqrt(2/pi) * (y + 0.044715 y^3), as y / (1 + exp(-2u)).
__device__ __forceinline__ float gelu(float y)
{
    constexpr float c = -2.0f * 0.7978845608028654f;
    const float e = __expf(y * fmaf(c * 0.044715f, y * y, c));
    return __fdividef(y, 1.0f + e);
}

}  // namespace sdv2
