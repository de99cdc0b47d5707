// Online softmax of a 128 x 128 score tile by a warpgroup whose threads own one row (tensor-memory lane)
// each, for the cross attention kernel.
#pragma once
#include <cuda_bf16.h>

#include <cmath>

#include "ptx.cuh"

namespace sdv2 {

constexpr float kGrowLog2 = 8.0f;      // the running max follows when a score exceeds it by more than 2^8

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// (a.lo*b.lo, a.hi*b.hi), each rounded once.
__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Columns at and past `valid` become -infinity.
__device__ __forceinline__ void mask_columns(uint32_t (&r)[32], int valid)
{
#pragma unroll
    for (int i = 0; i < 32; ++i)
        if (i >= valid) r[i] = 0xFF800000u;
}

// One step of the online softmax: reads the scores at tS, writes P as packed bf16 over their first 64
// columns, and rescales the row's accumulator at tO (128 columns) when the running max has to follow;
// `first` says that there is none yet.  m and l are the row's running max (log2 units) and sum.
// P is rounded to bf16 (by 2^-8 of itself at most) because the tensor cores take both operands of P V in one type, and
// V is bf16; the sum is taken of the probabilities before that.  Against 64 bits the output is off by 0.0022 in the
// 2-norm (4680 x 12 x 512), 0.0017 of which is its own rounding.
// Warp-collective.  The row is read twice, for its max and for the exponentials, in loops that are kept
// short: a prompt has few key tiles, and code that runs a few times costs more to fetch than to execute.
// (1.3B 480p chunk, 512 states: 20.7 us; one unrolled pass over 128 registers 25.8 us, unrolled quarters
// that guess the max 24.8 us.)
__device__ __forceinline__ void softmax_step(uint32_t tS, uint32_t tO, float sl2, int valid, bool first, float& m, float& l)
{
    float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
        uint32_t r[32];
        tmem_ld_x32_sync(tS + 32 * q, r);
        if (valid < 32 * (q + 1)) mask_columns(r, valid - 32 * q);
#pragma unroll
        for (int i = 0; i < 32; i += 8)
#pragma unroll
            for (int a = 0; a < 4; ++a) mx4[a] = fmax3(mx4[a], __uint_as_float(r[i + a]), __uint_as_float(r[i + 4 + a]));
    }
    const float m_new = fmaxf(m, fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sl2);
    const bool grow = m_new > m + kGrowLog2;
    if (__any_sync(0xffffffffu, grow)) {
        const float f = grow ? ex2_approx(m - m_new) : 1.0f;
        if (!first) {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t o[32];
                tmem_ld_x32_sync(tO + c * 32, o);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_st_x32(tO + c * 32, o);
            }
        }
        if (grow) {
            l *= f;
            m = m_new;
        }
    }
    // scores that have all been -infinity so far (keys of the type's lowest value) leave a max of -infinity: 2^(x - 0) is 0
    const float base = m == -INFINITY ? 0.f : m;
    const uint64_t sl2x2 = f32x2_pack(sl2, sl2), negm2 = f32x2_pack(-base, -base);
    uint64_t sum4[4] = {0, 0, 0, 0};
#pragma unroll 1
    for (int q = 0; q < 2; ++q) {
        uint32_t pk[32];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t r[32];
            tmem_ld_x32_sync(tS + 64 * q + 32 * h, r);
            if (valid < 64 * q + 32 * h + 32) mask_columns(r, valid - 64 * q - 32 * h);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint64_t x = ffma2(f32x2_pack(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), sl2x2, negm2);
                float x0, x1;
                f32x2_unpack(x, x0, x1);
                const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                sum4[i & 3] = fadd2(sum4[i & 3], f32x2_pack(p0, p1));
                pk[h * 16 + i] = bf16_pair(p0, p1);
            }
        }
        tmem_st_x32(tS + 32 * q, pk);
    }
    float lo, hi;
    f32x2_unpack(fadd2(fadd2(sum4[0], sum4[1]), fadd2(sum4[2], sum4[3])), lo, hi);
    l += lo + hi;
}

}  // namespace sdv2
