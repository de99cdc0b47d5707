// Online softmax of one 128 x 128 score tile by a warpgroup whose threads own one row (tensor-memory
// lane) each, for the cross attention kernel.
#pragma once
#include <cuda_bf16.h>

#include <cmath>

#include "ptx.cuh"

namespace sdv2 {

constexpr float kGrowLog2 = 8.0f;      // the running max follows when a score exceeds it by more than 2^8
constexpr float kGrowSum = 256.0f;     // a row sum up to 2^8 proves that no score did

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Columns at and past `valid` become -infinity.
__device__ __forceinline__ void mask_columns(uint32_t (&r)[128], int valid)
{
#pragma unroll
    for (int i = 0; i < 128; ++i)
        if (i >= valid) r[i] = 0xFF800000u;
}

// 64 probabilities 2^(s*sl2 - m) of columns [64*hf, 64*hf + 64) as packed bf16, and their sums in four chains.
__device__ __forceinline__ void exponentials(const uint32_t (&r)[128], int hf, uint64_t sl2x2, uint64_t negm2,
                                             uint32_t (&pk)[32], uint64_t (&sum4)[4])
{
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const int e = hf * 64 + 2 * i;
        const uint64_t x = ffma2(f32x2_pack(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), sl2x2, negm2);
        float x0, x1;
        f32x2_unpack(x, x0, x1);
        const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
        sum4[i & 3] = fadd2(sum4[i & 3], f32x2_pack(p0, p1));
        pk[i] = bf16_pair(p0, p1);
    }
}

__device__ __forceinline__ float add_chains(const uint64_t (&sum4)[4])
{
    float lo, hi;
    f32x2_unpack(fadd2(fadd2(sum4[0], sum4[1]), fadd2(sum4[2], sum4[3])), lo, hi);
    return lo + hi;
}

// One step of the online softmax: reads the scores at tS, writes P as packed bf16 over their first 64
// columns, and rescales the row's accumulator at tO (128 columns) when the running max grows; `first`
// says that there is none yet.  m and l are the row's running max (log2 units) and sum.  Warp-collective.
__device__ __forceinline__ void softmax_step(uint32_t tS, uint32_t tO, float sl2, int valid, bool first, float& m, float& l)
{
    uint32_t r[128];
    tmem_ld_x128_sync(tS, r);
    if (valid < 128) mask_columns(r, valid);
    const uint64_t sl2x2 = f32x2_pack(sl2, sl2);
    if (!first) {
        // exponentials against the running max, before this tile's own max is known: a row sum of at
        // most 2^8 proves that no score exceeds it by more than 2^8, and then it would not have moved
        const uint64_t negm2 = f32x2_pack(-m, -m);
        uint64_t sum4[4] = {0, 0, 0, 0};
        uint32_t pk[2][32];
        exponentials(r, 0, sl2x2, negm2, pk[0], sum4);
        exponentials(r, 1, sl2x2, negm2, pk[1], sum4);
        const float s = add_chains(sum4);
        if (__all_sync(0xffffffffu, s <= kGrowSum)) {
            tmem_st_x32(tS, pk[0]);
            tmem_st_x32(tS + 32, pk[1]);
            l += s;
            return;
        }
        tmem_ld_x128_sync(tS, r);
        if (valid < 128) mask_columns(r, valid);
    }
    float mx8[8];
#pragma unroll
    for (int a = 0; a < 8; ++a) {
        float x = fmax3(__uint_as_float(r[a]), __uint_as_float(r[a + 8]), __uint_as_float(r[a + 16]));
#pragma unroll
        for (int i = 24; i < 120; i += 16) x = fmax3(x, __uint_as_float(r[i + a]), __uint_as_float(r[i + 8 + a]));
        mx8[a] = fmaxf(x, __uint_as_float(r[120 + a]));
    }
    const float mx = fmaxf(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(fmax3(mx8[3], mx8[4], mx8[5]), mx8[6], mx8[7]));
    const float m_new = fmaxf(m, mx * sl2);
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
    const uint64_t negm2 = f32x2_pack(-m, -m);
    uint64_t sum4[4] = {0, 0, 0, 0};
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
        uint32_t pk[32];
        exponentials(r, hf, sl2x2, negm2, pk, sum4);
        tmem_st_x32(tS + hf * 32, pk);
    }
    l += add_chains(sum4);
}

}  // namespace sdv2
