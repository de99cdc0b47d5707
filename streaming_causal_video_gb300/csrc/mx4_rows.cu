// Products of a few rows with a 4-bit matrix, on the CUDA cores.
//
// out[m][n] = act(sum_k a[m][k] b[n][k] + bias[n]) for at most eight rows of a.  Every byte of b is read once and takes part
// in few operations, so that reading b, or at small sizes the latency of a launch, bounds this.  A block owns the four rows
// n = 128 t + r + 32 i of b whose scales share 16 bytes; each lane of its warps takes a block of 32 columns, which has one
// scale for each of them: 16 bytes of codes of every row in one load.
// The sum of a block's 32 products is exact: products of two e2m1 numbers are multiples of 1/4 up to 36, so that 8 of them
// in a lane of a half2 stay below 2^11 quarters.  It is scaled and added up in fp32.
#include <cuda_bf16.h>

#include <algorithm>

#include "chained.cuh"
#include "mx4.cuh"
#include "project.h"

namespace sdv2 {
namespace {

constexpr int kMaxWarps = 8;

__device__ __forceinline__ void numbers32(uint4 codes, __half2 (&x)[16])
{
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __half2 h[4];
        mx4_numbers(w[i], h);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[4 * i + j] = h[j];
    }
}

// V values of every lane to the sums over the warp: lane l is left with that of value (l >> (5 - log2 V)), in v[0].
template <int V>
__device__ __forceinline__ void sum_lanes(float (&v)[V])
{
    const int lane = threadIdx.x & 31;
    int have = V;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        if (have > 1) {
            have >>= 1;
            const bool upper = (lane & d) != 0;
#pragma unroll
            for (int i = 0; i < V / 2; ++i)
                if (i < have) {
                    const float give = upper ? v[i] : v[i + have];
                    const float keep = upper ? v[i + have] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, d);
                }
        } else {
            v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], d);
        }
    }
}

// R: rows of a that a thread has accumulators for, M <= R.
template <int R>
__global__ void __launch_bounds__(32 * kMaxWarps) rows_kernel(const Mx4Product p)
{
    constexpr int V = 4 * R;
    __shared__ float sums[kMaxWarps][V];
    wait_for_launch_before();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x >> 5) * 128 + (blockIdx.x & 31);     // rows n0 + 32 i of b
    const uint8_t* bs = p.bs + static_cast<int64_t>(blockIdx.x >> 5) * p.tiles * 512 + (blockIdx.x & 31) * 16;
    const int64_t pitch = static_cast<int64_t>(p.tiles) * kMx4TileBytes;
    const int blocks = p.tiles * 4, M = static_cast<int>(p.M);
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    for (int kb = warp * 32 + lane; kb < blocks; kb += warps * 32) {
        const int at = kb & 3;
        const uint4 scale4 = *reinterpret_cast<const uint4*>(bs + static_cast<int64_t>(kb >> 2) * 512);
        const uint32_t scales[4] = {scale4.x, scale4.y, scale4.z, scale4.w};
        uint4 bc[4], ac[R];
        uint32_t ab[R];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            bc[i] = n0 + 32 * i < p.N ? *reinterpret_cast<const uint4*>(p.b + (n0 + 32 * i) * pitch + kb * int64_t(16)) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int m = 0; m < R; ++m) {
            ac[m] = make_uint4(0, 0, 0, 0);
            ab[m] = 0;
            if (m < M) {
                ac[m] = *reinterpret_cast<const uint4*>(p.a + m * pitch + kb * int64_t(16));
                ab[m] = p.as[static_cast<int64_t>(kb >> 2) * 512 + m * 16 + at];
            }
        }
        __half2 b[4][16];
#pragma unroll
        for (int i = 0; i < 4; ++i) numbers32(bc[i], b[i]);
#pragma unroll
        for (int m = 0; m < R; ++m) {
            if (m >= M) break;
            __half2 a[16];
            numbers32(ac[m], a);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t bb = (scales[i] >> (8 * at)) & 255u;
                __half2 s0 = __hmul2(a[0], b[i][0]), s1 = __hmul2(a[8], b[i][8]);
#pragma unroll
                for (int j = 1; j < 8; ++j) {
                    s0 = __hfma2(a[j], b[i][j], s0);
                    s1 = __hfma2(a[j + 8], b[i][j + 8], s1);
                }
                const float2 f0 = __half22float2(s0), f1 = __half22float2(s1);
                const float dot = (f0.x + f0.y) + (f1.x + f1.y);
                // 2^(ea + eb) as two factors, neither of which leaves fp32's range before the product does
                const int e = static_cast<int>(ab[m] + bb) - 254;
                const int half = e >> 1;
                float scaled = dot * __uint_as_float(static_cast<uint32_t>(max(half + 127, 1)) << 23) *
                               __uint_as_float(static_cast<uint32_t>(max(e - half + 127, 1)) << 23);
                if (max(ab[m], bb) == 255u) scaled = __uint_as_float(0x7FC00000u);
                acc[4 * m + i] += scaled;
            }
        }
    }
    sum_lanes<V>(acc);
    if ((lane & (32 / V - 1)) == 0) sums[warp][lane / (32 / V)] = acc[0];
    __syncthreads();
    const int m = threadIdx.x >> 2;
    const int64_t n = n0 + 32 * (threadIdx.x & 3);
    if (m >= M || n >= p.N) return;
    float y = sums[0][threadIdx.x];
    for (int w = 1; w < warps; ++w) y += sums[w][threadIdx.x];
    if (p.bias) y += p.bias[n];
    if (p.gelu) y = gelu(y);
    const int64_t o = m * p.out_stride + n;
    if (p.out_f32) static_cast<float*>(p.out)[o] = y;
    else static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(y);
}

}  // namespace

cudaError_t launch_mx4_rows(const Mx4Product& p, cudaStream_t s)
{
    // a warp for every 32 blocks of columns, so that a block's loads are all under way at once
    const int warps = std::min(kMaxWarps, (p.tiles * 4 + 31) / 32);
    const unsigned grid = static_cast<unsigned>((p.N + 127) / 128 * 32);
    auto kernel = p.M == 1 ? rows_kernel<1> : p.M == 2 ? rows_kernel<2> : p.M <= 4 ? rows_kernel<4> : rows_kernel<8>;
    return launch_chained(kernel, grid, 32 * warps, 0, s, p);
}

}  // namespace sdv2
