// Products of a few rows with a 4-bit matrix: out[m][n] = act(sum_k a[m][k] b[n][k] + bias[n]) for at most 32 rows of a.
//
// Every byte of b is read once and takes part in few operations, so that reading b bounds this, and at small sizes the latency of
// a launch.  tcgen05's tiles would leave most SMs idle at the depths and widths of a layer; here a block takes 16 rows of b, whose
// warps share out the depth, and multiplies with mma.sync m16n8k16: rows of b by up to 8, 16 or 32 rows of a, both decoded to fp16,
// which holds every e2m1 number.  A thread's four bytes of a row are 8 columns, and any order of the columns will do as long as
// both operands have it: two MMAs take a block of 32, whose sum is exact (products are multiples of 1/4 up to 36).  It is scaled
// by the power of two of its row and its column and added up in fp32.
// The 16 rows are 4 neighbours and those 32, 64 and 96 behind them: their scales lie together, 64 bytes a tile of 128 columns.
#include <cuda_bf16.h>

#include <algorithm>

#include "chained.cuh"
#include "mx4.cuh"
#include "project.h"

namespace sdv2 {
namespace {

constexpr int kMaxWarps = 8;
constexpr int kTogether = 2;               // tiles of a warp whose loads are under way together

__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void decode(uint32_t codes, uint32_t (&x)[4])
{
    __half2 h[4];
    mx4_numbers(codes, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<uint32_t*>(&h[i]);
}

__device__ __forceinline__ int byte_of(uint32_t word, int i) { return static_cast<int>((word >> (8 * i)) & 255u); }

// NT: groups of 8 rows of a
template <int NT>
__global__ void __launch_bounds__(32 * kMaxWarps) rows_kernel(const Mx4Product p)
{
    constexpr int COLS = 8 * NT;
    __shared__ float sums[kMaxWarps][16 * COLS];
    wait_for_launch_before();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int g = lane >> 2, t = lane & 3, M = static_cast<int>(p.M);
    const int64_t row_tile = blockIdx.x >> 3;
    const int q0 = static_cast<int>(blockIdx.x & 7) * 4;
    const int64_t pitch = static_cast<int64_t>(p.tiles) * kMx4TileBytes;
    // rows g and g + 8 of the block's
    const uint8_t* b[2];
    const uint8_t* bs[2];
    bool have[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = g + 8 * h, in_tile = q0 + (i & 3) + 32 * (i >> 2);
        const int64_t n = row_tile * kMx4Tile + in_tile;
        have[h] = n < p.N;
        b[h] = p.b + (have[h] ? n : 0) * pitch + t * 4;
        bs[h] = p.bs + row_tile * p.tiles * 512 + (in_tile & 31) * 16 + (in_tile >> 5) * 4;
    }
    float acc[NT][4] = {};
    bool nan_b[2] = {}, nan_a[NT][2] = {};
    for (int k0 = warp; k0 < p.tiles; k0 += kTogether * warps) {
        uint32_t bc[kTogether][2][4], bw[kTogether][2], ac[kTogether][NT][4], aw[kTogether][NT][2];
#pragma unroll
        for (int u = 0; u < kTogether; ++u) {
            const int k = k0 + u * warps;
            const bool in = k < p.tiles;
            const int64_t at = static_cast<int64_t>(k) * kMx4TileBytes, scale_at = static_cast<int64_t>(k) * 512;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                bw[u][h] = in && have[h] ? *reinterpret_cast<const uint32_t*>(bs[h] + scale_at) : 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) bc[u][h][j] = in && have[h] ? *reinterpret_cast<const uint32_t*>(b[h] + at + j * 16) : 0;
            }
#pragma unroll
            for (int c = 0; c < NT; ++c) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int m = 8 * c + 2 * t + h;
                    aw[u][c][h] = in && m < M ? *reinterpret_cast<const uint32_t*>(p.as + scale_at + m * 16) : 0;
                }
                const int m = 8 * c + g;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    ac[u][c][j] = in && m < M ? *reinterpret_cast<const uint32_t*>(p.a + m * pitch + at + t * 4 + j * 16) : 0;
            }
        }
#pragma unroll
        for (int u = 0; u < kTogether; ++u) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                nan_b[h] |= __vcmpeq4(bw[u][h], 0xFFFFFFFFu) != 0;
#pragma unroll
                for (int c = 0; c < NT; ++c) nan_a[c][h] |= __vcmpeq4(aw[u][c][h], 0xFFFFFFFFu) != 0;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t x0[4], x1[4];
                decode(bc[u][0][j], x0);
                decode(bc[u][1][j], x1);
#pragma unroll
                for (int c = 0; c < NT; ++c) {
                    uint32_t y[4];
                    decode(ac[u][c][j], y);
                    float s[4] = {};
                    mma_16x8x16(s, x0[0], x1[0], x0[1], x1[1], y[0], y[1]);
                    mma_16x8x16(s, x0[2], x1[2], x0[3], x1[3], y[2], y[3]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        // 2^(eb + ea), 0 below fp32's normal numbers and 2^127 above them
                        const int e = byte_of(bw[u][i >> 1], j) + byte_of(aw[u][c][i & 1], j) - 127;
                        acc[c][i] = fmaf(s[i], __uint_as_float(static_cast<uint32_t>(min(max(e, 0), 254)) << 23), acc[c][i]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool bad = nan_b[i >> 1] || nan_a[c][i & 1];
            sums[warp][(g + 8 * (i >> 1)) * COLS + 8 * c + 2 * t + (i & 1)] = bad ? __uint_as_float(0x7FC00000u) : acc[c][i];
        }
    __syncthreads();
    for (int o = threadIdx.x; o < 16 * M; o += blockDim.x) {
        const int m = o >> 4, i = o & 15;
        const int64_t n = row_tile * kMx4Tile + q0 + (i & 3) + 32 * (i >> 2);
        if (n >= p.N) continue;
        float y = sums[0][i * COLS + m];
        for (int w = 1; w < warps; ++w) y += sums[w][i * COLS + m];
        if (p.bias) y += p.bias[n];
        if (p.gelu) y = gelu(y);
        const int64_t at = m * p.out_stride + n;
        if (p.out_f32) static_cast<float*>(p.out)[at] = y;
        else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(y);
    }
}

}  // namespace

cudaError_t launch_mx4_rows(const Mx4Product& p, cudaStream_t s)
{
    const int warps = std::min(kMaxWarps, (p.tiles + kTogether - 1) / kTogether);
    const unsigned grid = static_cast<unsigned>((p.N + kMx4Tile - 1) / kMx4Tile * 8);
    auto kernel = p.M <= 8 ? rows_kernel<1> : p.M <= 16 ? rows_kernel<2> : rows_kernel<4>;
    return launch_chained(kernel, grid, 32 * warps, 0, s, p);
}

}  // namespace sdv2
