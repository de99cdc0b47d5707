// Matrices to and from microscaled 4-bit numbers.
#include <cuda_bf16.h>

#include <algorithm>

#include "chained.cuh"
#include "mx4.cuh"
#include "project.h"

namespace sdv2 {
namespace {

constexpr int kThreads = 256;
constexpr int kGroups = kThreads / 16;     // 16 threads take a tile of a row: 128 numbers, 8 each

__device__ __forceinline__ int64_t scale_offset(int64_t row, int tile, int tiles)
{
    return ((row >> 7) * tiles + tile) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}

// Row and tile of a thread's units, which lie `step` units apart.
struct Units {
    int64_t row;
    int tile;
    int tiles, step_rows, step_tiles;
    __device__ __forceinline__ Units(int64_t first, int tiles_, int step) : tiles(tiles_)
    {
        row = first / tiles_;
        tile = static_cast<int>(first - row * tiles_);
        step_rows = step / tiles_;
        step_tiles = step - step_rows * tiles_;
    }
    __device__ __forceinline__ void next()
    {
        row += step_rows;
        tile += step_tiles;
        if (tile >= tiles) {
            tile -= tiles;
            ++row;
        }
    }
};

// Eight numbers from column c of a row of `cols` columns, zeros behind its end.
template <bool F32>
__device__ __forceinline__ void load8(const void* row, int64_t c, int64_t cols, bool vectors, float (&x)[8])
{
    if (vectors && c + 8 <= cols) {
        if constexpr (F32) {
            const float4* v = reinterpret_cast<const float4*>(static_cast<const float*>(row) + c);
            const float4 a = v[0], b = v[1];
            x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
        } else {
            const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + c);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v = 0.0f;
            if (c + i < cols) {
                if constexpr (F32) v = static_cast<const float*>(row)[c + i];
                else v = __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(row)[c + i]) << 16);
            }
            x[i] = v;
        }
    }
}

__device__ __forceinline__ uint32_t size_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// Four threads hold a block of 32; each finds the block's scale with two exchanges.
template <bool F32>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const Mx4Params p)
{
    constexpr int kUnits = 4;
    wait_for_launch_before();
    const int lane = threadIdx.x & 15;
    const int64_t padded = (p.rows + kMx4Tile - 1) / kMx4Tile * kMx4Tile;
    Units u(static_cast<int64_t>(blockIdx.x) * (kGroups * kUnits) + (threadIdx.x >> 4), p.tiles, kGroups);
    const size_t size = F32 ? 4 : 2;
    float x[kUnits][8];
    int64_t row[kUnits];
    int tile[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i, u.next()) {
        row[i] = u.row;
        tile[i] = u.tile;
        const int64_t cols = u.row < p.rows ? p.cols : 0;
        const unsigned char* src = static_cast<const unsigned char*>(p.x) + (cols ? u.row * p.stride * size : 0);
        load8<F32>(src, static_cast<int64_t>(u.tile) * kMx4Tile + lane * 8, cols, p.vectors != 0, x[i]);
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, size_bits(x[i][j]));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        const uint32_t byte = mx4_scale_byte(top);
        const float inverse = mx4_inverse(byte);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[i][j] *= inverse;
        const uint32_t codes = mx4_codes(x[i]);
        uint32_t word = byte << (8 * (lane >> 2));       // the tile's four scales in one word
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 8);
        if (row[i] < p.rows)
            *reinterpret_cast<uint32_t*>(p.codes + (row[i] * p.tiles + tile[i]) * kMx4TileBytes + lane * 4) = codes;
        if (lane == 0 && row[i] < padded) *reinterpret_cast<uint32_t*>(p.scales + scale_offset(row[i], tile[i], p.tiles)) = word;
    }
}

// Rows of the 4-bit matrix are columns of x: a block takes 64 of them and a tile of 128 rows of x.  Each warp reads 32 rows
// of x, a thread two neighbouring columns, so that blocks of 32 lie in its registers; codes and scales go out by way of
// shared memory, a row's 64 bytes together.
constexpr int kTRows = 64, kTThreads = 128;
constexpr int kTPitch = 80;                // bytes between rows of codes in shared memory: 16-byte stores of 8 rows do not collide

template <bool F32>
__global__ void __launch_bounds__(kTThreads) quantize_transposed_kernel(const Mx4Params p, unsigned row_blocks)
{
    __shared__ __align__(16) uint8_t codes[kTRows * kTPitch];
    __shared__ __align__(16) uint8_t scales[kTRows * 4];
    wait_for_launch_before();
    const int tile = static_cast<int>(blockIdx.x / row_blocks);
    const int64_t r0 = static_cast<int64_t>(blockIdx.x % row_blocks) * kTRows;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r = r0 + 2 * lane;
    const int64_t k0 = static_cast<int64_t>(tile) * kMx4Tile + warp * 32;
    const int depth = static_cast<int>(max(int64_t(0), min(int64_t(32), p.cols - k0)));
    float x[2][32];
    const bool pairs = (p.stride & 1) == 0 && r + 2 <= p.rows;
    const size_t size = F32 ? 4 : 2;
    const unsigned char* src = static_cast<const unsigned char*>(p.x) + (k0 * p.stride + r) * size;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        x[0][i] = x[1][i] = 0.0f;
        if (i < depth) {
            const unsigned char* at = src + i * p.stride * size;
            if (pairs) {
                if constexpr (F32) {
                    const float2 v = *reinterpret_cast<const float2*>(at);
                    x[0][i] = v.x, x[1][i] = v.y;
                } else {
                    const uint32_t v = *reinterpret_cast<const uint32_t*>(at);
                    x[0][i] = __uint_as_float(v << 16), x[1][i] = __uint_as_float(v & 0xFFFF0000u);
                }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (r + h < p.rows) {
                        if constexpr (F32) x[h][i] = reinterpret_cast<const float*>(at)[h];
                        else x[h][i] = __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(at)[h]) << 16);
                    }
            }
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) top = max(top, size_bits(x[h][i]));
        const uint32_t byte = mx4_scale_byte(top);
        const float inverse = mx4_inverse(byte);
        uint32_t w[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = x[h][8 * v + j] * inverse;
            w[v] = mx4_codes(y);
        }
        *reinterpret_cast<uint4*>(codes + (2 * lane + h) * kTPitch + warp * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        scales[(2 * lane + h) * 4 + warp] = static_cast<uint8_t>(byte);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTRows * 4 / kTThreads; ++i) {
        const int at = i * kTThreads + threadIdx.x, row = at >> 2, part = at & 3;
        if (r0 + row < p.rows)
            *reinterpret_cast<uint4*>(p.codes + ((r0 + row) * p.tiles + tile) * kMx4TileBytes + part * 16) =
                *reinterpret_cast<const uint4*>(codes + row * kTPitch + part * 16);
    }
    if (threadIdx.x < kTRows)
        *reinterpret_cast<uint32_t*>(p.scales + scale_offset(r0 + threadIdx.x, tile, p.tiles)) =
            *reinterpret_cast<const uint32_t*>(scales + 4 * threadIdx.x);
}

template <bool F32>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const Mx4Params p)
{
    constexpr int kUnits = 4;
    wait_for_launch_before();
    const int lane = threadIdx.x & 15;
    Units u(static_cast<int64_t>(blockIdx.x) * (kGroups * kUnits) + (threadIdx.x >> 4), p.tiles, kGroups);
    uint32_t codes[kUnits], byte[kUnits];
    int64_t row[kUnits];
    int tile[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i, u.next()) {
        row[i] = u.row;
        tile[i] = u.tile;
        codes[i] = byte[i] = 0;
        if (u.row < p.rows) {
            codes[i] = *reinterpret_cast<const uint32_t*>(p.codes + (u.row * p.tiles + u.tile) * kMx4TileBytes + lane * 4);
            byte[i] = p.scales[scale_offset(u.row, u.tile, p.tiles) + (lane >> 2)];
        }
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        if (row[i] >= p.rows) continue;
        const float scale = mx4_scale(byte[i]);
        __half2 n[4];
        mx4_numbers(codes[i], n);
        float y[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 v = __half22float2(n[j]);
            y[2 * j] = v.x * scale, y[2 * j + 1] = v.y * scale;
        }
        const int64_t c = static_cast<int64_t>(tile[i]) * kMx4Tile + lane * 8;
        const int64_t at = row[i] * p.stride + c;
        const bool whole = p.vectors && c + 8 <= p.cols;
        if constexpr (F32) {
            float* out = static_cast<float*>(p.y) + at;
            if (whole) {
                reinterpret_cast<float4*>(out)[0] = make_float4(y[0], y[1], y[2], y[3]);
                reinterpret_cast<float4*>(out)[1] = make_float4(y[4], y[5], y[6], y[7]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j < p.cols) out[j] = y[j];
            }
        } else {
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.y) + at;
            if (whole) {
                __nv_bfloat162 v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = __floats2bfloat162_rn(y[2 * j], y[2 * j + 1]);
                *reinterpret_cast<uint4*>(out) = *reinterpret_cast<uint4*>(v);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j < p.cols) out[j] = __float2bfloat16_rn(y[j]);
            }
        }
    }
}

// Blocks for so many units, or 0 if there are more than a grid holds.
unsigned blocks_for(int64_t units, int per)
{
    const int64_t n = (units + per - 1) / per;
    return n <= INT32_MAX ? static_cast<unsigned>(n) : 0;
}

}  // namespace

cudaError_t launch_mx4_quantize(const Mx4Params& p, bool transposed, cudaStream_t s)
{
    const int64_t padded = (p.rows + kMx4Tile - 1) / kMx4Tile * kMx4Tile;
    if (transposed) {
        const unsigned row_blocks = static_cast<unsigned>(padded / kTRows);
        const unsigned grid = blocks_for(static_cast<int64_t>(row_blocks) * p.tiles, 1);
        if (!grid) return cudaErrorInvalidConfiguration;
        return launch_chained(p.f32 ? quantize_transposed_kernel<true> : quantize_transposed_kernel<false>, grid, kTThreads, 0, s, p,
                              row_blocks);
    }
    const unsigned grid = blocks_for(padded * p.tiles, kGroups * 4);
    if (!grid) return cudaErrorInvalidConfiguration;
    return launch_chained(p.f32 ? quantize_rows_kernel<true> : quantize_rows_kernel<false>, grid, kThreads, 0, s, p);
}

cudaError_t launch_mx4_dequantize(const Mx4Params& p, cudaStream_t s)
{
    const unsigned grid = blocks_for(p.rows * p.tiles, kGroups * 4);
    if (!grid) return cudaErrorInvalidConfiguration;
    return launch_chained(p.f32 ? dequantize_kernel<true> : dequantize_kernel<false>, grid, kThreads, 0, s, p);
}

}  // namespace sdv2
