// Matrices to and from microscaled 4-bit numbers.
//
// Both read and write every byte once, so that memory bounds them as long as the arithmetic of a number stays below about 20
// instructions.  A block of 256 threads takes 16 rows, 16 threads a row; a thread has 8 neighbouring columns of a tile of 128 and
// two or four tiles, all of whose loads are under way together, at addresses that differ by constants.  The 16 rows are 4
// neighbours and those 32, 64 and 96 behind them, whose scales lie together (64 bytes a tile).
// Quantisation of rows lets the next launch set itself up at once, whose blocks then take the SMs that it leaves: quantisation and
// product of 512 x 1536, depth 4096, take 13.8 us without and 13.1 with that, 3 x 9216, depth 1536, 7.1 and 6.5.  (The others are
// slower with it: a transpose of 4680 x 1536 behind another one 5.1 and 6.3.)
// 4680 x 5120 takes 16.9 us from fp32 (6.4 TB/s) and 12.0 from bf16 (5.1 TB/s; 2.9 instructions a
// cycle and SM, so that both count), its values 10.7 to bf16 and 22.9 to fp32; 4680 x 1536 bf16 takes 5.0 us, its transpose 5.1.
// A row that is not whole vectors of 8 columns is read and written number by number, 16 neighbours at once, by way of shared
// memory.
#include <cuda_bf16.h>

#include <algorithm>

#include "chained.cuh"
#include "mx4.cuh"
#include "project.h"

namespace sdv2 {
namespace {

constexpr int kThreads = 256, kRows = 16;

// A thread's row and its tiles, kUnroll at most.
template <int kUnroll>
struct Place {
    int64_t row;
    int row_tile, in_tile, tile, tiles;
    __device__ __forceinline__ Place(const Mx4Params& p, unsigned row_groups)
    {
        const unsigned chunk = blockIdx.x / row_groups, group = blockIdx.x - chunk * row_groups;
        const int i = threadIdx.x >> 4;
        row_tile = static_cast<int>(group >> 3);
        in_tile = static_cast<int>(group & 7) * 4 + (i & 3) + 32 * (i >> 2);
        row = static_cast<int64_t>(row_tile) * kMx4Tile + in_tile;
        tile = static_cast<int>(chunk) * kUnroll;
        tiles = min(kUnroll, p.tiles - tile);
    }
    __device__ __forceinline__ int64_t codes(const Mx4Params& p) const { return (row * p.tiles + tile) * kMx4TileBytes; }
    __device__ __forceinline__ int64_t scales(const Mx4Params& p) const
    {
        return (static_cast<int64_t>(row_tile) * p.tiles + tile) * 512 + (in_tile & 31) * 16 + (in_tile >> 5) * 4;
    }
};

__device__ __forceinline__ float bf16_at(const void* x, int64_t i)
{
    return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(x)[i]) << 16);
}

template <bool F32, bool VECTORS, int kUnroll>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const Mx4Params p, unsigned row_groups)
{
    __shared__ __align__(16) float staged[VECTORS ? 1 : kRows * kMx4Tile];
    wait_for_launch_before();
    launch_dependents();
    const Place<kUnroll> at(p, row_groups);
    const int lane = threadIdx.x & 15;
    const bool live = at.row < p.rows;
    const int64_t c0 = static_cast<int64_t>(at.tile) * kMx4Tile;
    const int64_t first = live ? at.row * p.stride + c0 : 0;
    float x[kUnroll][8];
    if constexpr (VECTORS) {
        uint4 raw[kUnroll][F32 ? 2 : 1];
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(p.x) + first * (F32 ? 4 : 2)) + lane * (F32 ? 2 : 1);
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
#pragma unroll
            for (int h = 0; h < (F32 ? 2 : 1); ++h) {
                raw[i][h] = make_uint4(0, 0, 0, 0);
                if (live && c0 + i * kMx4Tile + lane * 8 < p.cols) raw[i][h] = src[i * (F32 ? 32 : 16) + h];
            }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const uint4 v = raw[i][0];
            if constexpr (F32) {
                const uint4 w = raw[i][1];
                const uint32_t all[8] = {v.x, v.y, v.z, v.w, w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 8; ++j) x[i][j] = __uint_as_float(all[j]);
            } else {
                const uint32_t all[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[i][2 * j] = __uint_as_float(all[j] << 16);
                    x[i][2 * j + 1] = __uint_as_float(all[j] & 0xFFFF0000u);
                }
            }
        }
    } else {
        float raw[kUnroll][8];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = i * kMx4Tile + j * 16 + lane;
                raw[i][j] = 0.0f;
                if (live && c0 + c < p.cols) raw[i][j] = F32 ? static_cast<const float*>(p.x)[first + c] : bf16_at(p.x, first + c);
            }
        float* mine = staged + (threadIdx.x >> 4) * kMx4Tile;
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) mine[j * 16 + lane] = raw[i][j];
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i][j] = mine[lane * 8 + j];
        }
    }
    uint8_t* codes = p.codes + at.codes(p) + lane * 4;
    uint8_t* scales = p.scales + at.scales(p);
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        uint32_t t;                                      // four threads hold a block of 32
        if constexpr (F32) {                             // (4680 x 5120 16.9 us; with max_size 18.1)
            t = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) t = max(t, __float_as_uint(x[i][j]) & 0x7FFFFFFFu);
        } else {
            t = __float_as_uint(max_size(max_size(x[i][0], x[i][1], x[i][2]), max_size(x[i][3], x[i][4], x[i][5]), max_size(x[i][6], x[i][7], 0.0f)));
        }
        t = max(t, __shfl_xor_sync(0xFFFFFFFFu, t, 1));
        t = max(t, __shfl_xor_sync(0xFFFFFFFFu, t, 2));
        const uint32_t byte = mx4_scale_byte(t);
        const float inverse = mx4_inverse(byte);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[i][j] *= inverse;
        const uint32_t four_bits = mx4_codes(x[i]);
        uint32_t word = byte << (8 * (lane >> 2));       // the tile's four scales in one word
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 8);
        if (i < at.tiles) {
            if (live) *reinterpret_cast<uint32_t*>(codes + i * kMx4TileBytes) = four_bits;
            if (lane == 0) *reinterpret_cast<uint32_t*>(scales + i * 512) = word;
        }
    }
}

// Rows of the 4-bit matrix are columns of x: a block takes 64 of them and a tile of 128 rows of x.  Each warp reads 32 rows
// of x, a thread two neighbouring columns, so that blocks of 32 lie in its registers; codes and scales go out by way of
// shared memory, a row's 64 bytes together.
constexpr int kTRows = 64, kTThreads = 128;
constexpr int kTPitch = 80;                // bytes between rows of codes in shared memory: 16-byte stores of 8 rows do not collide

template <bool F32, bool PAIRS>
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
    // bf16: both columns of a thread in a register.  Rows of x behind its last are read as that one and then count as 0, so that
    // all loads are under way together.  (One way through this for every block: a second one costs its instructions' first fetch.)
    uint32_t x[F32 ? 2 : 1][32] = {};
    const unsigned char* src = static_cast<const unsigned char*>(p.x) + (k0 * p.stride + r) * (F32 ? 4 : 2);
    const int64_t step = p.stride * (F32 ? 4 : 2);
    const bool one = depth > 0 && r < p.rows, two = depth > 0 && r + 1 < p.rows;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const unsigned char* from = src + min(i, depth - 1) * step;
        if (PAIRS && two) {
            if constexpr (F32) {
                const uint2 v = *reinterpret_cast<const uint2*>(from);
                x[0][i] = v.x, x[1][i] = v.y;
            } else {
                x[0][i] = *reinterpret_cast<const uint32_t*>(from);
            }
        } else if constexpr (F32) {
            if (one) x[0][i] = reinterpret_cast<const uint32_t*>(from)[0];
            if (two) x[1][i] = reinterpret_cast<const uint32_t*>(from)[1];
        } else {
            if (one) x[0][i] = reinterpret_cast<const uint16_t*>(from)[0];
            if (two) x[0][i] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(from)[1]) << 16;
        }
    }
    if (depth < 32) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i >= depth) {
                x[0][i] = 0;
                if constexpr (F32) x[1][i] = 0;
            }
    }
    uint32_t top[2] = {};
    if constexpr (F32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float t = 0.0f;
#pragma unroll
            for (int i = 0; i < 32; i += 2) t = max_size(t, __uint_as_float(x[F32 ? h : 0][i]), __uint_as_float(x[F32 ? h : 0][i + 1]));
            top[h] = __float_as_uint(t);
        }
    } else {
        uint32_t two = 0;
#pragma unroll
        for (int i = 0; i < 32; i += 2) two = __vimax3_u16x2(two, x[0][i] & 0x7FFF7FFFu, x[0][i + 1] & 0x7FFF7FFFu);
        top[0] = two << 16, top[1] = two & 0xFFFF0000u;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t byte = mx4_scale_byte(top[h]);
        const float inverse = mx4_inverse(byte);
        uint32_t w[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t bits = F32 ? x[F32 ? h : 0][8 * v + j] : h ? x[0][8 * v + j] & 0xFFFF0000u : x[0][8 * v + j] << 16;
                y[j] = __uint_as_float(bits) * inverse;
            }
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
    if (threadIdx.x < kTRows) {
        const int64_t row = r0 + threadIdx.x;
        *reinterpret_cast<uint32_t*>(p.scales + ((row >> 7) * p.tiles + tile) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4) =
            *reinterpret_cast<const uint32_t*>(scales + 4 * threadIdx.x);
    }
}

template <bool F32, bool VECTORS, int kUnroll>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const Mx4Params p, unsigned row_groups)
{
    __shared__ __align__(16) float staged[VECTORS ? 1 : kRows * kMx4Tile];
    wait_for_launch_before();
    const Place<kUnroll> at(p, row_groups);
    const int lane = threadIdx.x & 15;
    const bool live = at.row < p.rows;
    const uint8_t* codes = p.codes + at.codes(p) + lane * 4;
    const uint8_t* scales = p.scales + at.scales(p);
    uint32_t four_bits[kUnroll] = {}, word[kUnroll] = {};
#pragma unroll
    for (int i = 0; i < kUnroll; ++i)
        if (live && i < at.tiles) {
            four_bits[i] = *reinterpret_cast<const uint32_t*>(codes + i * kMx4TileBytes);
            word[i] = *reinterpret_cast<const uint32_t*>(scales + i * 512);
        }
    const int64_t c0 = static_cast<int64_t>(at.tile) * kMx4Tile;
    const int64_t first = at.row * p.stride + c0;
    float* mine = VECTORS ? staged : staged + (threadIdx.x >> 4) * kMx4Tile;
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        const float scale = mx4_scale((word[i] >> (8 * (lane >> 2))) & 255u);
        __half2 n[4];
        mx4_numbers(four_bits[i], n);
        float y[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 v = __half22float2(n[j]);
            y[2 * j] = v.x * scale, y[2 * j + 1] = v.y * scale;
        }
        if constexpr (VECTORS) {
            if (!live || c0 + i * kMx4Tile + lane * 8 >= p.cols) continue;
            const int64_t o = first + i * kMx4Tile + lane * 8;
            if constexpr (F32) {
                float4* out = reinterpret_cast<float4*>(static_cast<float*>(p.y) + o);
                out[0] = make_float4(y[0], y[1], y[2], y[3]);
                out[1] = make_float4(y[4], y[5], y[6], y[7]);
            } else {
                __nv_bfloat162 v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = __floats2bfloat162_rn(y[2 * j], y[2 * j + 1]);
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.y) + o) = *reinterpret_cast<uint4*>(v);
            }
        } else {
            __syncwarp();
            *reinterpret_cast<float4*>(mine + lane * 8) = make_float4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<float4*>(mine + lane * 8 + 4) = make_float4(y[4], y[5], y[6], y[7]);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = i * kMx4Tile + j * 16 + lane;
                if (!live || c0 + c >= p.cols) continue;
                if constexpr (F32) static_cast<float*>(p.y)[first + c] = mine[j * 16 + lane];
                else static_cast<__nv_bfloat16*>(p.y)[first + c] = __float2bfloat16_rn(mine[j * 16 + lane]);
            }
        }
    }
}

// Blocks of 16 rows and `unroll` tiles; false if there are more than a grid holds.
bool blocks_of(const Mx4Params& p, int unroll, unsigned* grid, unsigned* row_groups)
{
    const int64_t groups = (p.rows + kMx4Tile - 1) / kMx4Tile * (kMx4Tile / kRows);
    const int64_t n = groups * ((p.tiles + unroll - 1) / unroll);
    *grid = static_cast<unsigned>(n);
    *row_groups = static_cast<unsigned>(groups);
    return n <= INT32_MAX;
}

}  // namespace

cudaError_t launch_mx4_quantize(const Mx4Params& p, bool transposed, cudaStream_t s)
{
    unsigned grid, row_groups;
    if (transposed) {
        const int64_t row_blocks = (p.rows + kMx4Tile - 1) / kMx4Tile * (kMx4Tile / kTRows);
        if (row_blocks * p.tiles > INT32_MAX) return cudaErrorInvalidConfiguration;
        auto kernel = p.stride & 1 ? (p.f32 ? quantize_transposed_kernel<true, false> : quantize_transposed_kernel<false, false>)
                                   : (p.f32 ? quantize_transposed_kernel<true, true> : quantize_transposed_kernel<false, true>);
        return launch_chained(kernel, static_cast<unsigned>(row_blocks * p.tiles), kTThreads, 0, s, p, static_cast<unsigned>(row_blocks));
    }
    // two tiles of a thread: 4680 x 5120 fp32 16.8 us (one: 19.1, four: 18.1), 512 x 4096 bf16 2.6 us (2.5 and 3.0)
    if (!blocks_of(p, 2, &grid, &row_groups)) return cudaErrorInvalidConfiguration;
    auto kernel = p.vectors ? (p.f32 ? quantize_rows_kernel<true, true, 2> : quantize_rows_kernel<false, true, 2>)
                            : (p.f32 ? quantize_rows_kernel<true, false, 2> : quantize_rows_kernel<false, false, 2>);
    return launch_chained(kernel, grid, kThreads, 0, s, p, row_groups);
}

cudaError_t launch_mx4_dequantize(const Mx4Params& p, cudaStream_t s)
{
    unsigned grid, row_groups;
    // 4680 x 5120: bf16 10.7 us with four tiles of a thread and 11.7 with two, fp32 25.6 and 22.9
    if (!blocks_of(p, p.f32 ? 2 : 4, &grid, &row_groups)) return cudaErrorInvalidConfiguration;
    auto kernel = p.vectors ? (p.f32 ? dequantize_kernel<true, true, 2> : dequantize_kernel<false, true, 4>)
                            : (p.f32 ? dequantize_kernel<true, false, 2> : dequantize_kernel<false, false, 4>);
    return launch_chained(kernel, grid, kThreads, 0, s, p, row_groups);
}

}  // namespace sdv2
