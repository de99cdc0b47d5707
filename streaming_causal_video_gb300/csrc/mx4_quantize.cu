// Matrices to and from microscaled 4-bit numbers.
//
// Both read and write every byte once, so that memory bounds them as long as the arithmetic of a number stays below about 20
// instructions.  A block of 256 threads takes 16 rows, 16 threads a row; a thread has 8 neighbouring columns of a tile of 128 and
// one, two or four tiles, all of whose loads are under way together, at addresses that differ by constants.  The 16 rows are 4
// neighbours and those 32, 64 and 96 behind them, whose scales lie together (64 bytes a tile).
// Quantisation of rows lets the next launch set itself up at once, whose blocks then take the SMs that it leaves: quantisation and
// product of 512 x 1536, depth 4096, take 13.8 us without and 13.1 with that, 3 x 9216, depth 1536, 7.1 and 6.5.  (The others are
// slower with it: a transpose of 4680 x 1536 behind another one 5.1 and 6.3.)
// 4680 x 5120 takes 16.9 us from fp32 (6.4 TB/s) and 11.5 from bf16 (5.3 TB/s; 2.9 instructions a
// cycle and SM, so that both count), its values 10.7 to bf16 and 21.7 to fp32; 4680 x 1536 bf16 takes 4.6 us, its transpose 5.1.
// Transposes to 20480 x 4680 take 41.4 us from bf16 (5.9 TB/s) and 63.7 from fp32 (6.8).
// A row that is not whole vectors of 8 columns goes by way of shared memory, 16 neighbouring words of 4 bytes at once, from which
// bf16 rows that begin on odd places are shifted (4680 x 5111 14.4 us, its values 13.2; number by number 22.5 and 19.5).
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

// Words of shared memory for a row's tiles that are not read or written in vectors; 16 threads and 16 others do not collide.
template <bool F32, int kUnroll>
constexpr int kPitch = F32 ? kMx4Tile : kUnroll * (kMx4Tile / 2) + 16;

template <bool F32, bool VECTORS, int kUnroll>
__global__ void __launch_bounds__(kThreads, F32 ? 0 : 8) quantize_rows_kernel(const Mx4Params p, unsigned row_groups)
{
    constexpr int PITCH = kPitch<F32, kUnroll>;
    __shared__ __align__(16) uint32_t staged[VECTORS ? 1 : kRows * PITCH];
    wait_for_launch_before();
    launch_dependents();
    const Place<kUnroll> at(p, row_groups);
    const int lane = threadIdx.x & 15;
    const bool live = at.row < p.rows;
    const int64_t c0 = static_cast<int64_t>(at.tile) * kMx4Tile;
    const int64_t first = live ? at.row * p.stride + c0 : 0;
    const int room = live ? static_cast<int>(min(p.cols - c0, int64_t(kUnroll * kMx4Tile))) : 0;
    float x[kUnroll][8];
    if constexpr (VECTORS || !F32) {
        uint4 raw[kUnroll][F32 ? 2 : 1];
        if constexpr (VECTORS) {
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(p.x) + first * (F32 ? 4 : 2)) + lane * (F32 ? 2 : 1);
#pragma unroll
            for (int i = 0; i < kUnroll; ++i)
#pragma unroll
                for (int h = 0; h < (F32 ? 2 : 1); ++h) {
                    raw[i][h] = make_uint4(0, 0, 0, 0);
                    if (i * kMx4Tile + lane * 8 < room) raw[i][h] = src[i * (F32 ? 32 : 16) + h];
                }
        } else {
            // Words of two numbers from the even place at or before the first on; a last number that is alone in its word comes alone.
            constexpr int WORDS = kUnroll * (kMx4Tile / 2);
            const int odd = static_cast<int>(first & 1);
            const uint16_t* const row = static_cast<const uint16_t*>(p.x) + first;
            const uint32_t* const src = reinterpret_cast<const uint32_t*>(row - odd) + lane;
            uint32_t* const mine = staged + (threadIdx.x >> 4) * PITCH;
            uint32_t word[WORDS / 16], last = 0;
#pragma unroll
            for (int j = 0; j < WORDS / 16; ++j) {
                word[j] = 0;
                if (2 * (j * 16 + lane) - odd + 1 < room) word[j] = src[j * 16];
            }
            const bool alone = lane == 0 && ((room + odd) & 1);
            if (alone && room > 0) last = row[room - 1];
#pragma unroll
            for (int j = 0; j < WORDS / 16; ++j) mine[j * 16 + lane] = word[j];
            if (lane == 0) mine[WORDS] = 0;
            __syncwarp();
            if (alone) mine[(room - 1 + odd) >> 1] = last;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const uint32_t* const from = mine + i * (kMx4Tile / 2) + lane * 4;
                const uint4 v = *reinterpret_cast<const uint4*>(from);
                raw[i][0] = make_uint4(__funnelshift_r(v.x, v.y, 16 * odd), __funnelshift_r(v.y, v.z, 16 * odd), __funnelshift_r(v.z, v.w, 16 * odd),
                                       __funnelshift_r(v.w, from[4], 16 * odd));
            }
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
        const float* const src = static_cast<const float*>(p.x) + first + lane;
        float raw[kUnroll][8];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = i * kMx4Tile + j * 16;
                raw[i][j] = 0.0f;
                if (c + lane < room) raw[i][j] = src[c];
            }
        float* const mine = reinterpret_cast<float*>(staged) + (threadIdx.x >> 4) * PITCH;
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

__device__ __forceinline__ uint4 bf16_words(const float (&y)[8])
{
    __nv_bfloat162 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __floats2bfloat162_rn(y[2 * j], y[2 * j + 1]);
    return *reinterpret_cast<const uint4*>(v);
}

template <bool F32, bool VECTORS, int kUnroll>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const Mx4Params p, unsigned row_groups)
{
    constexpr int PITCH = kPitch<F32, kUnroll>;
    __shared__ __align__(16) uint32_t staged[VECTORS ? 1 : kRows * PITCH];
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
    const int room = live ? static_cast<int>(min(p.cols - c0, int64_t(kUnroll * kMx4Tile))) : 0;
    uint32_t* const mine = VECTORS ? staged : staged + (threadIdx.x >> 4) * PITCH;
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
            if (i * kMx4Tile + lane * 8 >= room) continue;
            const int64_t o = first + i * kMx4Tile + lane * 8;
            if constexpr (F32) {
                float4* out = reinterpret_cast<float4*>(static_cast<float*>(p.y) + o);
                out[0] = make_float4(y[0], y[1], y[2], y[3]);
                out[1] = make_float4(y[4], y[5], y[6], y[7]);
            } else {
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.y) + o) = bf16_words(y);
            }
        } else if constexpr (F32) {
            __syncwarp();
            *reinterpret_cast<float4*>(mine + lane * 8) = make_float4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<float4*>(mine + lane * 8 + 4) = make_float4(y[4], y[5], y[6], y[7]);
            __syncwarp();
            float* const out = static_cast<float*>(p.y) + first + lane;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = i * kMx4Tile + j * 16;
                if (c + lane < room) out[c] = __uint_as_float(mine[j * 16 + lane]);
            }
        } else {
            *reinterpret_cast<uint4*>(mine + i * (kMx4Tile / 2) + lane * 4) = bf16_words(y);
        }
    }
    if constexpr (!VECTORS && !F32) {
        // words of two numbers from an even place on, and by themselves a first and a last one that have none beside them
        __syncwarp();
        const int odd = static_cast<int>(first & 1);
        uint16_t* const row = static_cast<uint16_t*>(p.y) + first;
        uint32_t* const out = reinterpret_cast<uint32_t*>(row + odd) + lane;
#pragma unroll
        for (int j = 0; j < kUnroll * 4; ++j) {
            const int w = j * 16 + lane;
            if (2 * w + odd + 1 < room) out[j * 16] = __funnelshift_r(mine[w], mine[w + odd], 16 * odd);
        }
        if (lane == 0 && odd && room > 0) row[0] = static_cast<uint16_t>(mine[0]);
        if (lane == 1 && room > odd && ((room - odd) & 1)) row[room - 1] = static_cast<uint16_t>(mine[(room - 1) >> 1] >> (16 * ((room - 1) & 1)));
    }
}

// Blocks of 16 rows and `unroll` tiles.
int64_t row_groups_of(const Mx4Params& p) { return (p.rows + kMx4Tile - 1) / kMx4Tile * (kMx4Tile / kRows); }
int64_t blocks_of(const Mx4Params& p, int unroll) { return row_groups_of(p) * ((p.tiles + unroll - 1) / unroll); }

// Whether a thread's four tiles are all but an eighth of them there.
bool fills_four(const Mx4Params& p) { return (p.tiles + 3) / 4 * 4 * 7 <= p.tiles * 8; }

constexpr int64_t kWave = 152 * 8;         // blocks that the GPU holds at once

using RowsKernel = void (*)(const Mx4Params, unsigned);

cudaError_t launch_rows(RowsKernel kernel, const Mx4Params& p, int unroll, cudaStream_t s)
{
    const int64_t blocks = blocks_of(p, unroll);
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_chained(kernel, static_cast<unsigned>(blocks), kThreads, 0, s, p, static_cast<unsigned>(row_groups_of(p)));
}

}  // namespace

cudaError_t launch_mx4_quantize(const Mx4Params& p, bool transposed, cudaStream_t s)
{
    if (transposed) {
        const int64_t row_blocks = (p.rows + kMx4Tile - 1) / kMx4Tile * (kMx4Tile / kTRows);
        if (row_blocks * p.tiles > INT32_MAX) return cudaErrorInvalidConfiguration;
        auto kernel = p.stride & 1 ? (p.f32 ? quantize_transposed_kernel<true, false> : quantize_transposed_kernel<false, false>)
                                   : (p.f32 ? quantize_transposed_kernel<true, true> : quantize_transposed_kernel<false, true>);
        return launch_chained(kernel, static_cast<unsigned>(row_blocks * p.tiles), kTThreads, 0, s, p, static_cast<unsigned>(row_blocks));
    }
    // Tiles of a thread, us with one, two and four: as many as keep loads under way, but no more than leave work for every SM.
    //   fp32: 4680 x 5120 18.9, 16.8 and 17.7, 512 x 4096 3.2, 3.3 and 3.6; rows without vectors 3001 x 1001 5.0, 6.2 and 6.7
    //   bf16: 4680 x 20480 58.0, 42.0 and 37.6, 4680 x 1536 5.9, 5.0 and 4.6, 1024 x 4096 4.1, 3.4 and 3.5, 3 x 1536 1.2, 1.3 and 1.5;
    //   rows without vectors 4680 x 5111 19.1, 14.8 and 14.4, 4680 x 1050 (nine tiles) 5.3, 4.9 and 6.3
    const int unroll = blocks_of(p, 1) <= kWave || (p.f32 && !p.vectors) ? 1 : !p.f32 && blocks_of(p, 2) > kWave && fills_four(p) ? 4 : 2;
    RowsKernel kernel;
    if (p.f32) kernel = !p.vectors ? quantize_rows_kernel<true, false, 1> : unroll == 1 ? quantize_rows_kernel<true, true, 1> : quantize_rows_kernel<true, true, 2>;
    else if (p.vectors)
        kernel = unroll == 1 ? quantize_rows_kernel<false, true, 1> : unroll == 2 ? quantize_rows_kernel<false, true, 2> : quantize_rows_kernel<false, true, 4>;
    else
        kernel = unroll == 1 ? quantize_rows_kernel<false, false, 1> : unroll == 2 ? quantize_rows_kernel<false, false, 2> : quantize_rows_kernel<false, false, 4>;
    return launch_rows(kernel, p, unroll, s);
}

cudaError_t launch_mx4_dequantize(const Mx4Params& p, cudaStream_t s)
{
    // The same, us with one, two and four: 4680 x 5120 to fp32 21.7, 22.8 and 23.2, to bf16 15.1, 11.7 and 10.7; rows without vectors
    // 4680 x 5111 24.4, 23.2 and 22.4, and 18.7, 15.0 and 13.2; 1001 x 1050 (nine tiles) 2.3, 2.5 and 2.8, and 1.8, 1.7 and 1.9
    // (fp32 without vectors: two for all sizes, within 4 and 9 % of the best of these)
    const int unroll = p.f32 ? (p.vectors ? 1 : 2) : fills_four(p) && blocks_of(p, 4) >= 152 ? 4 : 2;
    RowsKernel kernel;
    if (p.f32) kernel = p.vectors ? dequantize_kernel<true, true, 1> : dequantize_kernel<true, false, 2>;
    else if (p.vectors) kernel = unroll == 2 ? dequantize_kernel<false, true, 2> : dequantize_kernel<false, true, 4>;
    else kernel = unroll == 2 ? dequantize_kernel<false, false, 2> : dequantize_kernel<false, false, 4>;
    return launch_rows(kernel, p, unroll, s);
}

}  // namespace sdv2
