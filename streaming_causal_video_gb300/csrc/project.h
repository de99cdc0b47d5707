// Launch parameters and launchers of the operators in sdv2_project.h (not installed).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "../../include/sdv2_project.h"

namespace sdv2 {

// ---- microscaled 4-bit matrices -----------------------------------------------------------------

constexpr int kMx4Block = 32;              // numbers that share a scale
constexpr int kMx4Tile = 128;              // rows and columns of a scale tile: 512 bytes [row % 32][row / 32][block]
constexpr int kMx4TileBytes = 64;          // bytes of a row's codes in a tile

struct Mx4Params {
    const void* x;                         // quantize: read; null otherwise
    void* y;                               // dequantize: written
    uint8_t* codes;                        // [rows][64 * tiles]
    uint8_t* scales;                       // [row tiles][tiles][32][4][4]
    int64_t rows, cols, stride;            // of the 4-bit matrix; elements between rows of x or y
    int32_t tiles;                         // ceil(cols / 128)
    int32_t f32;                           // x or y is fp32, else bf16
    int32_t vectors;                       // rows of x or y begin on 16 bytes and are whole groups of 8 columns
};

cudaError_t launch_mx4_quantize(const Mx4Params& p, bool transposed, cudaStream_t s);
cudaError_t launch_mx4_dequantize(const Mx4Params& p, cudaStream_t s);

struct Mx4Product {
    const uint8_t* a;                      // codes and scales of a: M rows, tiles * 128 columns
    const uint8_t* as;
    const uint8_t* b;                      // of b: N rows
    const uint8_t* bs;
    const float* bias;                     // [N] or null
    void* out;
    int64_t M, N, out_stride;
    int32_t tiles;                         // ceil(K / 128)
    int32_t out_f32, gelu;
    uint32_t* err;                         // device error word
    uint64_t timeout_ns;
    int64_t drop;                          // fault injection: 256-column step whose copies are left out, or -1
};

// Rows of a that go to launch_mx4_rows, us there and in tiles: 64 rows at 1536 x 8960 6.9 and 9.6, at 5120 x 20480 15.1 and 21.7, at
// 5120 x 5120 8.6 and 8.7, at 9216 x 1536 5.9 and 6.7, at 1536 x 1536 4.3 and 4.6; fewer rows are further apart.
constexpr int kMx4FewRows = 64;

// How a product runs: rows of b in a tile (of few rows: columns of an MMA, as many rows of a at most), parts of the depth, and the
// most tiles of a pair of SMs.
struct Mx4Plan {
    int width, parts, rounds;
};

Mx4Plan mx4_rows_plan(int64_t M, int64_t N, int tiles);
Mx4Plan mx4_product_plan(int64_t M, int64_t N, int tiles);

// Few rows of a.
cudaError_t launch_mx4_rows(const Mx4Product& p, cudaStream_t s);

cudaError_t launch_mx4_product(const Mx4Product& p, cudaStream_t s);

// ---- rotary positions -----------------------------------------------------------------------------

constexpr int kRopePairs = 128;            // head_dim 256

struct RopePair {
    uint64_t turn;                         // turns for a step of the position, as a 64-bit fraction of one
    int16_t u, v;                          // dims of the pair
    int16_t axis;                          // or -1: stays as it is (its turn is 0)
    int16_t pad;
};

struct RopeTensor {
    const void* in;
    void* out;
    sdv2_rope_strides is, os;
};

struct AxesRopeParams {
    RopeTensor t[2];                       // q and k
    const int32_t* positions;
    int64_t tokens;
    int32_t batch, heads, kv_heads, axes;
    int32_t shared;                        // one row of positions for all of the batch
    int32_t items;                         // threads for one row of heads
    int32_t per;                           // heads that a thread turns
    int32_t q_parts;                       // blocks in y for the heads of q; those of k follow
    RopePair pair[kRopePairs];
};

// adjacent: pairs of neighbours; else of two half segments, all of which are whole vectors of `width` elements (16 bytes, 2 or 1);
// all: every dim turns.
cudaError_t launch_axes_rope(AxesRopeParams& p, bool adjacent, int width, bool all, bool f32, int head_dim, cudaStream_t s);

}  // namespace sdv2
