// Launch parameters and launchers of the operators in sdv2_block.h (not installed).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "../../include/sdv2_block.h"

namespace sdv2 {

// Streams per launch: their lengths and tensor maps travel in the launch parameters.  A call with
// more streams is several launches over slices of the batch.
constexpr int kCrossStreams = 32;

// One operand of cross attention: element (b, token, head, d) at b*batch + token*tok + h*hd + d.
struct CrossStrides {
    int64_t tok, hd, batch;
};

struct CrossProblem {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    CrossStrides qs, kvs;
    int32_t B, H, Hk;          // streams, query heads, key heads
    int32_t Nq, Nk;
    float scale;
    uint32_t* err;             // device error word
    uint64_t timeout_ns;
    int32_t n[kCrossStreams];  // valid rows of k and v per stream (of this launch's slice)
};

struct CrossForward {
    CrossProblem c;
    uint16_t* out;             // [B][Nq][H][D]
    float* lse;                // [B][H][Nq] or null
};

struct CrossBackward {
    CrossProblem c;
    const uint16_t* out;
    const float* lse;
    const uint16_t* dout;
    uint16_t* dq;
    uint16_t* dk;              // [B][Nk][Hk][D]
    uint16_t* dv;
    float* stats;              // scratch: cross_backward_stats_bytes
    float* part;               // scratch: cross_backward_part_bytes
};

// Heads that share a key head and a 128-row query tile: the largest divisor of `group` up to 128.
int cross_pack(int group);

// Query tiles of 128 rows on the tensor cores.
cudaError_t launch_cross_attention(const CrossForward& p, cudaStream_t s);

// Gradients on the tensor cores, and the bytes of scratch for a batch of B streams: lse and delta by query
// tile, and the key tiles' partial sums.
cudaError_t launch_cross_backward(const CrossBackward& p, cudaStream_t s);
size_t cross_backward_stats_bytes(int B, int H, int Hk, int64_t Nq);
size_t cross_backward_part_bytes(int B, int H, int Hk, int64_t Nq, int64_t Nk);

// One or two rows per key head on the CUDA cores.
constexpr int kFewRows = 2, kFewKeys = 1024;       // where it is the faster of the two
cudaError_t launch_cross_rows(const CrossForward& p, cudaStream_t s);

struct NormParams {
    const void* x;
    const void* dy;            // backward only
    void* y;                   // forward: y; backward: dx
    const float* weight;       // or null
    const float* bias;         // or null; forward only
    float* mean;               // forward: written if not null; backward: read
    float* rstd;
    float* dweight;            // [groups][cols] or null
    float* dbias;
    float* partial;            // [groups][slices][2][cols]
    int64_t rows, xs, ys, gs;  // row strides of x/dx and y/dy, stride of weight groups
    int64_t rows_per_group;
    int32_t cols, slices;
    int32_t x_f32, y_f32, plus_one;
    int32_t aligned;           // 16-byte vectors of 8 columns can be used
    float eps;
};

// Blocks that share the rows of one group in the backward pass; the workspace holds one row of
// partial sums of dweight and dbias for each.
int norm_backward_slices(int64_t rows, int64_t rows_per_group, int cols, bool aligned);

cudaError_t launch_layer_norm(const NormParams& p, cudaStream_t s);
cudaError_t launch_layer_norm_backward(const NormParams& p, cudaStream_t s);

}  // namespace sdv2
