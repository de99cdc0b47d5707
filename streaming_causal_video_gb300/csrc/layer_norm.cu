// Layer norm, forward and backward, with a weight and bias for each group of rows.
//
// A DiT layer normalises its tokens twice: before the self-attention with a scale and shift of
// each latent frame (weight_plus_one, one group per frame), before the cross attention with a
// learned weight and bias (one group).
//   forward : mean and the mean square of the centred row, from registers in two passes (a
//             single pass over x and x^2 loses the variance of a row whose mean is large);
//             y = (x - mean) * rstd * gain + bias.
//   backward: xhat = (x - mean) * rstd, g = dy * gain,
//             dx = rstd * (g - mean(g) - xhat * mean(g * xhat));
//             dgain = sum over rows of dy * xhat, dbias = sum of dy.
// Both are bound by memory: each row is read once and written once and stays in registers in
// between.  The parameter sums of a group are split over `slices` blocks, each of which keeps its
// columns' sums in registers over all of its rows and writes them once; a second kernel adds the
// slices in index order, so the result does not depend on the order in which blocks run.
#include <cuda_bf16.h>

#include <algorithm>

#include "block.h"

namespace sdv2 {
namespace {

constexpr int kMaxThreads = 512;

template <bool F32>
__device__ __forceinline__ float load1(const void* base, int64_t i)
{
    if constexpr (F32) return static_cast<const float*>(base)[i];
    else return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(base)[i]) << 16);
}

// Eight consecutive columns from element offset `i` (a multiple of 8, 16-byte aligned rows).
template <bool F32>
__device__ __forceinline__ void load8(const void* base, int64_t i, float* v)
{
    if constexpr (F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
        const float4 a = p[0], b = p[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[2 * k] = __uint_as_float(u[k] << 16);
            v[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
        }
    }
}

template <bool F32>
__device__ __forceinline__ void store1(void* base, int64_t i, float v)
{
    if constexpr (F32) static_cast<float*>(base)[i] = v;
    else static_cast<__nv_bfloat16*>(base)[i] = __float2bfloat16_rn(v);
}

template <bool F32>
__device__ __forceinline__ void store8(void* base, int64_t i, const float* v)
{
    if constexpr (F32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
        p[0] = make_float4(v[0], v[1], v[2], v[3]);
        p[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint32_t u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
            u[k] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + i) = make_uint4(u[0], u[1], u[2], u[3]);
    }
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ void team_barrier(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Sum over the `warps` warps of one row's team; every thread gets the same value (the partial sums
// are added in warp order).  `scratch` holds one float per warp; `id` is the team's barrier.
__device__ __forceinline__ float team_sum(float v, int warps, int warp, float* scratch, int id)
{
    v = warp_sum(v);
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) scratch[warp] = v;
    team_barrier(id, warps * 32);
    float s = 0.f;
    for (int w = 0; w < warps; ++w) s += scratch[w];
    return s;
}

// A thread's columns: NV vectors of 8, vector i starting at column 8*(i*team + t) where the row can
// be read in 16-byte vectors, else 8*NV single columns i*team + t (still coalesced).
template <int NV, bool ALIGNED, typename F>
__device__ __forceinline__ void for_columns(int team, int t, int cols, F&& f)
{
    if constexpr (ALIGNED) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = 8 * (i * team + t);
            if (c < cols) f(i * 8, c);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV * 8; ++i) {
            const int c = i * team + t;
            if (c < cols) f(i, c);
        }
    }
}

// blockDim = (team, rows per block): one row per team of `team` threads (a multiple of 32).
template <int NV, bool ALIGNED, bool XF32, bool YF32>
__global__ void __launch_bounds__(kMaxThreads) norm_forward_kernel(const NormParams p)
{
    constexpr int W = ALIGNED ? 8 : 1;
    __shared__ float scratch[2][kMaxThreads / 32];
    const int team = blockDim.x, t = threadIdx.x;
    const int warps = team >> 5, warp = t >> 5;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (row >= p.rows) return;                         // whole team: its barrier is its own
    float* s0 = scratch[0] + threadIdx.y * warps;
    float* s1 = scratch[1] + threadIdx.y * warps;
    const int id = 1 + threadIdx.y;

    float v[NV * 8];
#pragma unroll
    for (int i = 0; i < NV * 8; ++i) v[i] = 0.f;
    for_columns<NV, ALIGNED>(team, t, p.cols, [&](int i, int c) {
        if constexpr (ALIGNED) load8<XF32>(p.x, row * p.xs + c, v + i);
        else v[i] = load1<XF32>(p.x, row * p.xs + c);
    });
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV * 8; ++i) sum += v[i];
    const float mean = team_sum(sum, warps, warp, s0, id) / static_cast<float>(p.cols);
    float sq = 0.f;
    for_columns<NV, ALIGNED>(team, t, p.cols, [&](int i, int) {
#pragma unroll
        for (int k = 0; k < W; ++k) {
            v[i + k] -= mean;
            sq = fmaf(v[i + k], v[i + k], sq);
        }
    });
    const float var = team_sum(sq, warps, warp, s1, id) / static_cast<float>(p.cols);
    const float rstd = 1.0f / sqrtf(var + p.eps);
    if (t == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    const int64_t g = (row / p.rows_per_group) * p.gs;
    const float base = p.plus_one ? 1.0f : 0.0f;
    for_columns<NV, ALIGNED>(team, t, p.cols, [&](int i, int c) {
        float w[W], b[W];
        if constexpr (ALIGNED) {
            if (p.weight) load8<true>(p.weight, g + c, w);
            if (p.bias) load8<true>(p.bias, g + c, b);
        } else {
            if (p.weight) w[0] = p.weight[g + c];
            if (p.bias) b[0] = p.bias[g + c];
        }
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const float gain = p.weight ? base + w[k] : 1.0f;
            v[i + k] = fmaf(v[i + k] * rstd, gain, p.bias ? b[k] : 0.f);
        }
        if constexpr (ALIGNED) store8<YF32>(p.y, row * p.ys + c, v + i);
        else store1<YF32>(p.y, row * p.ys + c, v[i]);
    });
}

// blockDim = (team, teams); block (group, slice) walks the group's rows slice*teams + team index,
// then every slices*teams further.  Each thread keeps dgain and dbias of its columns.
template <int NV, bool ALIGNED, bool XF32, bool YF32>
__global__ void __launch_bounds__(kMaxThreads) norm_backward_kernel(const NormParams p)
{
    constexpr int W = ALIGNED ? 8 : 1;
    extern __shared__ float dyn[];                     // [teams][2][cols] for the teams' sums
    __shared__ float scratch[4][kMaxThreads / 32];
    const int team = blockDim.x, t = threadIdx.x, teams = blockDim.y, slot = threadIdx.y;
    const int warps = team >> 5, warp = t >> 5;
    const int id = 1 + slot;
    const int64_t group = blockIdx.x / p.slices;
    const int slice = static_cast<int>(blockIdx.x - group * p.slices);
    const int64_t row_end = min(p.rows, (group + 1) * p.rows_per_group);
    const int64_t g = group * p.gs;
    const float base = p.plus_one ? 1.0f : 0.0f;
    const float inv_cols = 1.0f / static_cast<float>(p.cols);

    float dw[NV * 8], db[NV * 8], gain[NV * 8];
#pragma unroll
    for (int i = 0; i < NV * 8; ++i) {
        dw[i] = 0.f;
        db[i] = 0.f;
        gain[i] = 1.f;
    }
    if (p.weight)
        for_columns<NV, ALIGNED>(team, t, p.cols, [&](int i, int c) {
            if constexpr (ALIGNED) load8<true>(p.weight, g + c, gain + i);
            else gain[i] = p.weight[g + c];
#pragma unroll
            for (int k = 0; k < W; ++k) gain[i + k] += base;
        });
    int phase = 0;
    for (int64_t row = group * p.rows_per_group + static_cast<int64_t>(slice) * teams + slot; row < row_end;
         row += static_cast<int64_t>(p.slices) * teams) {
        float xh[NV * 8], gy[NV * 8];
#pragma unroll
        for (int i = 0; i < NV * 8; ++i) {
            xh[i] = 0.f;
            gy[i] = 0.f;
        }
        const float mean = p.mean[row], rstd = p.rstd[row];
        for_columns<NV, ALIGNED>(team, t, p.cols, [&](int i, int c) {
            if constexpr (ALIGNED) {
                load8<XF32>(p.x, row * p.xs + c, xh + i);
                load8<YF32>(p.dy, row * p.ys + c, gy + i);
            } else {
                xh[i] = load1<XF32>(p.x, row * p.xs + c);
                gy[i] = load1<YF32>(p.dy, row * p.ys + c);
            }
        });
        float s1 = 0.f, s2 = 0.f;
        for_columns<NV, ALIGNED>(team, t, p.cols, [&](int i, int) {
#pragma unroll
            for (int k = i; k < i + W; ++k) {
                xh[k] = (xh[k] - mean) * rstd;
                dw[k] = fmaf(gy[k], xh[k], dw[k]);
                db[k] += gy[k];
                gy[k] *= gain[k];
                s1 += gy[k];
                s2 = fmaf(gy[k], xh[k], s2);
            }
        });
        // two scratch rows in turn: a warp that is a row ahead does not touch what others still read
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        if (warps > 1) {
            float* a = scratch[2 * phase] + slot * warps;
            float* b = scratch[2 * phase + 1] + slot * warps;
            if ((t & 31) == 0) {
                a[warp] = s1;
                b[warp] = s2;
            }
            team_barrier(id, team);
            s1 = 0.f;
            s2 = 0.f;
            for (int w = 0; w < warps; ++w) {
                s1 += a[w];
                s2 += b[w];
            }
            phase ^= 1;
        }
        s1 *= inv_cols;
        s2 *= inv_cols;
        for_columns<NV, ALIGNED>(team, t, p.cols, [&](int i, int c) {
#pragma unroll
            for (int k = i; k < i + W; ++k) gy[k] = (gy[k] - s1 - xh[k] * s2) * rstd;
            if constexpr (ALIGNED) store8<XF32>(p.y, row * p.xs + c, gy + i);
            else store1<XF32>(p.y, row * p.xs + c, gy[i]);
        });
    }
    if (!p.dweight && !p.dbias) return;
    // the teams' sums, added in team order, then one row of partial sums for the block
    const int cols = p.cols;
    if (teams > 1) {
        for_columns<NV, ALIGNED>(team, t, cols, [&](int i, int c) {
#pragma unroll
            for (int k = 0; k < W; ++k) {
                dyn[(slot * 2) * cols + c + k] = dw[i + k];
                dyn[(slot * 2 + 1) * cols + c + k] = db[i + k];
            }
        });
        __syncthreads();
        for (int c = slot * team + t; c < 2 * cols; c += team * teams) {
            const int which = c >= cols, cc = c - which * cols;
            float s = 0.f;
            for (int j = 0; j < teams; ++j) s += dyn[(2 * j + which) * cols + cc];
            float* out = p.slices > 1 ? p.partial + (static_cast<int64_t>(blockIdx.x) * 2 + which) * cols
                                      : (which ? p.dbias : p.dweight);
            if (p.slices == 1 && out) out += group * cols;
            if (out) out[cc] = s;
        }
    } else {
        for_columns<NV, ALIGNED>(team, t, cols, [&](int i, int c) {
#pragma unroll
            for (int k = 0; k < W; ++k) {
                if (p.slices > 1) {
                    p.partial[(static_cast<int64_t>(blockIdx.x) * 2) * cols + c + k] = dw[i + k];
                    p.partial[(static_cast<int64_t>(blockIdx.x) * 2 + 1) * cols + c + k] = db[i + k];
                } else {
                    if (p.dweight) p.dweight[group * cols + c + k] = dw[i + k];
                    if (p.dbias) p.dbias[group * cols + c + k] = db[i + k];
                }
            }
        });
    }
}

// Sums the slices of 32 columns: thread (column, lane) adds slices lane, lane + 16, ..., then the
// 16 lanes' sums are added in order.  grid: (columns / 32, groups, 2).
constexpr int kFoldLanes = 16;

__global__ void __launch_bounds__(32 * kFoldLanes) norm_fold_kernel(const float* partial, int slices, int cols,
                                                                    float* dweight, float* dbias)
{
    float* out = blockIdx.z ? dbias : dweight;
    if (!out) return;
    __shared__ float part[kFoldLanes][32];
    const int c = blockIdx.x * 32 + threadIdx.x;
    const int64_t group = blockIdx.y;
    float s = 0.f;
    if (c < cols)
        for (int i = threadIdx.y; i < slices; i += kFoldLanes)
            s += partial[((group * slices + i) * 2 + blockIdx.z) * cols + c];
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < cols) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < kFoldLanes; ++i) s += part[i][threadIdx.x];
        out[group * cols + c] = s;
    }
}

int round32(int n) { return (n + 31) / 32 * 32; }

// Vectors of 8 columns per thread and threads per row.
struct Team {
    int nv, threads;
};

Team forward_team(int cols)
{
    const int vecs = (cols + 7) / 8;
    if (vecs <= 32) return {1, 32};
    if (vecs <= 64) return {2, 32};
    if (vecs <= 128) return {4, 32};
    if (vecs <= 192) return {6, 32};
    if (vecs <= 256) return {8, 32};
    if (vecs <= 512) return {1, round32(vecs)};
    if (vecs <= 1024) return {2, round32((vecs + 1) / 2)};
    return {4, round32((vecs + 3) / 4)};
}

Team backward_team(int cols)
{
    const int vecs = (cols + 7) / 8;
    if (vecs <= 512) return {1, round32(vecs)};
    if (vecs <= 1024) return {2, round32((vecs + 1) / 2)};
    return {4, round32((vecs + 3) / 4)};
}

int backward_teams(int cols) { return std::max(1, std::min(8, kMaxThreads / backward_team(cols).threads)); }

template <int NV, bool ALIGNED>
void forward_types(const NormParams& p, dim3 grid, dim3 block, cudaStream_t s)
{
    if (p.x_f32) {
        if (p.y_f32) norm_forward_kernel<NV, ALIGNED, true, true><<<grid, block, 0, s>>>(p);
        else norm_forward_kernel<NV, ALIGNED, true, false><<<grid, block, 0, s>>>(p);
    } else {
        if (p.y_f32) norm_forward_kernel<NV, ALIGNED, false, true><<<grid, block, 0, s>>>(p);
        else norm_forward_kernel<NV, ALIGNED, false, false><<<grid, block, 0, s>>>(p);
    }
}

template <int NV, bool ALIGNED>
void backward_types(const NormParams& p, dim3 grid, dim3 block, size_t smem, cudaStream_t s)
{
    if (p.x_f32) {
        if (p.y_f32) norm_backward_kernel<NV, ALIGNED, true, true><<<grid, block, smem, s>>>(p);
        else norm_backward_kernel<NV, ALIGNED, true, false><<<grid, block, smem, s>>>(p);
    } else {
        if (p.y_f32) norm_backward_kernel<NV, ALIGNED, false, true><<<grid, block, smem, s>>>(p);
        else norm_backward_kernel<NV, ALIGNED, false, false><<<grid, block, smem, s>>>(p);
    }
}

}  // namespace

int norm_backward_slices(int64_t rows, int64_t rows_per_group, int cols)
{
    // about two blocks for each of the 152 SMs, and no block without rows
    const int64_t groups = (rows + rows_per_group - 1) / rows_per_group;
    const int64_t want = (304 + groups - 1) / groups;
    const int64_t teams = backward_teams(cols);
    return static_cast<int>(std::max<int64_t>(1, std::min(want, (std::min(rows, rows_per_group) + teams - 1) / teams)));
}

cudaError_t launch_layer_norm(const NormParams& p, cudaStream_t s)
{
    const Team tm = forward_team(p.cols);
    const int teams = tm.threads == 32 ? 4 : 1;
    const dim3 block(static_cast<unsigned>(tm.threads), static_cast<unsigned>(teams));
    const dim3 grid(static_cast<unsigned>((p.rows + teams - 1) / teams));
    switch (tm.nv) {
    case 1: p.aligned ? forward_types<1, true>(p, grid, block, s) : forward_types<1, false>(p, grid, block, s); break;
    case 2: p.aligned ? forward_types<2, true>(p, grid, block, s) : forward_types<2, false>(p, grid, block, s); break;
    case 4: p.aligned ? forward_types<4, true>(p, grid, block, s) : forward_types<4, false>(p, grid, block, s); break;
    case 6: p.aligned ? forward_types<6, true>(p, grid, block, s) : forward_types<6, false>(p, grid, block, s); break;
    default: p.aligned ? forward_types<8, true>(p, grid, block, s) : forward_types<8, false>(p, grid, block, s); break;
    }
    return cudaGetLastError();
}

cudaError_t launch_layer_norm_backward(const NormParams& p, cudaStream_t s)
{
    const Team tm = backward_team(p.cols);
    const int teams = backward_teams(p.cols);
    const int64_t groups = (p.rows + p.rows_per_group - 1) / p.rows_per_group;
    const dim3 block(static_cast<unsigned>(tm.threads), static_cast<unsigned>(teams));
    const dim3 grid(static_cast<unsigned>(groups * p.slices));
    // at most 2 teams * 2 * 2048 columns * 4 bytes: a team of up to 256 threads holds 8 columns each
    const size_t smem = teams > 1 ? static_cast<size_t>(teams) * 2 * p.cols * sizeof(float) : 0;
    switch (tm.nv) {
    case 1: p.aligned ? backward_types<1, true>(p, grid, block, smem, s) : backward_types<1, false>(p, grid, block, smem, s); break;
    case 2: p.aligned ? backward_types<2, true>(p, grid, block, smem, s) : backward_types<2, false>(p, grid, block, smem, s); break;
    default: p.aligned ? backward_types<4, true>(p, grid, block, smem, s) : backward_types<4, false>(p, grid, block, smem, s); break;
    }
    if (p.slices > 1 && (p.dweight || p.dbias)) {
        const dim3 fold(static_cast<unsigned>((p.cols + 31) / 32), static_cast<unsigned>(groups), 2);
        norm_fold_kernel<<<fold, dim3(32, kFoldLanes), 0, s>>>(p.partial, p.slices, p.cols, p.dweight, p.dbias);
    }
    return cudaGetLastError();
}

}  // namespace sdv2
