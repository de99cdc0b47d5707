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
// between.  What decides the rate is how many rows are on their way while a row's sums are exchanged
// between threads, so a team of threads walks over rows that it copies ahead into its own part of
// shared memory (cp.async; every thread reads back only what it copied, so no barrier is needed for
// it).  A row at a time without that took 2 us a row: 38.7 us for the 14B forward, 18.7 us for the
// 1.3B backward.  Rows that do not start on 16 bytes are read element by element, one row ahead in
// registers.  A thread holds vectors of eight neighbouring columns (of four where x or y is fp32, so that a
// warp reads whole sectors: 32 bytes a thread in two copies of 16 took 42.9 us for the 14B forward),
// and as many of them as registers allow, with the group's gain and bias, and works on pairs of them (f32x2): with one instruction per
// operation and column, and a test of every vector against the row's end, a row took 695
// instructions a warp and the 14B forward 43.4 us.  Rows whose vectors fill their threads exactly need
// no such test (kFull).
// The forward pass takes rows in pairs where registers hold two: they share their barriers, and each hides the other's
// reductions (14B forward, 4680 x 5120 fp32 to bf16: 31.8 us one by one, 24.9 in pairs, 5.8 TB/s; a plain
// copy of the same bytes takes 21.7).  Fewer instructions did not help it (running pointers: 31.8 us).  The backward pass
// keeps three values a column over all rows besides the row's own two, and pairs spill (4680 x 1536 bf16: 16.1 us one by
// one, 21.9 in pairs): what bounds it is the issue of 430 instructions a warp and row by 15 warps of an SM.
// The parameter sums of a group are split over `slices` blocks, each of which keeps its columns' sums
// in registers over all of its rows and writes them once; a second kernel adds the slices in index
// order, so the result does not depend on the order in which blocks run.
#include <algorithm>

#include "block.h"
#include "chained.cuh"
#include "per_device.h"
#include "softmax_tile.cuh"

namespace sdv2 {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kSms = 152;

// How a row's elements are reached: one by one, in vectors of eight, and in vectors that fill all threads.
enum Rows { kSingle, kVector, kFull };

__device__ __forceinline__ uint64_t both(float v) { return f32x2_pack(v, v); }
__device__ __forceinline__ float add_pair(uint64_t v)
{
    float a, b;
    f32x2_unpack(v, a, b);
    return a + b;
}

// Columns of a vector.
constexpr int columns(bool x_f32, bool y_f32) { return x_f32 || y_f32 ? 4 : 8; }

// The first n of C consecutive columns of a row that is not aligned, and 0 in the rest, as pairs.
template <int C, bool F32>
__device__ __forceinline__ void load_part(const void* base, int64_t i, int n, uint64_t* v)
{
    float x[C];
#pragma unroll
    for (int k = 0; k < C; ++k) {
        x[k] = 0.f;
        if (k < n) {
            if constexpr (F32) x[k] = static_cast<const float*>(base)[i + k];
            else x[k] = __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(base)[i + k]) << 16);
        }
    }
#pragma unroll
    for (int k = 0; k < C / 2; ++k) v[k] = f32x2_pack(x[2 * k], x[2 * k + 1]);
}

// Stores n of C columns; all of them at once where VECTOR.
template <int C, bool F32, bool VECTOR>
__device__ __forceinline__ void store_columns(void* base, int64_t i, int n, const uint64_t* v)
{
    float x[C];
#pragma unroll
    for (int k = 0; k < C / 2; ++k) f32x2_unpack(v[k], x[2 * k], x[2 * k + 1]);
    if constexpr (!VECTOR) {
#pragma unroll
        for (int k = 0; k < C; ++k)
            if (k < n) {
                if constexpr (F32) static_cast<float*>(base)[i + k] = x[k];
                else static_cast<__nv_bfloat16*>(base)[i + k] = __float2bfloat16_rn(x[k]);
            }
    } else if constexpr (F32) {
        static_assert(C == 4, "fp32 vectors have four columns");
        *reinterpret_cast<float4*>(static_cast<float*>(base) + i) = make_float4(x[0], x[1], x[2], x[3]);
    } else if constexpr (C == 4) {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + i) = make_uint2(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]));
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + i) =
            make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
    }
}

// C parameters (fp32, which no output overlaps) as pairs.
template <int C>
__device__ __forceinline__ void load_param(const float* p, bool vector, int n, uint64_t* v)
{
    float x[C];
    if (vector) {
#pragma unroll
        for (int k = 0; k < C; k += 4) {
            const float4 a = *reinterpret_cast<const float4*>(p + k);
            x[k] = a.x; x[k + 1] = a.y; x[k + 2] = a.z; x[k + 3] = a.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < C; ++k) x[k] = k < n ? p[k] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < C / 2; ++k) v[k] = f32x2_pack(x[2 * k], x[2 * k + 1]);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void copy8(uint32_t dst, const void* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// All but the newest N groups of this thread's copies have landed.
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// 1 / sqrt(v) within a step: one of Newton's steps from the hardware's estimate, which is within two.  The step has no
// value where the estimate is 0 or infinite.  A division by a square root took two calls with branches.
__device__ __forceinline__ float reciprocal_root(float v)
{
    const float r = rsqrtf(v);
    const float better = fmaf(r, fmaf(-0.5f * v * r, r, 0.5f), r);
    return v > 0.f && v < INFINITY ? better : r;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The same over lanes 0-15, for every lane (a team has at most 16 warps).
__device__ __forceinline__ float warp_sum16(float v)
{
    v += __shfl_xor_sync(0xffffffffu, v, 8);
    v += __shfl_xor_sync(0xffffffffu, v, 4);
    v += __shfl_xor_sync(0xffffffffu, v, 2);
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return __shfl_sync(0xffffffffu, v, 0);
}

__device__ __forceinline__ void team_barrier(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// R sums over the `warps` warps of a team; every thread gets the same values (both levels are fixed trees).
// `scratch` holds R floats per warp; `id` is the team's barrier.
template <int R>
__device__ __forceinline__ void team_sums(float (&v)[R], int warps, int warp, float* scratch, int id)
{
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = warp_sum(v[r]);
    if (warps == 1) return;
    const int lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
        for (int r = 0; r < R; ++r) scratch[r * warps + warp] = v[r];
    team_barrier(id, warps * 32);
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = warp_sum16(lane < warps ? scratch[r * warps + lane] : 0.f);
}

// A thread's columns: N vectors of C, vector i starting at column C*(i*team + t).  f(first pair of the vector,
// column, how many of its columns the row has).
template <int N, int C, Rows MODE, typename F>
__device__ __forceinline__ void for_vectors(int team, int t, int cols, F&& f)
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = C * (i * team + t);
        if constexpr (MODE == kFull) f(i * (C / 2), c, C);
        else if (c < cols) f(i * (C / 2), c, min(C, cols - c));
    }
}

// A thread's vectors of one row of x or dy, copied ahead: vector i of slot `slot` lies at
// base + (slot*N + i) * threads * BYTES; base is the thread's own.
template <int N, int C, bool F32, Rows MODE>
struct Ring {
    static constexpr int BYTES = C * (F32 ? 4 : 2);
    uint32_t base;
    int threads;
    __device__ uint32_t at(int slot, int i) const { return base + (slot * N + i) * threads * BYTES; }
    // row: the row's first element
    __device__ void copy(int slot, const char* row, int team, int t, int cols) const
    {
        const char* src = row + t * BYTES;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (MODE == kFull || C * (i * team + t) < cols) {
                if constexpr (BYTES == 16) copy16(at(slot, i), src + i * team * BYTES);
                else copy8(at(slot, i), src + i * team * BYTES);
            }
    }
    __device__ void read(int slot, int team, int t, int cols, uint64_t* v) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            uint32_t w[BYTES / 4] = {};
            if (MODE == kFull || C * (i * team + t) < cols) {
                if constexpr (BYTES == 16)
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at(slot, i)) : "memory");
                else asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at(slot, i)) : "memory");
            }
#pragma unroll
            for (int k = 0; k < C / 2; ++k) {
                if constexpr (F32) v[(C / 2) * i + k] = f32x2_pack(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
                else v[(C / 2) * i + k] = f32x2_pack(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
            }
        }
    }
};

// Rows copied ahead: up to 384 bytes a thread, of at most 512 threads (the widest rows of two fp32 tensors have 256 each).
constexpr int stages(int bytes_per_row)
{
    return bytes_per_row <= 32 ? 6 : bytes_per_row <= 48 ? 4 : bytes_per_row <= 64 ? 3 : bytes_per_row <= 192 ? 2 : 1;
}
// In the forward pass, which takes rows in pairs where registers hold two: up to 256 bytes.
constexpr int forward_stages(int bytes_per_row) { return bytes_per_row <= 32 ? 6 : bytes_per_row <= 64 ? 4 : 2; }
// Threads that the kernel is compiled for, which caps its registers: by them the launch counts the blocks of an SM.
constexpr int forward_bound(int nv, Rows mode) { return mode == kSingle || nv > 2 ? 512 : nv == 2 ? 640 : 1024; }
constexpr int forward_registers(int nv, Rows mode) { return 65536 / forward_bound(nv, mode) / 8 * 8; }
constexpr int forward_rows(int nv, Rows mode, bool x_f32) { return mode != kSingle && (nv == 2 || (nv == 3 && !x_f32)) ? 2 : 1; }

__device__ __forceinline__ uint32_t shared_address(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ const char* row_of(const void* base, int64_t row, int64_t stride, bool f32)
{
    return static_cast<const char*>(base) + row * stride * (f32 ? 4 : 2);
}

// blockDim = (team, teams): a team takes the rows of its index, then every gridDim * teams further.
template <int NV, Rows MODE, bool XF32, bool YF32>
__global__ void __launch_bounds__(forward_bound(NV, MODE)) norm_forward_kernel(const NormParams p)
{
    constexpr bool VECTOR = MODE != kSingle;
    constexpr int C = columns(XF32, YF32), N = NV * 8 / C;
    constexpr int S = forward_stages(NV * 16 * (XF32 ? 2 : 1)), R = forward_rows(NV, MODE, XF32);
    constexpr bool EARLY = !VECTOR || NV == 1;
    extern __shared__ __align__(16) uint8_t copied[];
    __shared__ float scratch[2][2][R * kMaxThreads / 32];
    const int team = blockDim.x, t = threadIdx.x;
    const int warps = team >> 5, warp = t >> 5;
    const int id = 1 + threadIdx.y;
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.y;
    int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (row >= p.rows) return;                         // whole team: its barrier is its own
    wait_for_launch_before();
    using RingX = Ring<N, C, XF32, MODE>;
    const RingX ring{shared_address(copied) + (threadIdx.y * team + t) * RingX::BYTES, team * static_cast<int>(blockDim.y)};
    uint64_t next[VECTOR ? 1 : NV * 4];                // single elements: the next row
    auto fetch = [&](int64_t r) {
        for_vectors<N, C, MODE>(team, t, p.cols, [&](int i, int c, int n) { load_part<C, XF32>(p.x, r * p.xs + c, n, next + i); });
    };
    if constexpr (VECTOR) {
#pragma unroll
        for (int k = 0; k < S; ++k) {
            if (row + k * step < p.rows) ring.copy(k, row_of(p.x, row + k * step, p.xs, XF32), team, t, p.cols);
            copy_commit();
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV * 4; ++i) next[i] = 0;
        fetch(row);
    }
    const float inv_cols = 1.0f / static_cast<float>(p.cols);
    uint64_t gain[NV * 4], bias[NV * 4];
    int64_t group_end = 0;
    int slot = 0, phase = 0;
    auto parameters = [&](int64_t r) {
        if (r >= group_end) {
            const int64_t group = r / p.rows_per_group;
            group_end = (group + 1) * p.rows_per_group;
            for_vectors<N, C, MODE>(team, t, p.cols, [&](int i, int c, int n) {
#pragma unroll
                for (int k = i; k < i + C / 2; ++k) {
                    gain[k] = both(1.f);
                    bias[k] = 0;
                }
                if (p.weight) {
                    load_param<C>(p.weight + group * p.gs + c, VECTOR, n, gain + i);
                    if (p.plus_one)
#pragma unroll
                        for (int k = i; k < i + C / 2; ++k) gain[k] = fadd2(gain[k], both(1.f));
                }
                if (p.bias) load_param<C>(p.bias + group * p.gs + c, VECTOR, n, bias + i);
            });
        }
    };
#pragma unroll 1
    for (; row < p.rows; row += R * step) {
        // A short row's time is one latency after the other, so that they are loaded in front of the sums (72 x 256: 1.8 us,
        // 2.0 behind; 3001 x 1001: 14.0, 15.0); others have the registers for the row then (4680 x 5120: 27.3 us, 24.8 behind).
        if constexpr (EARLY) parameters(row);
        uint64_t v[R][NV * 4];
        if constexpr (VECTOR) {
            copy_wait<S - R>();
#pragma unroll
            for (int k = 0; k < R; ++k) {
                ring.read(slot, team, t, p.cols, v[k]);
                if (row + (S + k) * step < p.rows) ring.copy(slot, row_of(p.x, row + (S + k) * step, p.xs, XF32), team, t, p.cols);
                copy_commit();
                if (++slot == S) slot = 0;
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV * 4; ++i) v[0][i] = next[i];
            if (row + step < p.rows) fetch(row + step);
        }
        // a second row behind the last is worked on like any other (its slot holds something older) and not stored
        float mean[R], var[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            uint64_t two[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < NV * 4; ++i) two[i & 1] = fadd2(two[i & 1], v[k][i]);
            mean[k] = add_pair(fadd2(two[0], two[1]));
        }
        // two sets of scratch in turn: a warp that is an iteration ahead does not touch what others still read
        team_sums<R>(mean, warps, warp, scratch[phase][0] + threadIdx.y * warps * R, id);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            mean[k] *= inv_cols;
            uint64_t two[2] = {0, 0};
            const uint64_t minus = both(-mean[k]);
            for_vectors<N, C, MODE>(team, t, p.cols, [&](int i, int, int n) {
#pragma unroll
                for (int e = 0; e < C / 2; ++e) {
                    uint64_t d = fadd2(v[k][i + e], minus);
                    if constexpr (!VECTOR) {           // columns past the row's end stay 0
                        float a, b;
                        f32x2_unpack(d, a, b);
                        d = f32x2_pack(2 * e < n ? a : 0.f, 2 * e + 1 < n ? b : 0.f);
                    }
                    v[k][i + e] = d;
                    two[e & 1] = ffma2(d, d, two[e & 1]);
                }
            });
            var[k] = add_pair(fadd2(two[0], two[1]));
        }
        team_sums<R>(var, warps, warp, scratch[phase][1] + threadIdx.y * warps * R, id);
        phase ^= 1;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int64_t r = row + k * step;
            if (k > 0 && r >= p.rows) break;
            const float rstd = reciprocal_root(fmaf(var[k], inv_cols, p.eps));
            if (t == 0) {
                if (p.mean) p.mean[r] = mean[k];
                if (p.rstd) p.rstd[r] = rstd;
            }
            if constexpr (!EARLY) parameters(r);
            const uint64_t rstd2 = both(rstd);
            for_vectors<N, C, MODE>(team, t, p.cols, [&](int i, int c, int n) {
                uint64_t y[C / 2];
#pragma unroll
                for (int e = 0; e < C / 2; ++e) y[e] = ffma2(fmul2(v[k][i + e], rstd2), gain[i + e], bias[i + e]);
                store_columns<C, YF32, VECTOR>(p.y, r * p.ys + c, n, y);
            });
        }
    }
}

// blockDim = (team, teams); block (group, slice): its teams take the group's rows slice*teams + team, then
// every slices*teams further.  Each thread keeps dgain and dbias of its columns.
template <int NV, Rows MODE, bool XF32, bool YF32>
__global__ void __launch_bounds__(kMaxThreads, NV == 1 && MODE != kSingle ? 2 : 1) norm_backward_kernel(const NormParams p)
{
    launch_dependents();                       // the fold (4680 x 1536: 20.7 us in a stream unchained, 18.8 chained)
    constexpr bool VECTOR = MODE != kSingle;
    constexpr int C = columns(XF32, YF32), N = NV * 8 / C;
    constexpr int S = stages(NV * 16 * ((XF32 ? 2 : 1) + (YF32 ? 2 : 1)));
    extern __shared__ __align__(16) uint8_t copied[];  // the rows copied ahead; at the end the teams' sums [teams][2][cols]
    float* dyn = reinterpret_cast<float*>(copied);
    __shared__ float scratch[2][2 * kMaxThreads / 32];
    const int team = blockDim.x, t = threadIdx.x, teams = blockDim.y, slot_id = threadIdx.y;
    const int warps = team >> 5, warp = t >> 5;
    const int id = 1 + slot_id;
    const uint32_t group = blockIdx.x / static_cast<uint32_t>(p.slices);
    const int slice = static_cast<int>(blockIdx.x - group * p.slices);
    const int64_t row_end = min(p.rows, (group + int64_t(1)) * p.rows_per_group);
    const int64_t step = static_cast<int64_t>(p.slices) * teams;
    const int64_t g = group * p.gs;
    const float inv_cols = 1.0f / static_cast<float>(p.cols);
    const int threads = team * teams, tid = slot_id * team + t;
    using RingX = Ring<N, C, XF32, MODE>;
    using RingY = Ring<N, C, YF32, MODE>;
    const RingX ring_x{shared_address(copied) + tid * RingX::BYTES, threads};
    const RingY ring_y{shared_address(copied) + S * N * threads * RingX::BYTES + tid * RingY::BYTES, threads};

    int64_t row = group * p.rows_per_group + static_cast<int64_t>(slice) * teams + slot_id;
    uint64_t next_x[VECTOR ? 1 : NV * 4], next_y[VECTOR ? 1 : NV * 4];  // single elements: the next row
    auto fetch = [&](int64_t r) {
        for_vectors<N, C, MODE>(team, t, p.cols, [&](int i, int c, int n) {
            load_part<C, XF32>(p.x, r * p.xs + c, n, next_x + i);
            load_part<C, YF32>(p.dy, r * p.ys + c, n, next_y + i);
        });
    };
    auto copy = [&](int slot, int64_t r) {
        ring_x.copy(slot, row_of(p.x, r, p.xs, XF32), team, t, p.cols);
        ring_y.copy(slot, row_of(p.dy, r, p.ys, YF32), team, t, p.cols);
    };
    wait_for_launch_before();
    float next_mean = 0.f, next_rstd = 0.f;
    if (row < row_end) {
        next_mean = p.mean[row];
        next_rstd = p.rstd[row];
    }
    if constexpr (VECTOR) {
#pragma unroll
        for (int k = 0; k < S; ++k) {
            if (row + k * step < row_end) copy(k, row + k * step);
            copy_commit();
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV * 4; ++i) {
            next_x[i] = 0;
            next_y[i] = 0;
        }
        if (row < row_end) fetch(row);
    }
    uint64_t dw[NV * 4], db[NV * 4], gain[NV * 4];
#pragma unroll
    for (int i = 0; i < NV * 4; ++i) {
        dw[i] = 0;
        db[i] = 0;
        gain[i] = both(1.f);
    }
    if (p.weight)
        for_vectors<N, C, MODE>(team, t, p.cols, [&](int i, int c, int n) {
            load_param<C>(p.weight + g + c, VECTOR, n, gain + i);
            if (p.plus_one)
#pragma unroll
                for (int k = i; k < i + C / 2; ++k) gain[k] = fadd2(gain[k], both(1.f));
        });
    int slot = 0, phase = 0;
#pragma unroll 1
    for (; row < row_end; row += step) {
        uint64_t xh[NV * 4], gy[NV * 4];
        const uint64_t mean = both(-next_mean), rstd = both(next_rstd);
        if (row + step < row_end) {
            next_mean = p.mean[row + step];
            next_rstd = p.rstd[row + step];
        }
        if constexpr (VECTOR) {
            copy_wait<S - 1>();
            ring_x.read(slot, team, t, p.cols, xh);
            ring_y.read(slot, team, t, p.cols, gy);
            if (row + S * step < row_end) copy(slot, row + S * step);
            copy_commit();
            if (++slot == S) slot = 0;
        } else {
#pragma unroll
            for (int i = 0; i < NV * 4; ++i) {
                xh[i] = next_x[i];
                gy[i] = next_y[i];
            }
            if (row + step < row_end) fetch(row + step);
        }
        // past the row's end dy is 0, and so is what it multiplies
        uint64_t sum0[2] = {0, 0}, sum1[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < NV * 4; ++k) {
            xh[k] = fmul2(fadd2(xh[k], mean), rstd);
            dw[k] = ffma2(gy[k], xh[k], dw[k]);
            db[k] = fadd2(db[k], gy[k]);
            gy[k] = fmul2(gy[k], gain[k]);
            sum0[k & 1] = fadd2(sum0[k & 1], gy[k]);
            sum1[k & 1] = ffma2(gy[k], xh[k], sum1[k & 1]);
        }
        float s[2] = {add_pair(fadd2(sum0[0], sum0[1])), add_pair(fadd2(sum1[0], sum1[1]))};
        // two scratch rows in turn: a warp that is a row ahead does not touch what others still read
        team_sums<2>(s, warps, warp, scratch[phase] + slot_id * warps * 2, id);
        phase ^= 1;
        const uint64_t minus0 = both(-s[0] * inv_cols), minus1 = both(-s[1] * inv_cols);
        for_vectors<N, C, MODE>(team, t, p.cols, [&](int i, int c, int n) {
            uint64_t d[C / 2];
#pragma unroll
            for (int k = 0; k < C / 2; ++k) d[k] = fmul2(ffma2(xh[i + k], minus1, fadd2(gy[i + k], minus0)), rstd);
            store_columns<C, XF32, VECTOR>(p.y, row * p.xs + c, n, d);
        });
    }
    if (!p.dweight && !p.dbias) return;
    // the teams' sums, added in team order, then one row of partial sums for the block
    const int cols = p.cols;
    if (teams > 1) {
        if constexpr (VECTOR) copy_wait<0>();
        __syncthreads();                               // every team is done with the rows copied ahead
        for_vectors<N, C, MODE>(team, t, cols, [&](int i, int c, int n) {
            store_columns<C, true, false>(dyn, (slot_id * 2) * cols + c, n, dw + i);
            store_columns<C, true, false>(dyn, (slot_id * 2 + 1) * cols + c, n, db + i);
        });
        __syncthreads();
        for (int c = tid; c < 2 * cols; c += threads) {
            const int which = c >= cols, cc = c - which * cols;
            float sum = 0.f;
            for (int j = 0; j < teams; ++j) sum += dyn[(2 * j + which) * cols + cc];
            float* out = p.slices > 1 ? p.partial + (static_cast<int64_t>(blockIdx.x) * 2 + which) * cols
                                      : (which ? p.dbias : p.dweight);
            if (p.slices == 1 && out) out += static_cast<int64_t>(group) * cols;
            if (out) out[cc] = sum;
        }
    } else {
        for_vectors<N, C, MODE>(team, t, cols, [&](int i, int c, int n) {
            if (p.slices > 1) {
                store_columns<C, true, false>(p.partial, (static_cast<int64_t>(blockIdx.x) * 2) * cols + c, n, dw + i);
                store_columns<C, true, false>(p.partial, (static_cast<int64_t>(blockIdx.x) * 2 + 1) * cols + c, n, db + i);
            } else {
                if (p.dweight) store_columns<C, true, false>(p.dweight, static_cast<int64_t>(group) * cols + c, n, dw + i);
                if (p.dbias) store_columns<C, true, false>(p.dbias, static_cast<int64_t>(group) * cols + c, n, db + i);
            }
        });
    }
}

// Sums the slices of 32 columns: thread (column, lane) adds slices lane, lane + 32, ..., then the 32 lanes'
// sums are added in a fixed tree.  grid: (columns / 32, groups, 2).
constexpr int kFoldLanes = 32;

__global__ void __launch_bounds__(32 * kFoldLanes) norm_fold_kernel(const float* partial, int slices, int cols,
                                                                    float* dweight, float* dbias)
{
    float* out = blockIdx.z ? dbias : dweight;
    wait_for_launch_before();
    if (!out) return;
    __shared__ float part[kFoldLanes][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    const int64_t group = blockIdx.y;
    const float* src = partial + ((group * slices + threadIdx.y) * 2 + blockIdx.z) * cols + c;
    const int64_t step = static_cast<int64_t>(kFoldLanes) * 2 * cols;
    float s = 0.f;
    if (c < cols) {
#pragma unroll 4
        for (int i = threadIdx.y; i < slices; i += kFoldLanes, src += step) s += *src;
    }
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    // warp y adds column y: its lanes hold the 32 sums, added in a fixed tree
    s = warp_sum(part[threadIdx.x][threadIdx.y]);
    const int cc = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && cc < cols) out[group * cols + cc] = s;
}

int round32(int n) { return (n + 31) / 32 * 32; }

// Vectors of 8 columns per thread, threads per row, how its elements are reached.
struct Team {
    int nv, threads;
    Rows mode;
};

Team forward_team(int cols, bool aligned, bool x_f32)
{
    const int vecs = (cols + 7) / 8;
    if (!aligned) {                                    // the next row takes registers as well
        if (vecs <= 32) return {1, 32, kSingle};
        if (vecs <= 1024) return {2, round32((vecs + 1) / 2), kSingle};
        return {4, round32((vecs + 3) / 4), kSingle};
    }
    // Widths whose rows go in pairs first: three vectors where x is bf16 and the row narrow (fewer warps exchange: 768
    // columns 7.2 us, 11.5 with one; 1536: 8.1, 9.0 with two), two otherwise (1536 fp32: 11.9 us, 17.8 with three and
    // rows one by one; 2048: 10.5, 12.2 with four; 5120 before pairs: 32.3 with two, 35.3 with four).
    const int order[2][3] = {{3, 2, 1}, {2, 3, 1}};
    for (int nv : order[x_f32])
        if (vecs % (32 * nv) == 0 && vecs / nv <= kMaxThreads && (nv < 3 || vecs <= 256)) return {nv, vecs / nv, kFull};
    if (vecs <= 32) return {1, 32, kVector};
    if (vecs <= 64) return {2, 32, kVector};
    if (vecs <= 128) return {4, 32, kVector};          // one warp exchanges nothing (640: 8.6 us, 11.5 in pairs with two)
    if (vecs <= 1024) return {2, round32((vecs + 1) / 2), kVector};
    return {4, round32((vecs + 3) / 4), kVector};
}

Team backward_team(int cols, bool aligned)
{
    const int vecs = (cols + 7) / 8;
    if (!aligned) {
        if (vecs <= 512) return {1, round32(vecs), kSingle};
        if (vecs <= 1024) return {2, round32((vecs + 1) / 2), kSingle};
        return {4, round32((vecs + 3) / 4), kSingle};
    }
    for (int nv = 2; nv >= 1; --nv)
        if (vecs % (32 * nv) == 0 && vecs / nv <= kMaxThreads) return {nv, vecs / nv, kFull};
    if (vecs <= 32) return {1, 32, kVector};
    if (vecs <= 1024) return {2, round32((vecs + 1) / 2), kVector};
    return {4, round32((vecs + 3) / 4), kVector};
}

int backward_teams(int cols, bool aligned) { return std::max(1, std::min(15, kMaxThreads / backward_team(cols, aligned).threads)); }

// Blocks of the backward kernel that an SM holds, by its registers.
int backward_blocks(int cols, bool aligned) { return aligned && backward_team(cols, aligned).nv == 1 ? 2 : 1; }

// Dynamic shared memory that every kernel may take.  One limit, set once: it is the kernel's, not the launch's, and a
// call that set its own size would take it from a launch that another host thread is about to make.
constexpr size_t kMaxShared = 220 * 1024;

template <typename K>
cudaError_t allow_shared(K kernel, PerDevice& allowed)
{
    int dev = 0;
    cudaGetDevice(&dev);
    return allowed.run(dev, [&]() {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMaxShared));
    });
}

template <int NV, Rows MODE, bool XF32, bool YF32>
cudaError_t forward(const NormParams& p, int threads, cudaStream_t s)
{
    constexpr int S = forward_stages(NV * 16 * (XF32 ? 2 : 1));
    constexpr int kBytes = MODE != kSingle ? S * NV * 16 * (XF32 ? 2 : 1) : 0;          // of shared memory per thread
    // teams of a block: none idle while there are SMs without one
    const int64_t spread = (p.rows + kSms - 1) / kSms;
    const int teams = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min(15, kMaxThreads / threads), spread)));
    const int block = teams * threads;
    // resident blocks: by shared memory, and by registers
    const int fit = std::max(1, std::min(kBytes ? static_cast<int>(kMaxShared) / (kBytes * block + 1024) : 8, 65536 / (forward_registers(NV, MODE) * block)));
    const int64_t grid = std::min<int64_t>((p.rows + teams - 1) / teams, static_cast<int64_t>(kSms) * fit);
    const size_t smem = static_cast<size_t>(kBytes) * block;
    auto kernel = norm_forward_kernel<NV, MODE, XF32, YF32>;
    static PerDevice allowed;
    const cudaError_t e = allow_shared(kernel, allowed);
    if (e != cudaSuccess) return e;
    return launch_chained(kernel, dim3(static_cast<unsigned>(grid)), dim3(static_cast<unsigned>(threads), static_cast<unsigned>(teams)),
                          smem, s, p);
}

template <int NV, Rows MODE, bool XF32, bool YF32>
cudaError_t backward(const NormParams& p, int threads, cudaStream_t s)
{
    constexpr int S = stages(NV * 16 * ((XF32 ? 2 : 1) + (YF32 ? 2 : 1)));
    constexpr int kBytes = MODE != kSingle ? S * NV * 16 * ((XF32 ? 2 : 1) + (YF32 ? 2 : 1)) : 0;
    const int teams = backward_teams(p.cols, MODE != kSingle);
    const int64_t groups = (p.rows + p.rows_per_group - 1) / p.rows_per_group;
    const size_t sums = teams > 1 ? static_cast<size_t>(teams) * 2 * p.cols * sizeof(float) : 0;
    const size_t smem = std::max(sums, static_cast<size_t>(kBytes) * threads * teams);
    auto kernel = norm_backward_kernel<NV, MODE, XF32, YF32>;
    static PerDevice allowed;
    const cudaError_t e = allow_shared(kernel, allowed);
    if (e != cudaSuccess) return e;
    return launch_chained(kernel, dim3(static_cast<unsigned>(groups * p.slices)),
                          dim3(static_cast<unsigned>(threads), static_cast<unsigned>(teams)), smem, s, p);
}

// Calls f<NV, MODE, XF32, YF32>(p, threads, s) for the row's width, alignment and types.
#define SDV2_NORM_TYPES(f, NV, MODE)                                                                        \
    (p.x_f32 ? (p.y_f32 ? f<NV, MODE, true, true>(p, tm.threads, s) : f<NV, MODE, true, false>(p, tm.threads, s)) \
             : (p.y_f32 ? f<NV, MODE, false, true>(p, tm.threads, s) : f<NV, MODE, false, false>(p, tm.threads, s)))
#define SDV2_NORM(f, NV)                                   \
    (tm.mode == kFull ? SDV2_NORM_TYPES(f, NV, kFull)      \
                      : tm.mode == kVector ? SDV2_NORM_TYPES(f, NV, kVector) : SDV2_NORM_TYPES(f, NV, kSingle))

}  // namespace

int norm_backward_slices(int64_t rows, int64_t rows_per_group, int cols, bool aligned)
{
    // the blocks that the 152 SMs hold at once, and no block without rows
    const int64_t groups = (rows + rows_per_group - 1) / rows_per_group;
    const int64_t want = std::max<int64_t>(1, kSms * backward_blocks(cols, aligned) / groups);
    const int64_t teams = backward_teams(cols, aligned);
    return static_cast<int>(std::max<int64_t>(1, std::min(want, (std::min(rows, rows_per_group) + teams - 1) / teams)));
}

cudaError_t launch_layer_norm(const NormParams& p, cudaStream_t s)
{
    const Team tm = forward_team(p.cols, p.aligned, p.x_f32);
    switch (tm.nv) {
    case 1: return SDV2_NORM(forward, 1);
    case 2: return SDV2_NORM(forward, 2);
    case 3: return SDV2_NORM_TYPES(forward, 3, kFull);
    default: return tm.mode == kVector ? SDV2_NORM_TYPES(forward, 4, kVector) : SDV2_NORM_TYPES(forward, 4, kSingle);
    }
}

cudaError_t launch_layer_norm_backward(const NormParams& p, cudaStream_t s)
{
    const Team tm = backward_team(p.cols, p.aligned);
    cudaError_t e;
    switch (tm.nv) {
    case 1: e = SDV2_NORM(backward, 1); break;
    case 2: e = SDV2_NORM(backward, 2); break;
    default: e = tm.mode == kVector ? SDV2_NORM_TYPES(backward, 4, kVector) : SDV2_NORM_TYPES(backward, 4, kSingle); break;
    }
    if (e != cudaSuccess) return e;
    if (p.slices > 1 && (p.dweight || p.dbias)) {
        const int64_t groups = (p.rows + p.rows_per_group - 1) / p.rows_per_group;
        const dim3 fold(static_cast<unsigned>((p.cols + 31) / 32), static_cast<unsigned>(groups), 2);
        return launch_chained(norm_fold_kernel, fold, dim3(32, kFoldLanes), 0, s, p.partial, p.slices, p.cols, p.dweight, p.dbias);
    }
    return cudaSuccess;
}

#undef SDV2_NORM
#undef SDV2_NORM_TYPES

}  // namespace sdv2
