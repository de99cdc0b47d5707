// Rotary positions of several axes, forward and backward (the rotation by the negative angle).
//
// Every element is read and written once, so that memory bounds this.  A thread owns the same pairs of dims in many heads of a
// token: it finds their sines and cosines once and then only loads, turns and stores, six or twelve heads' loads under way together.  Pairs
// of neighbours lie in one vector of 16 bytes; pairs half a segment apart in two, as wide as every half segment is whole vectors of.
// q and k of 4680 x 12 heads in bf16 take 11.9 us, of 40 heads 32.9 (5.8 TB/s, 0.86 of a copy's rate), of one token 1.7.
// An angle in turns is position * scale * base^(-2j/d) / 2pi.  Its frequency is held as a 64-bit fraction of a turn (whole
// turns of it change nothing), so that the 64-bit product with the position, which wraps around, is the fraction of a turn that
// is left: off by 2^-64 of a turn per position.  The nearest quarter turn is taken off before the rest, at most an eighth, goes
// to fp32, where it is off by 2^-28 of a turn at most; sine and cosine of that are sums of their Taylor series.
#include <cuda_bf16.h>

#include <algorithm>

#include "chained.cuh"
#include "project.h"

namespace sdv2 {
namespace {

constexpr int kThreads = 128;              // of a block, at most: whole rows of items
// Heads whose loads are under way together.
template <int BYTES>
constexpr int kBatch = BYTES > 4 ? 6 : 12;

__device__ __forceinline__ float2 cos_sin(uint64_t turn)
{
    const uint32_t t = static_cast<uint32_t>(turn >> 32);
    const uint32_t quarter = (t + 0x20000000u) >> 30;
    const float a = static_cast<float>(static_cast<int32_t>(t - (quarter << 30))) * (6.2831853071795865f * 0x1p-32f);
    const float a2 = a * a;
    // terms up to a^9/9! and a^10/10!: at a = pi/4 the next are 2^-29 and 2^-33
    float s = fmaf(a2, 1.0f / 362880, -1.0f / 5040);
    s = fmaf(a2, s, 1.0f / 120);
    s = fmaf(a2, s, -1.0f / 6);
    s = fmaf(a * a2, s, a);
    float c = fmaf(a2, -1.0f / 3628800, 1.0f / 40320);
    c = fmaf(a2, c, -1.0f / 720);
    c = fmaf(a2, c, 1.0f / 24);
    c = fmaf(a2, c, -0.5f);
    c = fmaf(a2, c, 1.0f);
    const float x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;
    // a quarter turn takes (c, s) to (-s, c)
    return make_float2(__uint_as_float(__float_as_uint(x) ^ ((quarter + 1) << 30 & 0x80000000u)),
                       __uint_as_float(__float_as_uint(y) ^ (quarter << 30 & 0x80000000u)));
}

template <typename T, int N>
struct alignas(N * sizeof(T)) Pack {
    T e[N];
};

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }

template <int N>
__device__ __forceinline__ void narrow(Pack<float, N>& p, const float (&x)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) p.e[i] = x[i];
}

template <int N>
__device__ __forceinline__ void narrow(Pack<__nv_bfloat16, N>& p, const float (&x)[N])
{
    if constexpr (N == 1) {
        p.e[0] = __float2bfloat16_rn(x[0]);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const __nv_bfloat162 two = __floats2bfloat162_rn(x[i], x[i + 1]);
            p.e[i] = two.x;
            p.e[i + 1] = two.y;
        }
    }
}

// N: elements of a vector; ADJACENT: one of pairs of neighbours, else two of their first and second elements; ALL: every dim turns.
template <typename T, int N, bool ADJACENT, bool ALL>
__global__ void __launch_bounds__(kThreads) axes_rope_kernel(const __grid_constant__ AxesRopeParams p)
{
    constexpr int P = ADJACENT ? N / 2 : N, V = ADJACENT ? 1 : 2, BATCH = kBatch<N * sizeof(T)>;
    const int place = threadIdx.x / p.items, item = threadIdx.x - place * p.items;
    const int together = blockDim.x / p.items;               // tokens of a block
    const bool second = blockIdx.y >= p.q_parts;
    const RopeTensor& t = p.t[second];
    const int h0 = (second ? blockIdx.y - p.q_parts : blockIdx.y) * p.per;
    const int heads = min(p.per, (second ? p.kv_heads : p.heads) - h0);
    uint64_t turn[P];
    int axis[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        turn[i] = p.pair[item * P + i].turn;
        axis[i] = p.pair[item * P + i].axis;
    }
    const int u0 = p.pair[item * P].u, v0 = p.pair[item * P].v;
    const T* const in0 = static_cast<const T*>(t.in) + blockIdx.z * t.is.batch_stride + h0 * t.is.head_stride + u0;
    T* const out0 = static_cast<T*>(t.out) + blockIdx.z * t.os.batch_stride + h0 * t.os.head_stride + u0;
    const int32_t* const pos0 = p.positions + (p.shared ? 0 : blockIdx.z * p.tokens * p.axes);
    wait_for_launch_before();
    launch_dependents();                                     // 4680 x 12 heads 13.4 us without and 11.9 with this, one token 2.4 and 1.7
    for (int64_t n = static_cast<int64_t>(blockIdx.x) * together + place; n < p.tokens; n += static_cast<int64_t>(gridDim.x) * together) {
        int32_t pos[P];
#pragma unroll
        for (int i = 0; i < P; ++i) pos[i] = pos0[n * p.axes + max(axis[i], 0)];
        float2 cs[P];
        const T* in = in0 + n * t.is.token_stride;
        T* out = out0 + n * t.os.token_stride;
        for (int h = 0; h < heads; h += BATCH) {
            Pack<T, N> x[BATCH][V];
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const T* from = in + min(b, heads - 1 - h) * t.is.head_stride;
                x[b][0] = *reinterpret_cast<const Pack<T, N>*>(from);
                if constexpr (!ADJACENT) x[b][1] = *reinterpret_cast<const Pack<T, N>*>(from + (v0 - u0));
            }
            if (h == 0) {                                    // while the first heads are on their way
#pragma unroll
                for (int i = 0; i < P; ++i) cs[i] = cos_sin(static_cast<uint64_t>(static_cast<int64_t>(pos[i])) * turn[i]);
            }
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                if (h + b >= heads) break;
                float y[V][N];
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const float u = widen(ADJACENT ? x[b][0].e[2 * i] : x[b][0].e[i]);
                    const float v = widen(ADJACENT ? x[b][0].e[2 * i + 1] : x[b][V - 1].e[i]);
                    float a = fmaf(u, cs[i].x, -(v * cs[i].y)), c = fmaf(u, cs[i].y, v * cs[i].x);
                    if constexpr (!ALL)
                        if (axis[i] < 0) a = u, c = v;
                    y[0][ADJACENT ? 2 * i : i] = a;
                    y[V - 1][ADJACENT ? 2 * i + 1 : i] = c;
                }
                T* to = out + b * t.os.head_stride;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    Pack<T, N> w;
                    narrow(w, y[i]);
                    *reinterpret_cast<Pack<T, N>*>(to + (i ? v0 - u0 : 0)) = w;
                }
            }
            in += BATCH * t.is.head_stride;
            out += BATCH * t.os.head_stride;
        }
    }
}

template <typename T, int N, bool ADJACENT>
cudaError_t launch(AxesRopeParams& p, bool all, int head_dim, cudaStream_t s)
{
    constexpr int BATCH = kBatch<N * sizeof(T)>;
    p.items = head_dim / (ADJACENT ? N : 2 * N);
    const int together = std::max(1, kThreads / p.items);
    const int64_t places = (p.tokens + together - 1) / together;
    // Heads of a thread: all of a tensor's, unless that leaves SMs without work; a part of them costs its sines and cosines again.
    constexpr int64_t kFull = 152 * 12;
    const int heads = std::max(p.heads, p.kv_heads), tensors = p.kv_heads ? 2 : 1;
    const int64_t parts = std::max<int64_t>(1, std::min<int64_t>((heads + BATCH - 1) / BATCH, kFull / std::max<int64_t>(1, places * p.batch * tensors)));
    p.per = static_cast<int>((heads + parts - 1) / parts + BATCH - 1) / BATCH * BATCH;
    p.q_parts = (p.heads + p.per - 1) / p.per;
    const int all_parts = p.q_parts + (p.kv_heads + p.per - 1) / p.per;
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(places, INT32_MAX)), static_cast<unsigned>(all_parts), static_cast<unsigned>(p.batch));
    return launch_chained(all ? axes_rope_kernel<T, N, ADJACENT, true> : axes_rope_kernel<T, N, ADJACENT, false>, grid, together * p.items, 0, s, p);
}

}  // namespace

cudaError_t launch_axes_rope(AxesRopeParams& p, bool adjacent, int width, bool all, bool f32, int head_dim, cudaStream_t s)
{
    if (adjacent) return f32 ? launch<float, 4, true>(p, all, head_dim, s) : launch<__nv_bfloat16, 8, true>(p, all, head_dim, s);
    if (f32) return width == 4 ? launch<float, 4, false>(p, all, head_dim, s) : width == 2 ? launch<float, 2, false>(p, all, head_dim, s)
                                                                                         : launch<float, 1, false>(p, all, head_dim, s);
    return width == 8 ? launch<__nv_bfloat16, 8, false>(p, all, head_dim, s)
         : width == 2 ? launch<__nv_bfloat16, 2, false>(p, all, head_dim, s) : launch<__nv_bfloat16, 1, false>(p, all, head_dim, s);
}

}  // namespace sdv2
