// Rotary positions of several axes, forward and backward (the rotation by the negative angle).
//
// Every element is read and written once, so that memory bounds this.  A thread owns the same pairs of dims in many heads of a
// token: it finds their sines and cosines once and then only loads, turns and stores.
// An angle in turns is position * scale * base^(-2j/d) / 2pi.  Its frequency is held as a 64-bit fraction of a turn (whole
// turns of it change nothing), so that the 64-bit product with the position, which wraps around, is the fraction of a turn that
// is left: off by 2^-64 of a turn per position.  The nearest quarter turn is taken off before the rest, at most an eighth, goes
// to fp32, where it is off by 2^-28 of a turn at most.
#include <cuda_bf16.h>

#include <algorithm>

#include "chained.cuh"
#include "project.h"

namespace sdv2 {
namespace {

constexpr int kThreads = 128;
constexpr int kBatch = 4;                  // heads whose loads are under way together

__device__ __forceinline__ float2 cos_sin(uint64_t turn)
{
    const uint32_t t = static_cast<uint32_t>(turn >> 32);
    const uint32_t quarter = (t + 0x20000000u) >> 30;
    const float rest = static_cast<float>(static_cast<int32_t>(t - (quarter << 30))) * 0x1p-31f;   // half turns, at most a quarter
    float s, c;
    sincospif(rest, &s, &c);
    float2 r;
    r.x = quarter & 1 ? s : c;
    r.y = quarter & 1 ? c : s;
    if (quarter == 1 || quarter == 2) r.x = -r.x;
    if (quarter & 2) r.y = -r.y;
    return r;
}

template <typename T>
__device__ __forceinline__ float widen(T x) { return static_cast<float>(x); }
template <>
__device__ __forceinline__ float widen<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T narrow(float x) { return static_cast<T>(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// 16 bytes as elements.
template <typename T>
struct Vec {
    static constexpr int n = 16 / sizeof(T);
    union {
        uint4 bits;
        T e[16 / sizeof(T)];
    };
    __device__ __forceinline__ Vec() {}
};

template <typename T>
__device__ __forceinline__ void turn_pair(T& u, T& v, float2 cs, bool turns)
{
    if (!turns) return;
    const float a = widen<T>(u), b = widen<T>(v);
    u = narrow<T>(fmaf(a, cs.x, -(b * cs.y)));
    v = narrow<T>(fmaf(a, cs.y, b * cs.x));
}

template <typename T, RopeLayout L>
__global__ void __launch_bounds__(kThreads) axes_rope_kernel(const __grid_constant__ AxesRopeParams p)
{
    constexpr int VE = Vec<T>::n;
    constexpr int P = L == RopeLayout::adjacent ? VE / 2 : L == RopeLayout::halves ? VE : 1;   // pairs of a thread
    wait_for_launch_before();
    const int64_t g = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t place = g / p.items;                       // b * tokens + n
    if (place >= p.batch * p.tokens) return;
    const int item = static_cast<int>(g - place * p.items);
    const int64_t b = place / p.tokens, n = place - b * p.tokens;
    const int32_t* pos = p.positions + (p.shared ? n : place) * p.axes;
    float2 cs[P];
    bool turns[P];
    const int u0 = p.pair[item * P].u, v0 = p.pair[item * P].v;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const RopePair& r = p.pair[item * P + i];
        turns[i] = r.axis >= 0;
        cs[i] = make_float2(1.0f, 0.0f);
        if (turns[i]) cs[i] = cos_sin(static_cast<uint64_t>(static_cast<int64_t>(pos[r.axis])) * r.turn);
    }
    const int all = p.heads + p.kv_heads;
    const int last = min(all, static_cast<int>(blockIdx.y + 1) * p.per);
    for (int h0 = blockIdx.y * p.per; h0 < last; h0 += kBatch) {
        const T* in[kBatch];
        T* out[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int h = min(h0 + i, last - 1);
            const RopeTensor& t = p.t[h >= p.heads];
            const int64_t hh = h >= p.heads ? h - p.heads : h;
            in[i] = static_cast<const T*>(t.in) + b * t.is.batch_stride + n * t.is.token_stride + hh * t.is.head_stride;
            out[i] = static_cast<T*>(t.out) + b * t.os.batch_stride + n * t.os.token_stride + hh * t.os.head_stride;
        }
        if constexpr (L == RopeLayout::single) {
            T u[kBatch], v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) u[i] = in[i][u0], v[i] = in[i][v0];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (h0 + i < last) {
                    turn_pair<T>(u[i], v[i], cs[0], turns[0]);
                    out[i][u0] = u[i];
                    out[i][v0] = v[i];
                }
        } else if constexpr (L == RopeLayout::adjacent) {
            Vec<T> x[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) x[i].bits = *reinterpret_cast<const uint4*>(in[i] + u0);
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (h0 + i < last) {
#pragma unroll
                    for (int j = 0; j < P; ++j) turn_pair<T>(x[i].e[2 * j], x[i].e[2 * j + 1], cs[j], turns[j]);
                    *reinterpret_cast<uint4*>(out[i] + u0) = x[i].bits;
                }
        } else {
            Vec<T> u[kBatch], v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                u[i].bits = *reinterpret_cast<const uint4*>(in[i] + u0);
                v[i].bits = *reinterpret_cast<const uint4*>(in[i] + v0);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (h0 + i < last) {
#pragma unroll
                    for (int j = 0; j < P; ++j) turn_pair<T>(u[i].e[j], v[i].e[j], cs[j], turns[j]);
                    *reinterpret_cast<uint4*>(out[i] + u0) = u[i].bits;
                    *reinterpret_cast<uint4*>(out[i] + v0) = v[i].bits;
                }
        }
    }
}

template <typename T>
cudaError_t launch(const AxesRopeParams& p, RopeLayout layout, dim3 grid, cudaStream_t s)
{
    auto kernel = layout == RopeLayout::adjacent ? axes_rope_kernel<T, RopeLayout::adjacent>
                : layout == RopeLayout::halves   ? axes_rope_kernel<T, RopeLayout::halves>
                                                 : axes_rope_kernel<T, RopeLayout::single>;
    return launch_chained(kernel, grid, kThreads, 0, s, p);
}

}  // namespace

cudaError_t launch_axes_rope(AxesRopeParams& p, RopeLayout layout, bool f32, int head_dim, cudaStream_t s)
{
    const int lane = f32 ? 4 : 8;
    p.items = layout == RopeLayout::adjacent ? head_dim / lane : layout == RopeLayout::halves ? head_dim / lane / 2 : head_dim / 2;
    const int64_t threads = p.batch * p.tokens * p.items;
    const int64_t blocks = (threads + kThreads - 1) / kThreads;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    // Heads of a thread: all, unless that leaves SMs without work; a part of them costs its sines and cosines again.
    const int all = p.heads + p.kv_heads;
    constexpr int64_t kFull = 152 * 8;
    const int64_t parts = std::min<int64_t>({(all + kBatch - 1) / kBatch, std::max<int64_t>(1, kFull / blocks), 65535});
    p.per = static_cast<int>((all + parts - 1) / parts + kBatch - 1) / kBatch * kBatch;
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((all + p.per - 1) / p.per));
    return f32 ? launch<float>(p, layout, grid, s) : launch<__nv_bfloat16>(p, layout, grid, s);
}

}  // namespace sdv2
