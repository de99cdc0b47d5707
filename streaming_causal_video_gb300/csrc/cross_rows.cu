// Cross attention of one or two query rows on the CUDA cores: a half-warp per key.
//
// The keys and values have to be read and there is next to nothing to multiply them with, so what counts
// is the time until the first product, and a tile of 128 rows is mostly empty (12 heads, 512 states: one
// row 4.7 us, two 5.9 us, against 8.9 us on the tensor cores; at 20000 states the tensor cores' deeper
// loads win by far, 46 against 139 us).
//
// out = sum_j softmax_j(scale q.k_j) v_j in one pass over the keys.  The heads that share a key head and their
// queries form rows r = i*g + (h mod g); a cluster of CTAs holds the rows of one key head and splits its key
// range.  In a CTA each half-warp walks its own keys, a lane holding 8 of the 128 dims (one 16-byte load of k and
// of v), with its own running maximum and sum per row; half-warps are joined through shared memory, CTAs through
// the cluster's shared memory, in a fixed order.
#include <cuda_bf16.h>

#include <algorithm>

#include "block.h"
#include "chained.cuh"
#include "ptx.cuh"
#include "ptx_pair.cuh"

namespace sdv2 {
namespace {

constexpr int HD = 128;
constexpr int kMaxSplits = 8;
constexpr int kWarps = 8;
constexpr int kHalves = 2 * kWarps;    // half-warps per CTA
constexpr int kKeysAtOnce = 4;         // keys a half-warp loads before it computes
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Vec8 {
    float x[8];
};

__device__ __forceinline__ Vec8 unpack8(uint4 w)
{
    Vec8 r;
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r.x[2 * i] = __uint_as_float(u[i] << 16);
        r.x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
    return r;
}

__device__ __forceinline__ uint4 load_vec(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }

// Sum over the 16 lanes of a half-warp.
__device__ __forceinline__ float half_sum(float v)
{
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float dot8(const Vec8& a, const Vec8& b)
{
    float s = a.x[0] * b.x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) s = fmaf(a.x[i], b.x[i], s);
    return s;
}

// 2^(x - m) where nothing has been seen while m = -infinity (x is then -infinity too, unless NaN).
__device__ __forceinline__ float ex2_from(float x, float m) { return exp2f(x - (m == -INFINITY ? 0.f : m)); }

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// grid.x = units * splits, clusters of `splits` CTAs; unit = b * Hk + key head, whose rows are kRows.
template <int kRows>
__global__ void __launch_bounds__(kWarps * 32) cross_rows_kernel(const __grid_constant__ CrossForward p, int splits)
{
    __shared__ float s_m[kHalves][kRows], s_l[kHalves][kRows];
    __shared__ float s_acc[kWarps][kRows][HD];
    __shared__ float c_m[kRows], c_l[kRows], c_acc[kRows][HD];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int half = warp * 2 + (lane >> 4), sub = lane & 15;
    // 32-bit divisions: a 64-bit one costs as much as a key
    const uint32_t unit = blockIdx.x / static_cast<uint32_t>(splits);
    const int split = static_cast<int>(blockIdx.x - unit * splits);
    const int b = static_cast<int>(unit / static_cast<uint32_t>(p.c.Hk));
    const int hk = static_cast<int>(unit - b * p.c.Hk);
    const int g = p.c.H / p.c.Hk;
    const int n = p.c.n[b];
    const int j0 = static_cast<int>(static_cast<int64_t>(n) * split / splits);
    const int j1 = static_cast<int>(static_cast<int64_t>(n) * (split + 1) / splits);
    const float sl2 = p.c.scale * kLog2e;

    wait_for_launch_before();
    Vec8 q[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int i = r / g;
        const int h = hk * g + (r - i * g);
        q[r] = unpack8(load_vec(p.c.q + b * p.c.qs.batch + i * p.c.qs.tok + h * p.c.qs.hd + sub * 8));
    }
    const uint16_t* kb = p.c.k + b * p.c.kvs.batch + hk * p.c.kvs.hd + sub * 8;
    const uint16_t* vb = p.c.v + b * p.c.kvs.batch + hk * p.c.kvs.hd + sub * 8;

    float m[kRows], l[kRows];
    Vec8 acc[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int d = 0; d < 8; ++d) acc[r].x[d] = 0.f;
    }
    // warp-uniform trip count: the reductions are warp-collective
    for (int base = j0; base < j1; base += kHalves * kKeysAtOnce) {
        uint4 kw[kKeysAtOnce], vw[kKeysAtOnce];
#pragma unroll
        for (int u = 0; u < kKeysAtOnce; ++u) {
            const int j = base + u * kHalves + half;
            if (j < j1) {
                kw[u] = load_vec(kb + j * p.c.kvs.tok);
                vw[u] = load_vec(vb + j * p.c.kvs.tok);
            } else {
                kw[u] = make_uint4(0, 0, 0, 0);
                vw[u] = make_uint4(0, 0, 0, 0);
            }
        }
        float s[kRows][kKeysAtOnce];
#pragma unroll
        for (int u = 0; u < kKeysAtOnce; ++u) {
            const Vec8 kv = unpack8(kw[u]);
            const bool in = base + u * kHalves + half < j1;
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const float d = half_sum(dot8(q[r], kv));
                s[r][u] = in ? d * sl2 : -INFINITY;
            }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            float mx = m[r];
#pragma unroll
            for (int u = 0; u < kKeysAtOnce; ++u) mx = fmaxf(mx, s[r][u]);
            const float f = ex2_from(m[r], mx);
            m[r] = mx;
            l[r] *= f;
#pragma unroll
            for (int d = 0; d < 8; ++d) acc[r].x[d] *= f;
#pragma unroll
            for (int u = 0; u < kKeysAtOnce; ++u) {
                s[r][u] = ex2_from(s[r][u], mx);
                l[r] += s[r][u];
            }
        }
#pragma unroll
        for (int u = 0; u < kKeysAtOnce; ++u) {
            const Vec8 vv = unpack8(vw[u]);
#pragma unroll
            for (int r = 0; r < kRows; ++r)
#pragma unroll
                for (int d = 0; d < 8; ++d) acc[r].x[d] = fmaf(s[r][u], vv.x[d], acc[r].x[d]);
        }
    }
    // join the half-warps of a warp, then the warps, then the CTAs of the cluster
    if (sub == 0)
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            s_m[half][r] = m[r];
            s_l[half][r] = l[r];
        }
    __syncthreads();
    float big[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        float mx = s_m[0][r];
        for (int i = 1; i < kHalves; ++i) mx = fmaxf(mx, s_m[i][r]);
        big[r] = mx;
        const float f = ex2_from(m[r], mx);
#pragma unroll
        for (int d = 0; d < 8; ++d) {
            float a = l[r] == 0.f ? 0.f : acc[r].x[d] * f;
            a += __shfl_xor_sync(0xffffffffu, a, 16);
            if (lane < 16) s_acc[warp][r][sub * 8 + d] = a;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * HD; i += kWarps * 32) {
        const int r = i / HD, d = i - r * HD;
        float a = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) a += s_acc[w][r][d];
        c_acc[r][d] = a;
    }
    if (threadIdx.x == 0)
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            float sum = 0.f;
            for (int i = 0; i < kHalves; ++i)
                if (s_l[i][r] != 0.f) sum += s_l[i][r] * ex2_from(s_m[i][r], big[r]);
            c_m[r] = big[r];
            c_l[r] = sum;
        }
    cluster_sync_all();
    // the CTAs of the cluster share the rows' dims; a thread's loads from all of them are under way together
    for (int i = split * kWarps * 32 + threadIdx.x; i < kRows * HD; i += splits * kWarps * 32) {
        const int r = i / HD, d = i - r * HD;
        float mc[kMaxSplits], lc[kMaxSplits], ac[kMaxSplits];
#pragma unroll
        for (int c = 0; c < kMaxSplits; ++c)
            if (c < splits) {
                mc[c] = ld_cluster_f32(map_to_rank(smem_u32(&c_m[r]), c));
                lc[c] = ld_cluster_f32(map_to_rank(smem_u32(&c_l[r]), c));
                ac[c] = ld_cluster_f32(map_to_rank(smem_u32(&c_acc[r][d]), c));
            }
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < kMaxSplits; ++c)
            if (c < splits) mx = fmaxf(mx, mc[c]);
        float sum = 0.f, a = 0.f;
#pragma unroll
        for (int c = 0; c < kMaxSplits; ++c)
            if (c < splits && lc[c] != 0.f) {
                const float f = ex2_from(mc[c], mx);
                sum += lc[c] * f;
                a += ac[c] * f;
            }
        const int qi = r / g;
        const int h = hk * g + (r - qi * g);
        const float o = n == 0 ? 0.f : a / sum;
        reinterpret_cast<__nv_bfloat16*>(p.out)[((static_cast<int64_t>(b) * p.c.Nq + qi) * p.c.H + h) * HD + d] =
            __float2bfloat16_rn(o);
        if (d == 0 && p.lse)
            p.lse[(static_cast<int64_t>(b) * p.c.H + h) * p.c.Nq + qi] = n == 0 ? -INFINITY : (mx + log2f(sum)) * kLn2;
    }
    cluster_sync_all();                                  // no CTA leaves while others read its memory
}

}  // namespace

template <int kRows>
static cudaError_t launch_rows(const CrossForward& p, cudaStream_t s)
{
    const int64_t units = static_cast<int64_t>(p.c.B) * p.c.Hk;
    int longest = 0;
    for (int b = 0; b < p.c.B; ++b) longest = std::max(longest, p.c.n[b]);
    // a key split holds at least one round of loads of its half-warps; split until the SMs are full
    int splits = 1;
    while (splits < kMaxSplits && units * splits < 304 && longest > splits * kHalves * kKeysAtOnce) splits *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(units * splits));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attrs[2] = {chained_attribute(), {}};
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = static_cast<unsigned>(splits);
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, cross_rows_kernel<kRows>, p, splits);
}

cudaError_t launch_cross_rows(const CrossForward& p, cudaStream_t s)
{
    static_assert(kFewRows == 2, "a kernel for each number of rows");
    return static_cast<int64_t>(p.c.H / p.c.Hk) * p.c.Nq == 1 ? launch_rows<1>(p, s) : launch_rows<2>(p, s);
}

}  // namespace sdv2
