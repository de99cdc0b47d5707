// Cross attention on the CUDA cores, forward and backward: one half-warp per key or row, any size.
//
// Forward (a few queries, where the keys and values have to be read and there is next to nothing to
// multiply them with): out = sum_j softmax_j(scale q.k_j) v_j in one pass over the keys.  The heads
// that share a key head and their queries form rows r = i*g + (h mod g); a cluster of CTAs holds
// up to kRows rows and splits the key range.  In a CTA each half-warp walks its own keys, a lane
// holding 8 of the 128 dims (one 16-byte load of k and of v), with its own running maximum and sum
// per row; half-warps are joined through shared memory, CTAs through the cluster's shared memory, in
// a fixed order.
//
// Backward: delta = rowsum(dO * O); dQ with a half-warp per query row over the keys; dK and dV with
// a half-warp per key over the queries of every head that shares it.  No atomics: each output row
// has one owner.
#include <cuda_bf16.h>

#include <algorithm>

#include "block.h"
#include "ptx.cuh"
#include "ptx_pair.cuh"

namespace sdv2 {
namespace {

constexpr int HD = 128;
constexpr int kRows = 4;               // query rows per cluster
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

__device__ __forceinline__ uint4 pack8(const float* v)
{
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
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

// grid.x = units * splits, clusters of `splits` CTAs; unit = ((b * Hk) + key head) * row blocks + block.
__global__ void __launch_bounds__(kWarps * 32) cross_rows_kernel(const __grid_constant__ CrossForward p, int splits,
                                                                 int row_blocks)
{
    __shared__ float s_m[kHalves][kRows], s_l[kHalves][kRows];
    __shared__ float s_acc[kWarps][kRows][HD];
    __shared__ float c_m[kRows], c_l[kRows], c_acc[kRows][HD];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int half = warp * 2 + (lane >> 4), sub = lane & 15;
    const int64_t unit = blockIdx.x / splits;
    const int split = static_cast<int>(blockIdx.x - unit * splits);
    const int rb = static_cast<int>(unit % row_blocks);
    const int64_t bh = unit / row_blocks;
    const int hk = static_cast<int>(bh % p.c.Hk);
    const int b = static_cast<int>(bh / p.c.Hk);
    const int g = p.c.H / p.c.Hk;
    const int64_t rows = static_cast<int64_t>(g) * p.c.Nq;
    const int64_t row0 = static_cast<int64_t>(rb) * kRows;
    const int n = p.c.n[b];
    const int j0 = static_cast<int>(static_cast<int64_t>(n) * split / splits);
    const int j1 = static_cast<int>(static_cast<int64_t>(n) * (split + 1) / splits);
    const float sl2 = p.c.scale * kLog2e;

    Vec8 q[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int64_t row = row0 + r < rows ? row0 + r : rows - 1;       // rows past the end repeat the last
        const int64_t i = row / g;
        const int h = hk * g + static_cast<int>(row - i * g);
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
    // the CTAs of the cluster share the rows' dims
    for (int i = split * kWarps * 32 + threadIdx.x; i < kRows * HD; i += splits * kWarps * 32) {
        const int r = i / HD, d = i - r * HD;
        if (row0 + r >= rows) continue;
        float mx = -INFINITY;
        for (int c = 0; c < splits; ++c) mx = fmaxf(mx, ld_cluster_f32(map_to_rank(smem_u32(&c_m[r]), c)));
        float sum = 0.f, a = 0.f;
        for (int c = 0; c < splits; ++c) {
            const float lc = ld_cluster_f32(map_to_rank(smem_u32(&c_l[r]), c));
            if (lc == 0.f) continue;
            const float f = ex2_from(ld_cluster_f32(map_to_rank(smem_u32(&c_m[r]), c)), mx);
            sum += lc * f;
            a += ld_cluster_f32(map_to_rank(smem_u32(&c_acc[r][d]), c)) * f;
        }
        const int64_t row = row0 + r, qi = row / g;
        const int h = hk * g + static_cast<int>(row - qi * g);
        const float o = n == 0 ? 0.f : a / sum;
        reinterpret_cast<__nv_bfloat16*>(p.out)[((static_cast<int64_t>(b) * p.c.Nq + qi) * p.c.H + h) * HD + d] =
            __float2bfloat16_rn(o);
        if (d == 0 && p.lse)
            p.lse[(static_cast<int64_t>(b) * p.c.H + h) * p.c.Nq + qi] = n == 0 ? -INFINITY : (mx + log2f(sum)) * kLn2;
    }
    cluster_sync_all();                                  // no CTA leaves while others read its memory
}

// ---- backward ---------------------------------------------------------------------------------

// delta[b][h][i] = sum_d dout * out; a half-warp per row.
__global__ void __launch_bounds__(256) cross_delta_kernel(const __grid_constant__ CrossBackward p)
{
    const int sub = threadIdx.x & 15;
    const int64_t row = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 4;   // (b, i, h)
    const int64_t rows = static_cast<int64_t>(p.c.B) * p.c.Nq * p.c.H;
    const int64_t safe = row < rows ? row : rows - 1;
    const Vec8 a = unpack8(load_vec(p.out + safe * HD + sub * 8));
    const Vec8 d = unpack8(load_vec(p.dout + safe * HD + sub * 8));
    const float s = half_sum(dot8(a, d));
    if (row < rows && sub == 0) {
        const int64_t bi = row / p.c.H;
        const int h = static_cast<int>(row - bi * p.c.H);
        const int64_t b = bi / p.c.Nq;
        p.stats[(b * p.c.H + h) * p.c.Nq + (bi - b * p.c.Nq)] = s;
    }
}

// dQ: half-warp per (b, h, i); a block's 16 rows are consecutive queries of one head.
__global__ void __launch_bounds__(256) cross_rows_dq_kernel(const __grid_constant__ CrossBackward p, int blocks_per_head)
{
    const int half = threadIdx.x >> 4, sub = threadIdx.x & 15;
    const int64_t bh = blockIdx.x / blocks_per_head;
    const int64_t i = static_cast<int64_t>(blockIdx.x - bh * blocks_per_head) * 16 + half;
    const int h = static_cast<int>(bh % p.c.H), b = static_cast<int>(bh / p.c.H);
    const int hk = h / (p.c.H / p.c.Hk);
    const int64_t safe = i < p.c.Nq ? i : p.c.Nq - 1;
    const int n = p.c.n[b];
    const float sl2 = p.c.scale * kLog2e;
    const int64_t o = ((static_cast<int64_t>(b) * p.c.Nq + safe) * p.c.H + h) * HD + sub * 8;
    const Vec8 q = unpack8(load_vec(p.c.q + b * p.c.qs.batch + safe * p.c.qs.tok + h * p.c.qs.hd + sub * 8));
    const Vec8 dout = unpack8(load_vec(p.dout + o));
    const float lse2 = p.lse[bh * p.c.Nq + safe] * kLog2e, delta = p.stats[bh * p.c.Nq + safe];
    const uint16_t* kb = p.c.k + b * p.c.kvs.batch + hk * p.c.kvs.hd + sub * 8;
    const uint16_t* vb = p.c.v + b * p.c.kvs.batch + hk * p.c.kvs.hd + sub * 8;
    float acc[8] = {};
    for (int j = 0; n > 1 && j < n; ++j) {
        const Vec8 k = unpack8(load_vec(kb + j * p.c.kvs.tok));
        const Vec8 v = unpack8(load_vec(vb + j * p.c.kvs.tok));
        const float s = half_sum(dot8(q, k)), dp = half_sum(dot8(dout, v));
        const float ds = exp2f(fmaf(s, sl2, -lse2)) * (dp - delta);
#pragma unroll
        for (int d = 0; d < 8; ++d) acc[d] = fmaf(ds, k.x[d], acc[d]);
    }
    if (i < p.c.Nq) {
#pragma unroll
        for (int d = 0; d < 8; ++d) acc[d] *= p.c.scale;
        *reinterpret_cast<uint4*>(p.dq + o) = pack8(acc);
    }
}

// dK, dV: half-warp per (b, key head, j).
__global__ void __launch_bounds__(256) cross_rows_dkv_kernel(const __grid_constant__ CrossBackward p, int blocks_per_head)
{
    const int half = threadIdx.x >> 4, sub = threadIdx.x & 15;
    const int64_t bh = blockIdx.x / blocks_per_head;
    const int64_t j = static_cast<int64_t>(blockIdx.x - bh * blocks_per_head) * 16 + half;
    const int hk = static_cast<int>(bh % p.c.Hk), b = static_cast<int>(bh / p.c.Hk);
    const int g = p.c.H / p.c.Hk, n = p.c.n[b];
    const float sl2 = p.c.scale * kLog2e;
    const int64_t first = j - half;                       // the block's first key
    float dk[8] = {}, dv[8] = {};
    if (first < n) {
        const int64_t safe = j < n ? j : n - 1;
        const Vec8 k = unpack8(load_vec(p.c.k + b * p.c.kvs.batch + safe * p.c.kvs.tok + hk * p.c.kvs.hd + sub * 8));
        const Vec8 v = unpack8(load_vec(p.c.v + b * p.c.kvs.batch + safe * p.c.kvs.tok + hk * p.c.kvs.hd + sub * 8));
        for (int h = hk * g; h < (hk + 1) * g; ++h) {
            const int64_t stat = (static_cast<int64_t>(b) * p.c.H + h) * p.c.Nq;
            for (int64_t i = 0; i < p.c.Nq; ++i) {
                const Vec8 q = unpack8(load_vec(p.c.q + b * p.c.qs.batch + i * p.c.qs.tok + h * p.c.qs.hd + sub * 8));
                const Vec8 dout =
                    unpack8(load_vec(p.dout + ((static_cast<int64_t>(b) * p.c.Nq + i) * p.c.H + h) * HD + sub * 8));
                const float s = half_sum(dot8(q, k)), dp = half_sum(dot8(dout, v));
                const float pr = exp2f(fmaf(s, sl2, -p.lse[stat + i] * kLog2e));
                const float ds = n > 1 ? pr * (dp - p.stats[stat + i]) : 0.f;
#pragma unroll
                for (int d = 0; d < 8; ++d) {
                    dk[d] = fmaf(ds, q.x[d], dk[d]);
                    dv[d] = fmaf(pr, dout.x[d], dv[d]);
                }
            }
        }
    }
    if (j < p.c.Nk) {
        const int64_t o = ((static_cast<int64_t>(b) * p.c.Nk + j) * p.c.Hk + hk) * HD + sub * 8;
        const bool live = j < n;
#pragma unroll
        for (int d = 0; d < 8; ++d) {
            dk[d] = live ? dk[d] * p.c.scale : 0.f;
            dv[d] = live ? dv[d] : 0.f;
        }
        *reinterpret_cast<uint4*>(p.dk + o) = pack8(dk);
        *reinterpret_cast<uint4*>(p.dv + o) = pack8(dv);
    }
}

}  // namespace

cudaError_t launch_cross_rows(const CrossForward& p, cudaStream_t s)
{
    const int64_t rows = static_cast<int64_t>(p.c.H / p.c.Hk) * p.c.Nq;
    const int64_t row_blocks = (rows + kRows - 1) / kRows;
    const int64_t units = row_blocks * p.c.B * p.c.Hk;
    int longest = 0;
    for (int b = 0; b < p.c.B; ++b) longest = std::max(longest, p.c.n[b]);
    // a key split holds at least one round of loads of its half-warps; split until the SMs are full
    int splits = 1;
    while (splits < 8 && units * splits < 304 && longest > splits * kHalves * kKeysAtOnce) splits *= 2;
    if (units * splits > INT32_MAX) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(units * splits));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(splits);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, cross_rows_kernel, p, splits, static_cast<int>(row_blocks));
}

cudaError_t launch_cross_rows_backward(const CrossBackward& p, cudaStream_t s)
{
    const int64_t rows = static_cast<int64_t>(p.c.B) * p.c.Nq * p.c.H;
    const int64_t qb = (static_cast<int64_t>(p.c.Nq) + 15) / 16, kb = (static_cast<int64_t>(p.c.Nk) + 15) / 16;
    const int64_t dq_blocks = qb * p.c.B * p.c.H, dkv_blocks = kb * p.c.B * p.c.Hk;
    if ((rows + 15) / 16 > INT32_MAX || dq_blocks > INT32_MAX || dkv_blocks > INT32_MAX)
        return cudaErrorInvalidConfiguration;
    cross_delta_kernel<<<static_cast<unsigned>((rows + 15) / 16), 256, 0, s>>>(p);
    cross_rows_dq_kernel<<<static_cast<unsigned>(dq_blocks), 256, 0, s>>>(p, static_cast<int>(qb));
    if (dkv_blocks > 0) cross_rows_dkv_kernel<<<static_cast<unsigned>(dkv_blocks), 256, 0, s>>>(p, static_cast<int>(kb));
    return cudaGetLastError();
}

}  // namespace sdv2
