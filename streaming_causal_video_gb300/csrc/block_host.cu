// Host side of the operators in sdv2_block.h: argument checks, strides and dispatch.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "block.h"
#include "internal.h"

namespace sdv2 {
namespace {

sdv2_status bad(sdv2_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
sdv2_status bad(sdv2_status s, const char* fmt, ...)
{
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    set_last_error(buf);
    return s;
}

sdv2_status done(cudaError_t e, const char* what)
{
    if (e != cudaSuccess) return bad(SDV2_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    set_last_error("");
    return SDV2_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool usable(const void* p) { return p && aligned16(p); }

constexpr int64_t kMaxStride = int64_t(1) << 38;       // tensor maps take byte strides below 2^40
constexpr size_t kHeaderBytes = 256;                    // error word, as sdv2_check_device_error reads it

// Strides of q or of k and v with the defaults filled in.
CrossStrides strides_of(int64_t tok, int64_t hd, int64_t batch, int64_t heads, int64_t len)
{
    CrossStrides s;
    s.hd = hd ? hd : 128;
    s.tok = tok ? tok : heads * 128;
    s.batch = batch ? batch : std::max(std::max<int64_t>(len, 1) * s.tok, heads * s.hd);
    return s;
}

int kv_heads_of(const sdv2_cross_cfg* c) { return c->kv_heads ? c->kv_heads : c->heads; }

sdv2_status check_strides(const char* name, const CrossStrides& s)
{
    if (s.tok < 128 || s.hd < 128 || s.batch < 8 || ((s.tok | s.hd | s.batch) & 7))
        return bad(SDV2_ERR_INVALID_ARG, "%s token (%lld) and head (%lld) strides must be >= 128, the batch stride (%lld) "
                   ">= 8, all multiples of 8", name, (long long)s.tok, (long long)s.hd, (long long)s.batch);
    if (s.tok > kMaxStride || s.hd > kMaxStride || s.batch > kMaxStride)
        return bad(SDV2_ERR_UNSUPPORTED, "%s strides must be at most 2^38", name);
    return SDV2_OK;
}

sdv2_status check_cross(const sdv2_cross_cfg* c, CrossStrides* qs, CrossStrides* kvs)
{
    if (!c) return bad(SDV2_ERR_INVALID_ARG, "cfg is NULL");
    if (c->batch < 1 || c->heads < 1) return bad(SDV2_ERR_INVALID_ARG, "batch and heads must be >= 1");
    if (c->batch > 65535 || c->heads > 65535) return bad(SDV2_ERR_UNSUPPORTED, "batch and heads must be <= 65535");
    if (c->kv_heads < 0 || c->heads % kv_heads_of(c))
        return bad(SDV2_ERR_INVALID_ARG, "kv_heads (%d) must divide heads (%d)", c->kv_heads, c->heads);
    if (c->head_dim != 128) return bad(SDV2_ERR_UNSUPPORTED, "only head_dim 128 is built (got %d)", c->head_dim);
    if (c->q_len < 1 || c->q_len > (int64_t(1) << 30))
        return bad(SDV2_ERR_INVALID_ARG, "q_len (%lld) must be in [1, 2^30]", (long long)c->q_len);
    if (c->kv_len < 0 || c->kv_len > (int64_t(1) << 30))
        return bad(SDV2_ERR_INVALID_ARG, "kv_len (%lld) must be in [0, 2^30]", (long long)c->kv_len);
    if (std::min({c->q_token_stride, c->q_head_stride, c->q_batch_stride, c->kv_token_stride, c->kv_head_stride,
                  c->kv_batch_stride}) < 0)
        return bad(SDV2_ERR_INVALID_ARG, "strides must be >= 0");
    // checked before the defaults multiply them by lengths
    if (std::max({c->q_token_stride, c->q_head_stride, c->q_batch_stride, c->kv_token_stride, c->kv_head_stride,
                  c->kv_batch_stride}) > kMaxStride)
        return bad(SDV2_ERR_UNSUPPORTED, "strides must be at most 2^38");
    const __int128 dense = static_cast<__int128>(std::max<int64_t>(c->q_token_stride, int64_t(c->heads) * 128)) * c->q_len;
    const __int128 dense_kv =
        static_cast<__int128>(std::max<int64_t>(c->kv_token_stride, int64_t(c->heads) * 128)) * std::max<int64_t>(c->kv_len, 1);
    if (dense > (static_cast<__int128>(1) << 60) || dense_kv > (static_cast<__int128>(1) << 60))
        return bad(SDV2_ERR_UNSUPPORTED, "q or k and v are too large");
    *qs = strides_of(c->q_token_stride, c->q_head_stride, c->q_batch_stride, c->heads, c->q_len);
    *kvs = strides_of(c->kv_token_stride, c->kv_head_stride, c->kv_batch_stride, kv_heads_of(c), c->kv_len);
    sdv2_status s = check_strides("q", *qs);
    if (s == SDV2_OK) s = check_strides("kv", *kvs);
    return s;
}

// Lengths, scale and the pieces of the problem that all streams share.
sdv2_status check_call(const sdv2_cross_cfg* c, const int64_t* kv_lens, float* scale)
{
    if (!(*scale > 0.f)) *scale = 1.0f / std::sqrt(128.0f);
    if (!std::isfinite(*scale)) return bad(SDV2_ERR_INVALID_ARG, "scale must be finite");
    if (kv_lens)
        for (int b = 0; b < c->batch; ++b)
            if (kv_lens[b] < 0 || kv_lens[b] > c->kv_len)
                return bad(SDV2_ERR_INVALID_ARG, "kv_lens[%d] (%lld) must be in [0, kv_len]", b, (long long)kv_lens[b]);
    return SDV2_OK;
}

CrossProblem slice_of(const sdv2_cross_cfg* c, const int64_t* kv_lens, const CrossStrides& qs, const CrossStrides& kvs,
                      const void* q, const void* k, const void* v, float scale, void* ws, int b0, int nb)
{
    CrossProblem p{};
    p.q = static_cast<const uint16_t*>(q) + b0 * qs.batch;
    p.k = k ? static_cast<const uint16_t*>(k) + b0 * kvs.batch : nullptr;
    p.v = v ? static_cast<const uint16_t*>(v) + b0 * kvs.batch : nullptr;
    p.qs = qs;
    p.kvs = kvs;
    p.B = nb;
    p.H = c->heads;
    p.Hk = kv_heads_of(c);
    p.Nq = static_cast<int32_t>(c->q_len);
    p.Nk = static_cast<int32_t>(c->kv_len);
    p.scale = scale;
    p.err = static_cast<uint32_t*>(ws);
    p.timeout_ns = wait_timeout_ns();
    for (int b = 0; b < nb; ++b) p.n[b] = static_cast<int32_t>(kv_lens ? kv_lens[b0 + b] : c->kv_len);
    return p;
}

// Scratch of the backward pass for one launch's streams: statistics, then partial sums.
size_t stats_bytes(const sdv2_cross_cfg* c)
{
    return (cross_backward_stats_bytes(std::min(c->batch, kCrossStreams), c->heads, kv_heads_of(c), c->q_len) + 255) / 256 * 256;
}

int64_t rows_of(const sdv2_norm_cfg* c) { return c->rows_per_group ? c->rows_per_group : c->rows; }

sdv2_status check_norm(const sdv2_norm_cfg* c)
{
    if (!c) return bad(SDV2_ERR_INVALID_ARG, "cfg is NULL");
    if (c->rows < 1 || c->rows > INT32_MAX) return bad(SDV2_ERR_INVALID_ARG, "rows must be in [1, 2^31 - 1]");
    if (c->cols < 1) return bad(SDV2_ERR_INVALID_ARG, "cols must be >= 1");
    if (c->cols > 16384) return bad(SDV2_ERR_UNSUPPORTED, "cols (%d) must be <= 16384", c->cols);
    if ((c->x_dtype != SDV2_BF16 && c->x_dtype != SDV2_F32) || (c->y_dtype != SDV2_BF16 && c->y_dtype != SDV2_F32))
        return bad(SDV2_ERR_INVALID_ARG, "x_dtype and y_dtype must be SDV2_BF16 or SDV2_F32");
    if (c->weight_plus_one != 0 && c->weight_plus_one != 1) return bad(SDV2_ERR_INVALID_ARG, "weight_plus_one must be 0 or 1");
    if ((c->x_row_stride && c->x_row_stride < c->cols) || (c->y_row_stride && c->y_row_stride < c->cols) ||
        (c->group_stride && c->group_stride < c->cols))
        return bad(SDV2_ERR_INVALID_ARG, "row and group strides must be 0 or >= cols");
    if (c->x_row_stride > kMaxStride || c->y_row_stride > kMaxStride || c->group_stride > kMaxStride)
        return bad(SDV2_ERR_UNSUPPORTED, "strides must be at most 2^38");
    if (c->rows_per_group < 0) return bad(SDV2_ERR_INVALID_ARG, "rows_per_group must be >= 0");
    if (!(c->eps >= 0.f) || !std::isfinite(c->eps)) return bad(SDV2_ERR_INVALID_ARG, "eps must be finite and >= 0");
    return SDV2_OK;
}

NormParams norm_params(const sdv2_norm_cfg* c, const void* x, const float* weight)
{
    NormParams p{};
    p.x = x;
    p.weight = weight;
    p.rows = c->rows;
    p.cols = c->cols;
    p.xs = c->x_row_stride ? c->x_row_stride : c->cols;
    p.ys = c->y_row_stride ? c->y_row_stride : c->cols;
    p.gs = c->group_stride ? c->group_stride : c->cols;
    p.rows_per_group = std::min(rows_of(c), c->rows);
    p.x_f32 = c->x_dtype == SDV2_F32;
    p.y_f32 = c->y_dtype == SDV2_F32;
    p.plus_one = c->weight_plus_one;
    p.eps = c->eps;
    p.aligned = ((p.cols | p.xs | p.ys | p.gs) & 7) == 0;
    return p;
}

}  // namespace
}  // namespace sdv2

using namespace sdv2;

extern "C" {

size_t sdv2_cross_workspace_bytes(const sdv2_cross_cfg* c, int32_t backward)
{
    CrossStrides qs, kvs;
    if (check_cross(c, &qs, &kvs) != SDV2_OK) return 0;
    size_t bytes = kHeaderBytes;
    if (backward) {
        // the streams left over behind whole launches are fewer units, so that they may be cut into more ranges
        auto parts = [&](int streams) {
            return streams ? cross_backward_part_bytes(streams, c->heads, kv_heads_of(c), c->q_len, c->kv_len) : 0;
        };
        bytes += stats_bytes(c) + std::max(parts(std::min(c->batch, kCrossStreams)), parts(c->batch % kCrossStreams));
    }
    return bytes;
}

sdv2_status sdv2_cross_workspace_init(const sdv2_cross_cfg* c, void* ws, void* stream)
{
    CrossStrides qs, kvs;
    sdv2_status s = check_cross(c, &qs, &kvs);
    if (s != SDV2_OK) return s;
    if (!usable(ws)) return bad(SDV2_ERR_INVALID_ARG, "ws must be a non-null 16-byte aligned pointer");
    if ((s = require_device()) != SDV2_OK) return s;
    return done(cudaMemsetAsync(ws, 0, kHeaderBytes, static_cast<cudaStream_t>(stream)), "cross workspace");
}

sdv2_status sdv2_cross_attention(const sdv2_cross_cfg* c, const int64_t* kv_lens, const void* q, const void* k,
                                 const void* v, float scale, void* out, float* lse, void* ws, void* stream)
{
    CrossStrides qs, kvs;
    sdv2_status s = check_cross(c, &qs, &kvs);
    if (s != SDV2_OK) return s;
    if (!usable(q) || !usable(out) || !usable(ws) || !aligned16(k) || !aligned16(v) || (c->kv_len && (!k || !v)))
        return bad(SDV2_ERR_INVALID_ARG, "device pointers must be non-null and 16-byte aligned");
    if (!aligned16(lse)) return bad(SDV2_ERR_INVALID_ARG, "lse must be 16-byte aligned");
    if ((s = check_call(c, kv_lens, &scale)) != SDV2_OK) return s;
    if ((s = require_device()) != SDV2_OK) return s;
    for (int b0 = 0; b0 < c->batch; b0 += kCrossStreams) {
        CrossForward p{};
        p.c = slice_of(c, kv_lens, qs, kvs, q, k, v, scale, ws, b0, std::min(kCrossStreams, c->batch - b0));
        const int64_t rows = static_cast<int64_t>(b0) * c->heads * c->q_len;
        p.out = static_cast<uint16_t*>(out) + rows * 128;
        p.lse = lse ? lse + rows : nullptr;
        const bool few = static_cast<int64_t>(p.c.H / p.c.Hk) * p.c.Nq <= kFewRows && *std::max_element(p.c.n, p.c.n + p.c.B) <= kFewKeys;
        const cudaError_t e = few ? launch_cross_rows(p, static_cast<cudaStream_t>(stream))
                                  : launch_cross_attention(p, static_cast<cudaStream_t>(stream));
        if (e != cudaSuccess) return done(e, "cross attention launch");
    }
    return done(cudaSuccess, "");
}

sdv2_status sdv2_cross_attention_backward(const sdv2_cross_cfg* c, const int64_t* kv_lens, const void* q,
                                          const void* k, const void* v, const void* out, const float* lse,
                                          const void* dout, float scale, void* dq, void* dk, void* dv, void* ws,
                                          void* stream)
{
    CrossStrides qs, kvs;
    sdv2_status s = check_cross(c, &qs, &kvs);
    if (s != SDV2_OK) return s;
    for (const void* p : {q, out, dout, static_cast<const void*>(lse), static_cast<const void*>(dq), static_cast<const void*>(ws)})
        if (!usable(p)) return bad(SDV2_ERR_INVALID_ARG, "device pointers must be non-null and 16-byte aligned");
    for (const void* p : {k, v, static_cast<const void*>(dk), static_cast<const void*>(dv)})
        if (!aligned16(p) || (c->kv_len && !p))
            return bad(SDV2_ERR_INVALID_ARG, "device pointers must be non-null and 16-byte aligned");
    if ((s = check_call(c, kv_lens, &scale)) != SDV2_OK) return s;
    if ((s = require_device()) != SDV2_OK) return s;
    for (int b0 = 0; b0 < c->batch; b0 += kCrossStreams) {
        CrossBackward p{};
        p.c = slice_of(c, kv_lens, qs, kvs, q, k, v, scale, ws, b0, std::min(kCrossStreams, c->batch - b0));
        const int64_t rows = static_cast<int64_t>(b0) * c->heads * c->q_len;
        const int64_t kv_rows = static_cast<int64_t>(b0) * p.c.Hk * c->kv_len;
        p.out = static_cast<const uint16_t*>(out) + rows * 128;
        p.dout = static_cast<const uint16_t*>(dout) + rows * 128;
        p.lse = lse + rows;
        p.dq = static_cast<uint16_t*>(dq) + rows * 128;
        p.dk = static_cast<uint16_t*>(dk) + (dk ? kv_rows * 128 : 0);
        p.dv = static_cast<uint16_t*>(dv) + (dv ? kv_rows * 128 : 0);
        p.stats = reinterpret_cast<float*>(static_cast<unsigned char*>(ws) + kHeaderBytes);
        p.part = reinterpret_cast<float*>(static_cast<unsigned char*>(ws) + kHeaderBytes + stats_bytes(c));
        const cudaError_t e = launch_cross_backward(p, static_cast<cudaStream_t>(stream));
        if (e != cudaSuccess) return done(e, "cross attention backward launch");
    }
    return done(cudaSuccess, "");
}

sdv2_status sdv2_layer_norm(const sdv2_norm_cfg* c, const void* x, const float* weight, const float* bias, void* y,
                            float* mean, float* rstd, void* stream)
{
    sdv2_status s = check_norm(c);
    if (s != SDV2_OK) return s;
    if (!usable(x) || !usable(y)) return bad(SDV2_ERR_INVALID_ARG, "x and y must be non-null and 16-byte aligned");
    for (const void* p : {static_cast<const void*>(weight), static_cast<const void*>(bias), static_cast<const void*>(mean),
                          static_cast<const void*>(rstd)})
        if (!aligned16(p)) return bad(SDV2_ERR_INVALID_ARG, "weight, bias, mean and rstd must be 16-byte aligned");
    if ((s = require_device()) != SDV2_OK) return s;
    NormParams p = norm_params(c, x, weight);
    p.bias = bias;
    p.y = y;
    p.mean = mean;
    p.rstd = rstd;
    return done(launch_layer_norm(p, static_cast<cudaStream_t>(stream)), "layer norm launch");
}

size_t sdv2_norm_workspace_bytes(const sdv2_norm_cfg* c)
{
    if (check_norm(c) != SDV2_OK) return 0;
    const int64_t per = std::min(rows_of(c), c->rows);
    const int slices = norm_backward_slices(c->rows, per, c->cols, norm_params(c, nullptr, nullptr).aligned);
    const size_t groups = static_cast<size_t>((c->rows + per - 1) / per);
    return slices > 1 ? (groups * slices * 2 * c->cols * sizeof(float) + 255) / 256 * 256 : 256;
}

sdv2_status sdv2_layer_norm_backward(const sdv2_norm_cfg* c, const void* dy, const void* x, const float* weight,
                                     const float* mean, const float* rstd, void* dx, float* dweight, float* dbias,
                                     void* ws, void* stream)
{
    sdv2_status s = check_norm(c);
    if (s != SDV2_OK) return s;
    for (const void* p : {dy, x, static_cast<const void*>(mean), static_cast<const void*>(rstd), static_cast<const void*>(dx)})
        if (!usable(p)) return bad(SDV2_ERR_INVALID_ARG, "dy, x, mean, rstd and dx must be non-null and 16-byte aligned");
    for (const void* p : {static_cast<const void*>(weight), static_cast<const void*>(dweight), static_cast<const void*>(dbias),
                          static_cast<const void*>(ws)})
        if (!aligned16(p)) return bad(SDV2_ERR_INVALID_ARG, "weight, dweight, dbias and ws must be 16-byte aligned");
    if ((dweight || dbias) && !ws) return bad(SDV2_ERR_INVALID_ARG, "ws is required for dweight and dbias");
    if ((s = require_device()) != SDV2_OK) return s;
    NormParams p = norm_params(c, x, weight);
    p.dy = dy;
    p.y = dx;
    p.mean = const_cast<float*>(mean);
    p.rstd = const_cast<float*>(rstd);
    p.dweight = dweight;
    p.dbias = dbias;
    p.partial = static_cast<float*>(ws);
    p.slices = norm_backward_slices(p.rows, p.rows_per_group, p.cols, p.aligned);
    return done(launch_layer_norm_backward(p, static_cast<cudaStream_t>(stream)), "layer norm backward launch");
}

}  // extern "C"
