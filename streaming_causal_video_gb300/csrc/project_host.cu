// Host side of the operators in sdv2_project.h: argument checks, derived sizes and dispatch.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <utility>

#include "host_checks.h"
#include "project.h"

namespace sdv2 {
namespace {

constexpr int64_t kMaxLength = int64_t(1) << 30;
constexpr int64_t kMaxStride = int64_t(1) << 38;
constexpr size_t kHeaderBytes = 256;                    // error word, as sdv2_check_device_error reads it

bool is_dtype(int32_t t) { return t == SDV2_BF16 || t == SDV2_F32; }

int tiles_of(int64_t cols) { return static_cast<int>((cols + kMx4Tile - 1) / kMx4Tile); }

sdv2_status check_mx4(const sdv2_mx4_cfg* c)
{
    if (!c) return refuse(SDV2_ERR_INVALID_ARG, "cfg is NULL");
    if (c->rows < 1 || c->rows > kMaxLength || c->cols < 1 || c->cols > kMaxLength)
        return refuse(SDV2_ERR_INVALID_ARG, "rows (%lld) and cols (%lld) must be in [1, 2^30]", (long long)c->rows, (long long)c->cols);
    if (!is_dtype(c->x_dtype)) return refuse(SDV2_ERR_INVALID_ARG, "x_dtype must be SDV2_BF16 or SDV2_F32");
    if (c->transposed != 0 && c->transposed != 1) return refuse(SDV2_ERR_INVALID_ARG, "transposed must be 0 or 1");
    const int64_t width = c->transposed ? c->rows : c->cols;
    if (c->x_row_stride && c->x_row_stride < width)
        return refuse(SDV2_ERR_INVALID_ARG, "x_row_stride (%lld) must be 0 or >= %lld", (long long)c->x_row_stride, (long long)width);
    if (c->x_row_stride > kMaxStride) return refuse(SDV2_ERR_UNSUPPORTED, "x_row_stride must be at most 2^38");
    return SDV2_OK;
}

Mx4Params mx4_params(const sdv2_mx4_cfg* c)
{
    Mx4Params p{};
    p.rows = c->rows;
    p.cols = c->cols;
    p.stride = c->x_row_stride ? c->x_row_stride : c->transposed ? c->rows : c->cols;
    p.tiles = tiles_of(c->cols);
    p.f32 = c->x_dtype == SDV2_F32;
    p.vectors = (p.stride % (p.f32 ? 4 : 8) | p.cols % 8) == 0;
    return p;
}

sdv2_status check_product(const sdv2_mx4_product_cfg* c)
{
    if (!c) return refuse(SDV2_ERR_INVALID_ARG, "cfg is NULL");
    if (std::min({c->rows, c->cols, c->depth}) < 1 || std::max({c->rows, c->cols, c->depth}) > kMaxLength)
        return refuse(SDV2_ERR_INVALID_ARG, "rows (%lld), cols (%lld) and depth (%lld) must be in [1, 2^30]", (long long)c->rows,
                      (long long)c->cols, (long long)c->depth);
    if (!is_dtype(c->out_dtype)) return refuse(SDV2_ERR_INVALID_ARG, "out_dtype must be SDV2_BF16 or SDV2_F32");
    if (c->activation != SDV2_NO_ACTIVATION && c->activation != SDV2_GELU)
        return refuse(SDV2_ERR_INVALID_ARG, "activation must be SDV2_NO_ACTIVATION or SDV2_GELU");
    if (c->out_row_stride && c->out_row_stride < c->cols)
        return refuse(SDV2_ERR_INVALID_ARG, "out_row_stride must be 0 or >= cols");
    if (c->out_row_stride > kMaxStride) return refuse(SDV2_ERR_UNSUPPORTED, "out_row_stride must be at most 2^38");
    if (((c->rows + 255) / 256) * ((c->cols + 255) / 256) > (int64_t(1) << 28))
        return refuse(SDV2_ERR_UNSUPPORTED, "out is larger than 2^28 tiles of 256 x 256");
    return SDV2_OK;
}

// Strides with the defaults filled in, checked.
sdv2_status rope_strides(const char* name, const sdv2_axes_rope_cfg* c, int heads, const sdv2_rope_strides& given_strides,
                         sdv2_rope_strides* s)
{
    *s = given_strides;
    const int64_t low = std::min({s->token_stride, s->head_stride, s->batch_stride});
    const int64_t high = std::max({s->token_stride, s->head_stride, s->batch_stride});
    if (low < 0) return refuse(SDV2_ERR_INVALID_ARG, "%s strides must be >= 0", name);
    if (high > kMaxStride) return refuse(SDV2_ERR_UNSUPPORTED, "%s strides must be at most 2^38", name);
    if (!s->head_stride) s->head_stride = c->head_dim;
    if (!s->token_stride) s->token_stride = static_cast<int64_t>(heads) * c->head_dim;
    const __int128 dense = std::max(static_cast<__int128>(c->tokens) * s->token_stride, static_cast<__int128>(heads) * s->head_stride);
    if (!s->batch_stride) {
        if (c->batch > 1 && dense > kMaxStride) return refuse(SDV2_ERR_UNSUPPORTED, "%s is too large", name);
        s->batch_stride = static_cast<int64_t>(std::min<__int128>(dense, kMaxStride));
    }
    if (s->head_stride < c->head_dim || s->token_stride < c->head_dim || s->batch_stride < 8 ||
        ((s->head_stride | s->token_stride | s->batch_stride) & 7))
        return refuse(SDV2_ERR_INVALID_ARG, "%s token (%lld) and head (%lld) strides must be at least head_dim, the batch stride "
                      "(%lld) at least 8, all multiples of 8", name, (long long)s->token_stride, (long long)s->head_stride,
                      (long long)s->batch_stride);
    return SDV2_OK;
}

// Whether the rows of a result lie apart: from the smallest stride of an axis longer than one on, each passes over all that those
// before it reach.
bool rows_apart(const sdv2_axes_rope_cfg* c, int heads, const sdv2_rope_strides& s)
{
    std::pair<int64_t, int64_t> axis[3] = {{s.head_stride, heads}, {s.token_stride, c->tokens}, {s.batch_stride, c->batch}};
    std::sort(axis, axis + 3);
    __int128 reach = c->head_dim;
    for (const auto& [stride, n] : axis) {
        if (n == 1) continue;
        if (stride < reach) return false;
        reach += static_cast<__int128>(n - 1) * stride;
    }
    return true;
}

sdv2_status check_rope(const sdv2_axes_rope_cfg* c)
{
    if (!c) return refuse(SDV2_ERR_INVALID_ARG, "cfg is NULL");
    if (c->batch < 1 || c->batch > 65535 || c->heads < 1 || c->heads > 65535 || c->kv_heads < 0 || c->kv_heads > 65535)
        return refuse(SDV2_ERR_INVALID_ARG, "batch and heads must be in [1, 65535], kv_heads in [0, 65535]");
    if (c->head_dim < 8 || c->head_dim > 2 * kRopePairs || c->head_dim % 8)
        return refuse(SDV2_ERR_INVALID_ARG, "head_dim (%d) must be a multiple of 8 in [8, %d]", c->head_dim, 2 * kRopePairs);
    if (c->tokens < 1 || c->tokens > kMaxLength)
        return refuse(SDV2_ERR_INVALID_ARG, "tokens (%lld) must be in [1, 2^30]", (long long)c->tokens);
    if (!is_dtype(c->dtype)) return refuse(SDV2_ERR_INVALID_ARG, "dtype must be SDV2_BF16 or SDV2_F32");
    if (c->axes < 1 || c->axes > 4) return refuse(SDV2_ERR_INVALID_ARG, "axes (%d) must be in [1, 4]", c->axes);
    int64_t sum = 0;
    for (int a = 0; a < c->axes; ++a) {
        if (c->dims[a] < 0 || c->dims[a] % 2) return refuse(SDV2_ERR_INVALID_ARG, "dims[%d] (%d) must be even and >= 0", a, c->dims[a]);
        if (!(std::fabs(c->scale[a]) <= 0x1p20)) return refuse(SDV2_ERR_INVALID_ARG, "scale[%d] must be a number of at most 2^20", a);
        sum += c->dims[a];
    }
    if (sum > c->head_dim) return refuse(SDV2_ERR_INVALID_ARG, "the axes' dims (%lld) exceed head_dim (%d)", (long long)sum, c->head_dim);
    if ((c->halves | 1) != 1 || (c->shared_positions | 1) != 1)
        return refuse(SDV2_ERR_INVALID_ARG, "halves and shared_positions must be 0 or 1");
    if (!(c->base > 1.0 && c->base <= 1e100)) return refuse(SDV2_ERR_INVALID_ARG, "base must be in (1, 1e100]");
    return SDV2_OK;
}

// A number as the sum of two doubles, 106 bits: a frequency times a position of 2^31 has 31 bits of whole turns, and the rest
// of it has to be good in 32 bits and more.
struct Twofold {
    double hi, lo;
};

Twofold times(Twofold a, Twofold b)
{
    const double p = a.hi * b.hi;
    const double e = std::fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi);
    const double s = p + e;
    return {s, e - (s - p)};
}

// base^(-2/d), d even: a root in double, made good to twice its bits by a Newton step on root^(d/2) * base = 1.
Twofold frequency_ratio(double base, int d)
{
    const double r = std::pow(base, -2.0 / d);
    Twofold power{1.0, 0.0}, square{r, 0.0};
    for (int n = d / 2; n; n >>= 1) {
        if (n & 1) power = times(power, square);
        square = times(square, square);
    }
    power = times(power, {base, 0.0});
    const double step = -((power.hi - 1.0) + power.lo) / (d / 2) * r;
    const double s = r + step;
    return {s, step - (s - r)};
}

// Turns as a 64-bit fraction of one: whole turns drop out, and a position times the fraction wraps around to what is left.
uint64_t turn_fraction(Twofold turns)
{
    const double part = turns.hi - std::floor(turns.hi);                     // exact for hi >= 0
    const uint64_t f = static_cast<uint64_t>(std::ldexp(part, 64));
    return f + static_cast<uint64_t>(std::llrint(std::ldexp(turns.lo, 64)));
}

// The pairs of a head; the elements of a vector that every half segment is whole ones of.
int rope_pairs(const sdv2_axes_rope_cfg* c, bool backward, AxesRopeParams* p)
{
    constexpr Twofold kTurns{0.15915494309189535, -9.839338337591243e-18};      // 1 / 2pi
    const int lane = c->dtype == SDV2_F32 ? 4 : 8;       // elements of a vector
    int n = 0, first = 0, width = lane;
    auto fits = [&](int half) { width = half % width == 0 ? width : half % 2 == 0 ? 2 : 1; };
    for (int a = 0; a < c->axes; ++a) {
        const int d = c->dims[a];
        if (d == 0) continue;
        fits(d / 2);
        const double scale = c->scale[a] == 0.0 ? 1.0 : c->scale[a];
        const bool negative = (scale < 0) != backward;
        const Twofold ratio = frequency_ratio(c->base, d);
        Twofold turns = times(kTurns, {std::fabs(scale), 0.0});
        for (int j = 0; j < d / 2; ++j, turns = times(turns, ratio)) {
            RopePair& q = p->pair[n++];
            const uint64_t f = turn_fraction(turns);
            q.turn = negative ? 0 - f : f;
            q.u = static_cast<int16_t>(c->halves ? first + j : first + 2 * j);
            q.v = static_cast<int16_t>(c->halves ? first + j + d / 2 : first + 2 * j + 1);
            q.axis = static_cast<int16_t>(a);
        }
        first += d;
    }
    const int rest = c->head_dim - first;
    if (rest) fits(rest / 2);
    for (int j = 0; j < rest / 2; ++j) {
        RopePair& q = p->pair[n++];
        q = RopePair{};
        q.u = static_cast<int16_t>(c->halves ? first + j : first + 2 * j);
        q.v = static_cast<int16_t>(c->halves ? first + j + rest / 2 : first + 2 * j + 1);
        q.axis = -1;
    }
    return width;
}

// The same from the calling thread's last configuration, as most calls have the one of the call before: its pairs depend on
// nothing else.
int rope_table(const sdv2_axes_rope_cfg* c, bool backward, AxesRopeParams* p)
{
    struct Key {
        double base, scale[4];
        int32_t dims[4];
        int32_t axes, head_dim, dtype, halves, backward, pad;
    };
    thread_local Key last{};
    thread_local RopePair pairs[kRopePairs];
    thread_local int width = 0;
    Key key{};
    key.base = c->base;
    for (int a = 0; a < c->axes; ++a) key.scale[a] = c->scale[a], key.dims[a] = c->dims[a];
    key.axes = c->axes;
    key.head_dim = c->head_dim;
    key.dtype = c->dtype;
    key.halves = c->halves;
    key.backward = backward;
    const size_t bytes = static_cast<size_t>(c->head_dim / 2) * sizeof(RopePair);
    if (width == 0 || std::memcmp(&key, &last, sizeof(key)) != 0) {
        width = rope_pairs(c, backward, p);
        std::memcpy(pairs, p->pair, bytes);
        last = key;
    } else {
        std::memcpy(p->pair, pairs, bytes);
    }
    return width;
}

sdv2_status rope_call(const sdv2_axes_rope_cfg* c, const int32_t* positions, const void* q, void* q_new, const void* k,
                      void* k_new, bool backward, void* stream)
{
    sdv2_status s = check_rope(c);
    if (s != SDV2_OK) return s;
    AxesRopeParams p{};
    const sdv2_rope_strides* ends[2][2] = {{&c->q_in, &c->q_out}, {&c->k_in, &c->k_out}};
    for (int t = 0; t < (c->kv_heads ? 2 : 1); ++t) {
        const int heads = t ? c->kv_heads : c->heads;
        sdv2_rope_strides in, out;
        if ((s = rope_strides(t ? "k_in" : "q_in", c, heads, *ends[t][0], &in)) != SDV2_OK) return s;
        if ((s = rope_strides(t ? "k_out" : "q_out", c, heads, *ends[t][1], &out)) != SDV2_OK) return s;
        p.t[t] = {t ? k : q, t ? k_new : q_new, backward ? out : in, backward ? in : out};
        if (!rows_apart(c, heads, p.t[t].os))
            return refuse(SDV2_ERR_INVALID_ARG, "rows of %c_%s overlap: a stride must pass over all that the smaller ones reach", t ? 'k' : 'q',
                          backward ? "in" : "out");
        if (!given(p.t[t].in) || !given(p.t[t].out))
            return refuse(SDV2_ERR_INVALID_ARG, "device pointers must be non-null and 16-byte aligned");
        if (p.t[t].in == p.t[t].out && (in.token_stride != out.token_stride || in.head_stride != out.head_stride ||
                                        (c->batch > 1 && in.batch_stride != out.batch_stride)))
            return refuse(SDV2_ERR_INVALID_ARG, "%s in place needs the same strides in and out", t ? "k" : "q");
    }
    if (!given(positions)) return refuse(SDV2_ERR_INVALID_ARG, "positions must be a non-null 16-byte aligned pointer");
    if ((s = require_device()) != SDV2_OK) return s;
    p.positions = positions;
    p.tokens = c->tokens;
    p.batch = c->batch;
    p.heads = c->heads;
    p.kv_heads = c->kv_heads;
    p.axes = c->axes;
    p.shared = c->shared_positions;
    const int width = rope_table(c, backward, &p);
    const bool all = p.pair[c->head_dim / 2 - 1].axis >= 0;
    return launched(launch_axes_rope(p, !c->halves, width, all, c->dtype == SDV2_F32, c->head_dim, static_cast<cudaStream_t>(stream)),
                    "axes rope launch");
}

}  // namespace
}  // namespace sdv2

using namespace sdv2;

extern "C" {

size_t sdv2_mx4_codes_bytes(const sdv2_mx4_cfg* c)
{
    return check_mx4(c) == SDV2_OK ? static_cast<size_t>(c->rows) * tiles_of(c->cols) * kMx4TileBytes : 0;
}

size_t sdv2_mx4_scales_bytes(const sdv2_mx4_cfg* c)
{
    return check_mx4(c) == SDV2_OK ? static_cast<size_t>(tiles_of(c->rows)) * tiles_of(c->cols) * 512 : 0;
}

sdv2_status sdv2_mx4_quantize(const sdv2_mx4_cfg* c, const void* x, void* codes, void* scales, void* stream)
{
    sdv2_status s = check_mx4(c);
    if (s != SDV2_OK) return s;
    if (!given(x) || !given(codes) || !given(scales))
        return refuse(SDV2_ERR_INVALID_ARG, "x, codes and scales must be non-null and 16-byte aligned");
    if ((s = require_device()) != SDV2_OK) return s;
    Mx4Params p = mx4_params(c);
    p.x = x;
    p.codes = static_cast<uint8_t*>(codes);
    p.scales = static_cast<uint8_t*>(scales);
    return launched(launch_mx4_quantize(p, c->transposed != 0, static_cast<cudaStream_t>(stream)), "4-bit quantisation launch");
}

sdv2_status sdv2_mx4_dequantize(const sdv2_mx4_cfg* c, const void* codes, const void* scales, void* y, void* stream)
{
    sdv2_status s = check_mx4(c);
    if (s != SDV2_OK) return s;
    if (c->transposed) return refuse(SDV2_ERR_UNSUPPORTED, "values are written as the matrix lies: transposed must be 0");
    if (!given(y) || !given(codes) || !given(scales))
        return refuse(SDV2_ERR_INVALID_ARG, "codes, scales and y must be non-null and 16-byte aligned");
    if ((s = require_device()) != SDV2_OK) return s;
    Mx4Params p = mx4_params(c);
    p.y = y;
    p.codes = static_cast<uint8_t*>(const_cast<void*>(codes));
    p.scales = static_cast<uint8_t*>(const_cast<void*>(scales));
    return launched(launch_mx4_dequantize(p, static_cast<cudaStream_t>(stream)), "4-bit values launch");
}

size_t sdv2_mx4_workspace_bytes(const sdv2_mx4_product_cfg* c)
{
    return check_product(c) == SDV2_OK ? kHeaderBytes : 0;
}

sdv2_status sdv2_mx4_workspace_init(const sdv2_mx4_product_cfg* c, void* ws, void* stream)
{
    sdv2_status s = check_product(c);
    if (s != SDV2_OK) return s;
    if (!given(ws)) return refuse(SDV2_ERR_INVALID_ARG, "ws must be a non-null 16-byte aligned pointer");
    if ((s = require_device()) != SDV2_OK) return s;
    return launched(cudaMemsetAsync(ws, 0, kHeaderBytes, static_cast<cudaStream_t>(stream)), "4-bit product workspace");
}

sdv2_status sdv2_mx4_product(const sdv2_mx4_product_cfg* c, const void* a_codes, const void* a_scales, const void* b_codes,
                             const void* b_scales, const float* bias, void* out, void* ws, void* stream)
{
    sdv2_status s = check_product(c);
    if (s != SDV2_OK) return s;
    for (const void* p : {a_codes, a_scales, b_codes, b_scales, static_cast<const void*>(out), static_cast<const void*>(ws)})
        if (!given(p)) return refuse(SDV2_ERR_INVALID_ARG, "device pointers must be non-null and 16-byte aligned");
    if (!on_16_bytes(bias)) return refuse(SDV2_ERR_INVALID_ARG, "bias must be 16-byte aligned");
    if ((s = require_device()) != SDV2_OK) return s;
    Mx4Product p{};
    p.a = static_cast<const uint8_t*>(a_codes);
    p.as = static_cast<const uint8_t*>(a_scales);
    p.b = static_cast<const uint8_t*>(b_codes);
    p.bs = static_cast<const uint8_t*>(b_scales);
    p.bias = bias;
    p.out = out;
    p.M = c->rows;
    p.N = c->cols;
    p.out_stride = c->out_row_stride ? c->out_row_stride : c->cols;
    p.tiles = tiles_of(c->depth);
    p.out_f32 = c->out_dtype == SDV2_F32;
    p.gelu = c->activation == SDV2_GELU;
    p.err = static_cast<uint32_t*>(ws);
    p.timeout_ns = wait_timeout_ns();
    p.drop = debug_drop_tile();
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return launched(p.M <= kMx4FewRows ? launch_mx4_rows(p, st) : launch_mx4_product(p, st), "4-bit product launch");
}

sdv2_status sdv2_debug_mx4_plan(const sdv2_mx4_product_cfg* c, int32_t* plan)
{
    const sdv2_status s = check_product(c);
    if (s != SDV2_OK) return s;
    if (!plan) return refuse(SDV2_ERR_INVALID_ARG, "plan is NULL");
    const int tiles = tiles_of(c->depth);
    const Mx4Plan p = c->rows <= kMx4FewRows ? mx4_rows_plan(c->rows, c->cols, tiles) : mx4_product_plan(c->rows, c->cols, tiles);
    plan[0] = p.width;
    plan[1] = p.parts;
    plan[2] = p.rounds;
    set_last_error("");
    return SDV2_OK;
}

sdv2_status sdv2_axes_rope(const sdv2_axes_rope_cfg* c, const int32_t* positions, const void* q, void* q_out, const void* k,
                           void* k_out, void* stream)
{
    return rope_call(c, positions, q, q_out, k, k_out, false, stream);
}

sdv2_status sdv2_axes_rope_backward(const sdv2_axes_rope_cfg* c, const int32_t* positions, const void* dq_out, void* dq,
                                    const void* dk_out, void* dk, void* stream)
{
    return rope_call(c, positions, dq_out, dq, dk_out, dk, true, stream);
}

}  // extern "C"
