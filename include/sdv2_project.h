/*
 * sdv2_project.h -- C ABI of the operators around a layer's projections: matrices of microscaled
 * 4-bit numbers and their products, and rotary positions of several axes with their gradient.
 *
 * A layer's linear products (queries of the cross attention, outputs, feed-forward, modulation) run
 * between matrices that sdv2_mx4_quantize wrote:
 *   sdv2_mx4_quantize          a matrix, or its transpose, to 4 bits; weights once, activations per call;
 *   sdv2_mx4_product           out = act(a b^T + bias) of two such matrices;
 *   sdv2_mx4_dequantize        the values that the 4 bits stand for.
 * Queries and keys turn by their places in time, height and width (or any other axes):
 *   sdv2_axes_rope             by any positions, in any of the layouts below, in place if wanted;
 *   sdv2_axes_rope_backward    gradients of q and k from those of its results.
 * sdv2_rope_append_kv and sdv2_qkv_rope_append of sdv2.h remain the way into the chunk's cache.
 *
 * The conventions of sdv2.h and sdv2_block.h hold: the caller owns all device memory, work is
 * enqueued on the caller's stream, arguments are checked on the host before anything is launched,
 * device pointers are 16-byte aligned, bf16 results are rounded to nearest even, the same inputs
 * give the same bits on every call, work runs on the current device, outputs do not overlap inputs
 * or one another except where a comment says so.
 */
#ifndef SDV2_PROJECT_H
#define SDV2_PROJECT_H

#include "sdv2_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- matrices of microscaled 4-bit numbers ------------------------------------------------ */

/*
 * A matrix of `rows` rows whose products run along its `cols` columns.  Each 32 consecutive columns
 * of a row share a scale, a power of two; a number is held as e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and
 * their negatives) times it: the element and scale types of the OCP microscaling formats.
 *
 * codes:  [rows][64*T] bytes, T = ceil(cols/128); column c is in byte c/2, an even one in the low
 *         four bits.  Columns at and past `cols` hold 0.
 * scales: [ceil(rows/128)][T][32][4][4] bytes; the byte [r/128][c/128][r%32][(r%128)/32][(c%128)/32]
 *         holds e + 127 for the scale 2^e of row r and column c, or 255 for NaN.  Rows and columns
 *         past the matrix's hold 0.
 * So rows from a multiple of 128 on are a matrix of their own: its codes begin 64*T bytes a row, its
 * scales 512*T bytes for every 128 rows later (the q part of a packed q|k|v weight, say).
 *
 * The scale: with a the block's largest magnitude, 2^e is the least power of two (at least 2^-127)
 * for which a <= 7 * 2^e.  Magnitudes in (6, 7] * 2^e become 6 * 2^e.  (On normally distributed
 * numbers this bound gives the least mean square error: 1.25 % of the mean square, against 1.32 %
 * for a < 8 * 2^e and 1.33 % for a <= 6 * 2^e.)  A number goes to the nearest of the eight
 * magnitudes, from the middle of two to the one with the even code.  A block that holds an infinity
 * or a NaN has the scale NaN, and so every product with it is NaN.
 */
typedef struct {
    int64_t rows;              /* in [1, 2^30]                                                  */
    int64_t cols;              /* in [1, 2^30]                                                  */
    int32_t x_dtype;           /* sdv2_dtype of x                                               */
    int32_t transposed;        /* 0: x is [rows][cols]; 1: x is [cols][rows] (quantize only)    */
    int64_t x_row_stride;      /* elements between rows of x; 0 = dense                         */
} sdv2_mx4_cfg;

/* Bytes of the two arrays; 0 on an invalid configuration. */
size_t sdv2_mx4_codes_bytes(const sdv2_mx4_cfg* cfg);
size_t sdv2_mx4_scales_bytes(const sdv2_mx4_cfg* cfg);

/* x: device, as the configuration says.  codes, scales: device, written whole.  Exact: there is no
 * rounding but that of each number to its four bits. */
sdv2_status sdv2_mx4_quantize(const sdv2_mx4_cfg* cfg, const void* x, void* codes, void* scales, void* stream);

/* y[rows][cols] of type x_dtype, rows x_row_stride apart (columns between rows are left as they
 * were): the values, which bf16 holds exactly.  A magnitude of 2^128 becomes an infinity, and every
 * number of a block with the scale NaN a NaN.  transposed must be 0. */
sdv2_status sdv2_mx4_dequantize(const sdv2_mx4_cfg* cfg, const void* codes, const void* scales, void* y, void* stream);

typedef enum {
    SDV2_NO_ACTIVATION = 0,
    SDV2_GELU = 1              /* y/2 * (1 + tanh(sqrt(2/pi) * (y + 0.044715 y^3))); y below     */
                               /* -7.2 as -7.2, whose result is -2^-52                          */
} sdv2_activation;

typedef struct {
    int64_t rows;              /* M in [1, 2^30]: rows of a and of out                          */
    int64_t cols;              /* N in [1, 2^30]: rows of b, columns of out                     */
    int64_t depth;             /* K in [1, 2^30]: columns of a and of b                         */
    int32_t out_dtype;         /* sdv2_dtype of out                                             */
    int32_t activation;        /* sdv2_activation                                               */
    int64_t out_row_stride;    /* elements between rows of out; 0 = cols                        */
} sdv2_mx4_product_cfg;

/* Bytes of the workspace of products with this configuration: the device error word (256 bytes).
 * 0 on an invalid configuration. */
size_t sdv2_mx4_workspace_bytes(const sdv2_mx4_product_cfg* cfg);

/* Zeroes the error word and enqueues nothing else; one workspace serves every configuration, and calls
 * that overlap on the GPU.  Waits on the device are bounded by sdv2_set_wait_timeout_ns;
 * sdv2_check_device_error(ws, stream) reads the word.  With sdv2_debug_drop_kv_tile set, a product
 * leaves out the copy of the 256 columns of a and b with this number. */
sdv2_status sdv2_mx4_workspace_init(const sdv2_mx4_product_cfg* cfg, void* ws, void* stream);

/*
 * out[m][n] = act(sum_k a[m][k] * b[n][k] + bias[n]).
 *
 * a_codes, a_scales: a matrix of `rows` rows and `depth` columns; b_codes, b_scales: one of `cols`
 *   rows and `depth` columns, both as sdv2_mx4_quantize writes them (a and b may be the same).
 * bias: device fp32 [cols], or NULL.
 * out: device, rows out_row_stride apart; columns between rows are left as they were.
 * Numerics: products of the 4-bit numbers are exact, their sums, the bias and the activation are
 *   fp32, and out is rounded once.
 *
 * Gradients of a product y = x w^T, x [M][K], w [N][K], are products too: with dy quantised along N
 * and w transposed, dx = dy w is a product of depth N; with dy and x both transposed, and so
 * quantised along M, dw = dy^T x is one of depth M.  (The gradient of the rounding to 4 bits is
 * taken to be 1; the library has no gradient of the activation.)
 */
sdv2_status sdv2_mx4_product(const sdv2_mx4_product_cfg* cfg, const void* a_codes, const void* a_scales,
                             const void* b_codes, const void* b_scales, const float* bias, void* out, void* ws,
                             void* stream);

/*
 * How sdv2_mx4_product runs a configuration on a GB300, for tests and measurements; host only.
 *   plan[0]: 16, 32 or 64 where the rows of a, at most that many, are the columns of the MMAs; otherwise
 *            128, 192 or 256, the rows of b in a tile of 256 rows of a;
 *   plan[1]: the parts that the depth of each tile is cut in;
 *   plan[2]: the most tiles that a pair of SMs takes one after another (1 for the few rows).
 */
sdv2_status sdv2_debug_mx4_plan(const sdv2_mx4_product_cfg* cfg, int32_t* plan);

/* ---- rotary positions of several axes ------------------------------------------------------- */

/* Element (b, n, h, d) lies batch_stride*b + token_stride*n + head_stride*h + d elements after a tensor's pointer.  0
 * selects the dense token-major value: head stride head_dim, token stride heads*head_dim, batch
 * stride max(tokens*token stride, heads*head stride). */
typedef struct {
    int64_t token_stride, head_stride, batch_stride;
} sdv2_rope_strides;

/*
 * q is [batch][tokens][heads][head_dim], k (if kv_heads > 0) [batch][tokens][kv_heads][head_dim].
 * The first dims[0] dims of a head turn by the token's place on axis 0, the next dims[1] by axis 1,
 * and so on; dims behind the last axis stay as they are.  Inside a segment of d dims, pair j turns
 * by the angle scale[a] * position[a] * base^(-2j/d):
 *   (u, v) -> (u cos - v sin, u sin + v cos).
 * halves = 0: pair j is dims (2j, 2j+1) of its segment; halves = 1: dims (j, j + d/2).
 * Strides are multiples of 8 elements (the token and the head stride at least head_dim) and at most 2^38.  Rows of a result
 * (q_out and k_out; of the gradients q_in and k_in) lie apart: ordered by size, each stride of an axis longer than one passes over
 * all that those before it reach.  Rows that are only read may share memory.
 */
typedef struct {
    int32_t batch;             /* in [1, 65535]                                                 */
    int32_t heads;             /* in [1, 65535]                                                 */
    int32_t kv_heads;          /* 0: there is no k; otherwise in [1, 65535]                     */
    int32_t head_dim;          /* a multiple of 8 in [8, 256]                                   */
    int64_t tokens;            /* in [1, 2^30]                                                  */
    int32_t dtype;             /* sdv2_dtype of q and k, in and out                             */
    int32_t axes;              /* in [1, 4]                                                     */
    int32_t dims[4];           /* each even and >= 0, their sum <= head_dim                     */
    int32_t halves;
    int32_t shared_positions;  /* 0: positions [batch][tokens][axes]; 1: [tokens][axes]         */
    double base;               /* in (1, 1e100]                                                 */
    double scale[4];           /* in [-2^20, 2^20]; 0 selects 1                                 */
    sdv2_rope_strides q_in, q_out, k_in, k_out;
} sdv2_axes_rope_cfg;

/*
 * positions: device int32, any values.  q, k: device; q_out, k_out: device, each of which may be its
 * input itself if their strides are the same.  k and k_out are not read if kv_heads is 0.
 * Numerics: a position's whole turns drop out exactly (64-bit fixed point), so far positions are as
 * good as near ones; sine, cosine and rotation are fp32; results are rounded once.
 */
sdv2_status sdv2_axes_rope(const sdv2_axes_rope_cfg* cfg, const int32_t* positions, const void* q, void* q_out,
                           const void* k, void* k_out, void* stream);

/* dq, dk from the gradients dq_out, dk_out of q_out and k_out: the rotation by the negative angle.
 * dq_out, dk_out have the strides q_out, k_out, and dq, dk the strides q_in, k_in; each result may be
 * its gradient itself if the two are the same. */
sdv2_status sdv2_axes_rope_backward(const sdv2_axes_rope_cfg* cfg, const int32_t* positions, const void* dq_out,
                                    void* dq, const void* dk_out, void* dk, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SDV2_PROJECT_H */
