/*
 * sdv2_block.h -- C ABI of the operators around the chunk attention in a streaming video DiT's
 * layer: cross attention to the states of a prompt encoder, and layer norm, each with its
 * backward pass.
 *
 * A layer normalises its tokens (scale and shift of each latent frame), projects and appends them
 * (sdv2_qkv_rope_append), attends to the chunk's cache (sdv2_chunk_attention), normalises again
 * (learned weight and bias), and attends to the prompt:
 *   sdv2_layer_norm            y = (x - mean) / sqrt(var + eps), times a weight, plus a bias;
 *   sdv2_cross_attention       the chunk's queries attend to each stream's prompt states.
 * sdv2_layer_norm_backward and sdv2_cross_attention_backward give the gradients of these two, so
 * that what the prompt passes through (adapters, prompt states, norms) can be trained.  The library
 * has no gradient of the chunk attention, of RoPE or of the projections: a loss that has to pass
 * through those needs the caller's own.
 *
 * The conventions of sdv2.h hold: the caller owns all device memory, work is enqueued on the
 * caller's stream, arguments are checked on the host before anything is launched, host arrays are
 * read before the call returns, device pointers are 16-byte aligned, bf16 results are rounded to
 * nearest even.  Every result is deterministic: the same inputs give the same bits on every call.
 * Outputs must not overlap inputs or one another, except where a comment says so.  Work runs on
 * the current device, which must be the one that the pointers and the stream belong to.  A call's
 * kernels may start while the stream's kernel before them ends; they wait for it before they touch
 * memory.
 */
#ifndef SDV2_BLOCK_H
#define SDV2_BLOCK_H

#include "sdv2.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- cross attention -------------------------------------------------------------------- */

/*
 * Shapes and strides.  Element (b, i, h, d) of q lies q_batch_stride*b + q_token_stride*i +
 * q_head_stride*h + d elements after its pointer; k and v share their three strides.  A stride of
 * 0 selects the dense token-major value: head stride D, token stride heads*D, batch stride
 * max(length*token stride, heads*head stride).  So a packed [token][2][Hk][D] projection is read
 * in place as two pointers with kv_token_stride = 2*Hk*D, and head-major rows [H][length][D] with
 * token stride D and head stride length*D.  Token and head strides are at least 128, and all
 * strides are multiples of 8 and at most 2^38.
 * With kv_heads < heads, query head h reads key head h / (heads / kv_heads).
 * Streams that share one prompt and whose queries follow one another in memory are one stream of
 * batch * q_len queries.
 */
typedef struct {
    int32_t batch;             /* B >= 1 streams                                               */
    int32_t heads;             /* H >= 1 query heads                                           */
    int32_t kv_heads;          /* Hk >= 1, divides H; 0 = H                                    */
    int32_t head_dim;          /* D; only 128 is built                                         */
    int64_t q_len;             /* Nq in [1, 2^30]: queries of every stream                     */
    int64_t kv_len;            /* Nk in [0, 2^30]: rows of k and v of every stream             */
    int64_t q_token_stride, q_head_stride, q_batch_stride;
    int64_t kv_token_stride, kv_head_stride, kv_batch_stride;
} sdv2_cross_cfg;

/* Bytes of the workspace of cross attention calls with this configuration: the device error word
 * (256 bytes), and with backward != 0 the scratch of sdv2_cross_attention_backward as well.  The
 * workspace holds nothing from one call to the next but the error word.  Calls that use it must
 * not overlap on the GPU.  0 on an invalid configuration. */
size_t sdv2_cross_workspace_bytes(const sdv2_cross_cfg* cfg, int32_t backward);

/* Zeroes the error word (the workspace's first 256 bytes) and enqueues nothing else; one workspace
 * serves every configuration that it is large enough for.  Waits on the device are bounded by
 * sdv2_set_wait_timeout_ns; sdv2_check_device_error(ws, stream) reads the word.  With
 * sdv2_debug_drop_kv_tile set, sdv2_cross_attention leaves out the copy of that key tile, and
 * sdv2_cross_attention_backward, where dQ is formed, that of the key tile, and where dK and dV are
 * formed, that of the query tile with this number.  It has no effect where no tiles are copied: on
 * the forward pass of one or two query rows per key head (q_len * heads / kv_heads) whose streams
 * have at most 1024 valid states. */
sdv2_status sdv2_cross_workspace_init(const sdv2_cross_cfg* cfg, void* ws, void* stream);

/*
 * out[b][i][h][:] = sum_{j < n_b} softmax_j(scale * <q[b][i][h], k[b][j][h']>) v[b][j][h'].
 *
 * kv_lens: HOST array of B int64, n_b in [0, Nk]: the valid rows of each stream's k and v; NULL =
 *   Nk for all.  Rows at and past n_b have no influence, whatever they hold.  A stream with
 *   n_b = 0 gets out = 0 and lse = -infinity.
 * q, k, v: device bf16 as described above (k and v may be NULL if Nk = 0).
 * scale: softmax scale; <= 0 (or no number) selects 1/sqrt(D).
 * out: device bf16 [B][Nq][H][D]; lse: device fp32 [B][H][Nq], natural log-sum-exp of the scaled
 *   scores, or NULL.
 * Numerics: bf16 products with fp32 accumulation, online softmax in fp32, probabilities rounded
 * to bf16 for the product with v on the tensor cores (their sum is taken before the rounding).
 */
sdv2_status sdv2_cross_attention(const sdv2_cross_cfg* cfg, const int64_t* kv_lens, const void* q, const void* k,
                                 const void* v, float scale, void* out, float* lse, void* ws, void* stream);

/*
 * Gradients of sdv2_cross_attention.  With P = softmax(scale Q K^T), dP = dO V^T and
 * delta = rowsum(dO * O):  dS = P * (dP - delta),  dQ = scale dS K,  dK = scale dS^T Q,
 * dV = P^T dO; dK and dV of a key head are summed over the query heads that share it.
 *
 * out, lse: what sdv2_cross_attention wrote for the same arguments (lse is required).
 * dout: device bf16 [B][Nq][H][D].  dq: device bf16 [B][Nq][H][D]; dk, dv: device bf16
 * [B][Nk][Hk][D], written whole: rows at and past n_b are 0 (dk, dv may be NULL if Nk = 0).
 * A stream with n_b = 1 has dq = dk = 0, as a softmax over one key is constant.
 * ws: workspace of sdv2_cross_workspace_bytes(cfg, 1) bytes.
 * Numerics: P and dS are rounded to bf16 for the tensor-core products; sums are fp32.  A stream of
 * 128 keys or fewer takes delta = rowsum(P * dP), which does not carry the rounding of out.
 */
sdv2_status sdv2_cross_attention_backward(const sdv2_cross_cfg* cfg, const int64_t* kv_lens, const void* q,
                                          const void* k, const void* v, const void* out, const float* lse,
                                          const void* dout, float scale, void* dq, void* dk, void* dv, void* ws,
                                          void* stream);

/* ---- layer norm ------------------------------------------------------------------------- */

typedef enum { SDV2_BF16 = 0, SDV2_F32 = 1 } sdv2_dtype;

/*
 * Rows are normalised over their `cols` columns.  weight and bias (fp32) have one row of `cols`
 * values for every group of rows_per_group consecutive rows (the last group may be shorter):
 * one group for a learned affine, one per latent frame for the scale and shift of a modulated
 * norm, whose weight is an offset from 1 (weight_plus_one = 1).
 */
typedef struct {
    int64_t rows;              /* in [1, 2^31 - 1]                                             */
    int32_t cols;              /* in [1, 16384]                                                */
    int32_t x_dtype, y_dtype;  /* sdv2_dtype of x, dx and of y, dy                             */
    int32_t weight_plus_one;   /* 0: y = xhat*weight + bias; 1: y = xhat*(1 + weight) + bias   */
    int64_t x_row_stride;      /* elements between rows of x; 0 = cols                         */
    int64_t y_row_stride;      /* elements between rows of y and of dy; 0 = cols               */
    int64_t rows_per_group;    /* 0 = all rows are one group                                   */
    int64_t group_stride;      /* elements between groups of weight and of bias; 0 = cols      */
    float eps;                 /* >= 0, finite                                                 */
} sdv2_norm_cfg;

/*
 * mean = sum(x)/cols, var = sum((x - mean)^2)/cols, rstd = 1/sqrt(var + eps),
 * y = (x - mean) * rstd * (weight or 1 + weight) + bias, all in fp32, one rounding to y's type.
 * x: device [rows][cols], rows x_row_stride apart; y: device, rows y_row_stride apart (y may be x
 *   itself if types and strides are the same; columns past cols are left as they were).
 * weight, bias: device fp32, or NULL (weight 1, bias 0; weight_plus_one then has no effect).
 * mean, rstd: device fp32 [rows] for the backward pass, or NULL.
 */
sdv2_status sdv2_layer_norm(const sdv2_norm_cfg* cfg, const void* x, const float* weight, const float* bias, void* y,
                            float* mean, float* rstd, void* stream);

/* Bytes of the workspace of sdv2_layer_norm_backward (partial sums of dweight and dbias); 0 on an
 * invalid configuration.  It needs no initialisation and holds nothing between calls; calls that
 * use it must not overlap on the GPU. */
size_t sdv2_norm_workspace_bytes(const sdv2_norm_cfg* cfg);

/*
 * Gradients of sdv2_layer_norm.  With xhat = (x - mean)*rstd and g = dy * (weight or 1 + weight):
 *   dx = rstd * (g - mean(g) - xhat * mean(g * xhat)),
 *   dweight[group] = sum of dy * xhat, dbias[group] = sum of dy over the group's rows.
 * dy: device [rows][cols] of y's type, rows y_row_stride apart; x, mean, rstd: as the forward pass
 * had and wrote them; dx: device of x's type, rows x_row_stride apart (it may be x itself, or dy
 * if types and strides are the same).  dweight, dbias: device fp32 [groups][cols], dense; each may
 * be NULL.  ws: may be NULL if both are NULL.
 */
sdv2_status sdv2_layer_norm_backward(const sdv2_norm_cfg* cfg, const void* dy, const void* x, const float* weight,
                                     const float* mean, const float* rstd, void* dx, float* dweight, float* dbias,
                                     void* ws, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SDV2_BLOCK_H */
