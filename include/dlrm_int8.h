/*
 * dlrm_int8.h -- C ABI of the 8-bit layers on B200: rows rounded to 8-bit
 * integers with one f32 scale each (after a root-mean-square norm of
 * x + residual, or as they are), and the layer that multiplies them by 8-bit
 * weights with one scale for each output channel.
 *
 * They stand beside the bf16 and f32-activation layers of dlrm_mlp.h: a layer
 * here reads half of the bytes of a bf16 one, and the tensor cores multiply
 * 8-bit integers at twice the bf16 rate with an exact int32 sum.
 *
 * A row v of K values is held as q (int8) and s (f32): v[k] ~ q[k] * s with
 * s = max|v| / 127 and q[k] = v[k] / s rounded to nearest, ties to even, so
 * |q| <= 127 (q is that of the unrounded s, also where s is a subnormal of f32 or
 * below). A row of zeros has s = 0 and q = 0. A row that holds a NaN or an infinity
 * has s = NaN and q = 0: what is computed from it is NaN.
 *
 * Conventions as in dlrm_tokens.h (the same library, libdlrm_tokens.so).
 */
#ifndef DLRM_INT8_H
#define DLRM_INT8_H

#include <stdint.h>

#include "dlrm_mlp.h"
#include "dlrm_sparse.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest inner size of dlrm_linear_int8: 2^17 - 1 products of two 8-bit
 * integers, each at most 2^14 in size, cannot leave int32. */
#define DLRM_INT8_MAX_K 131071

/*
 * dlrm_rms_norm_int8 -- for each row: h = x + residual, y = h * weight /
 * sqrt(mean(h^2) + eps), (q, scale) = y in 8 bits.
 *   x         dev (M, ldx) of dtype (dlrm_table_dtype_t).
 *   residual  dev (M, ldr) of dtype, or NULL for none (h = x).
 *   weight    dev f32 (K,), or NULL for ones.
 *   eps       >= 0.
 *   h_out     dev (M, ldh) of dtype: h rounded once, or NULL. It may be the
 *             residual's own buffer (same pointer and pitch) or x's.
 *   q         dev int8 (M, ldq); columns past K are left as they were.
 *   scale     dev f32 (M,).
 * The sum h is f32 (it is not rounded to dtype before it is normed; where it
 * leaves f32 it is an infinity). Squares and products with the weight are f32, and
 * 64 bits for rows where those would leave f32 or vanish in it. M >= 0 (with
 * M == 0 nothing is enqueued), K >= 1, pitches >= K, M and K < 2^31.
 */
DLRM_API int dlrm_rms_norm_int8(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                                int dtype, const float* weight, int64_t M, int64_t K, float eps,
                                void* h_out, int64_t ldh, int8_t* q, int64_t ldq, float* scale,
                                dlrm_stream_t stream);

/* dlrm_quantize_int8 -- (q, scale) of the rows of x themselves; arguments as
 * for dlrm_rms_norm_int8. Rows of activations, or of weights (N, K): one scale
 * for each output channel. */
DLRM_API int dlrm_quantize_int8(const void* x, int64_t ldx, int dtype, int64_t M, int64_t K,
                                int8_t* q, int64_t ldq, float* scale, dlrm_stream_t stream);

/* dlrm_dequantize_int8 -- y[m][k] = q[m][k] * scale[m], rounded once to dtype.
 * q dev int8 (M, ldq), y dev (M, ldy). */
DLRM_API int dlrm_dequantize_int8(const int8_t* q, int64_t ldq, const float* scale, int64_t M,
                                  int64_t K, void* y, int dtype, int64_t ldy,
                                  dlrm_stream_t stream);

/*
 * dlrm_linear_int8 -- y[m][n] = act(x_scale[m] * w_scale[n] * sum_k x[m][k] w[n][k] + bias[n]).
 *   x        dev int8 (M, ldx), columns [0, K); any values, -128 included.
 *   x_scale  dev f32 (M,).
 *   w        dev int8 (N, ldw), columns [0, K).
 *   w_scale  dev f32 (N,).
 *   bias     dev f32 (N,), or NULL.
 *   act      dlrm_act_t.
 *   y        dev (M, ldy) of y_dtype (dlrm_table_dtype_t); columns past N are
 *            left as they were.
 *   status_dev dev int32, or NULL: DLRM_FLAG_TIMEOUT is OR-ed in if a bounded
 *            wait of the kernel ran out (the results are then not valid).
 * The sum over k is exact in int32; the scales, the bias and the activation
 * are applied in f32, from left to right (sum * x_scale, times w_scale, plus bias:
 * a product of the first two that leaves f32 stays infinite whatever w_scale is),
 * and the result is rounded once.
 * Requirements (DLRM_ERR_SHAPE / DLRM_ERR_ALIGN otherwise): M >= 0 (with
 * M == 0 nothing is enqueued), N >= 1, 1 <= K <= DLRM_INT8_MAX_K, M and N <
 * 2^31 - 1024; ldx, ldw >= K and ldy >= N; ldx and ldw multiples of 16 and x, w
 * 16-byte aligned (the TMA loads); the others aligned to their elements.
 * Columns past K of x and w are never used.
 */
DLRM_API int dlrm_linear_int8(const int8_t* x, int64_t ldx, const float* x_scale, const int8_t* w,
                              int64_t ldw, const float* w_scale, const float* bias, int64_t M,
                              int64_t N, int64_t K, int act, void* y, int y_dtype, int64_t ldy,
                              int32_t* status_dev, dlrm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DLRM_INT8_H */
