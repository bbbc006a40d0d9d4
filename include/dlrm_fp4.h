/*
 * dlrm_fp4.h -- C ABI of the 4-bit layers on B200: rows rounded to 4-bit floating
 * point with a power of two for every 32 elements (microscaling, MXFP4), and the
 * layer that multiplies them on the tensor cores.
 *
 * They stand beside the 8-bit layers of dlrm_int8.h: half of their bytes at twice
 * their tensor rate, with scales along K in place of one for each row.
 *
 * An element is e2m1: a sign (bit 3) and a magnitude of 0, 0.5, 1, 1.5, 2, 3, 4 or 6
 * (codes 0 .. 7). 32 neighbours along K, from a multiple of 32 on, share a scale
 * byte E that stands for 2^(E - 127) (E8M0; 255 is NaN). The rounding takes the least
 * power of two that brings the block's largest magnitude to 7 or less (6 is nearest to all
 * from 5 to 7), but 2^-127 at least, and each element times its inverse to the nearest
 * magnitude, ties to the even code. A block that holds a NaN or an infinity gets the
 * scale NaN and codes 0: what is computed from it is NaN. A block of zeros has E = 0.
 *
 * A matrix of M rows and K columns is
 *   q      bytes (M, ldq): column 2i in the low and 2i + 1 in the high half of byte i;
 *          with K odd the last half is zero.
 *   scale  bytes in tiles of 128 rows x 4 blocks, as the tensor cores read them:
 *          (ceil(M / 128), ceil(K / 128), 512), where row r and block b of a tile are
 *          at (r % 32) * 16 + (r / 32) * 4 + b. Bytes past the matrix are zero.
 *          dlrm_fp4_scale_bytes() in all.
 *
 * Conventions as in dlrm_optim.h (the same library, libdlrm_narrow.so).
 */
#ifndef DLRM_FP4_H
#define DLRM_FP4_H

#include <stdint.h>

#include "dlrm_mlp.h"
#include "dlrm_sparse.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Elements of a row that share a scale. */
#define DLRM_FP4_BLOCK 32

/* Bytes of the scales of an (M, K) matrix, or DLRM_ERR_SHAPE. M 0 .. 2^31 - 1025,
 * K 1 .. 2^31 - 1025, and M K, both rounded up to multiples of 128, at most 2^38 (M K itself below
 * it); so it is for the two calls below. */
DLRM_API int64_t dlrm_fp4_scale_bytes(int64_t M, int64_t K);

/* dlrm_quantize_fp4 -- (q, scale) of the rows of x.
 *   x      dev (M, ldx) of dtype (dlrm_table_dtype_t).
 *   q      dev bytes (M, ldq), ldq >= (K + 1) / 2; bytes past those are left as they
 *          were.
 *   scale  dev, 4-byte aligned, dlrm_fp4_scale_bytes(M, K) bytes, all written.
 * With M == 0 nothing is enqueued. */
DLRM_API int dlrm_quantize_fp4(const void* x, int64_t ldx, int dtype, int64_t M, int64_t K,
                               uint8_t* q, int64_t ldq, uint8_t* scale, dlrm_stream_t stream);

/* dlrm_dequantize_fp4 -- y[m][k] = the value that q and scale hold, rounded once to dtype.
 * y dev (M, ldy); columns past K are left as they were. scale 4-byte aligned. */
DLRM_API int dlrm_dequantize_fp4(const uint8_t* q, int64_t ldq, const uint8_t* scale, int64_t M,
                                 int64_t K, void* y, int dtype, int64_t ldy,
                                 dlrm_stream_t stream);

/*
 * dlrm_linear_fp4 -- y[m][n] = act(sum_k x[m][k] w[n][k] + bias[n]).
 *   x, x_scale  an (M, K) matrix as above, dev.
 *   w, w_scale  an (N, K) matrix, dev.
 *   bias        dev f32 (N,), or NULL.
 *   act         dlrm_act_t.
 *   y           dev (M, ldy) of y_dtype (dlrm_table_dtype_t); columns past N are
 *               left as they were.
 *   status_dev  dev int32, or NULL: DLRM_FLAG_TIMEOUT is OR-ed in if a bounded wait of
 *               the kernel ran out (the results are then not valid).
 * Products are exact, sums are f32 (in an order that the sizes fix: equal calls give equal
 * bits), the bias and the activation are applied in f32 and the result is rounded once.
 * Requirements (DLRM_ERR_SHAPE / DLRM_ERR_ALIGN otherwise): M >= 0 (with M == 0
 * nothing is enqueued), N >= 1, K >= 1, all below 2^31 - 1024, and no more than 2^31 - 1 tiles of 64
 * rows of x by 128 of w; ldx, ldw >= (K + 1) / 2 and below 2^40 (where there is more than one row),
 * multiples of 16, ldy >= N; x, w and the scales 16-byte aligned (the TMA loads), the
 * others aligned to their elements. Bytes of x and w past (K + 1) / 2 are never
 * used; scale bytes past the matrix must be zero, and so must the last half byte of x or
 * of w where K is odd.
 */
DLRM_API int dlrm_linear_fp4(const uint8_t* x, int64_t ldx, const uint8_t* x_scale,
                             const uint8_t* w, int64_t ldw, const uint8_t* w_scale,
                             const float* bias, int64_t M, int64_t N, int64_t K, int act, void* y,
                             int y_dtype, int64_t ldy, int32_t* status_dev, dlrm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DLRM_FP4_H */
