/*
 * dlrm_tokens.h -- C ABI of the token-level table operators on B200: the rows
 * of an embedding table by id, and the table's gradient.
 *
 * The pooled stage (dlrm_sparse.h) reads its tables; these two calls are what
 * a program needs beside it to use a table token by token (histories that a
 * sequence tower reads unpooled) and to train it:
 *
 *   dlrm_embedding_lookup   Y[t]  = scale * W[ids[t]]
 *   dlrm_embedding_grad     dW[r] = scale * sum over t with ids[t] == r of dY[t / L]
 *
 * With L = 1 the second is the gradient of the first; with L > 1 it is the
 * gradient of a sum-pooled bag of L ids (embbag_sum_multi, one table), where
 * dY has one row for each bag.
 *
 * The library (libdlrm_tokens.so, with the calls of dlrm_int8.h) follows the
 * conventions of dlrm_sparse.h: "dev" pointers are device pointers on the
 * current device, the caller owns every buffer (the gradient's scratch
 * included), nothing is allocated or kept between calls, calls are
 * asynchronous on `stream` and can be captured into CUDA graphs, a negative
 * return is a dlrm_status_t, and host-side checks run before anything is
 * enqueued. Element types are dlrm_table_dtype_t. Outputs must not alias
 * inputs unless a call says so.
 */
#ifndef DLRM_TOKENS_H
#define DLRM_TOKENS_H

#include <stdint.h>

#include "dlrm_sparse.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * dlrm_embedding_lookup -- Y[t, :] = scale * W[ids[t], :], t < T.
 *   table       dev (rows, ldw) of table_dtype; columns [0, D) are used.
 *   rows        1 .. 2^31 - 2; D is 1 .. 2^22.
 *   ids         dev int32 (T,); may be NULL iff T == 0.
 *   T           0 .. 2^31 - 1; with T == 0 nothing is enqueued (but the status
 *               word is cleared).
 *   scale       multiplied in f32; the product is rounded once to out_dtype.
 *   padding_idx an id whose rows of Y are zero, or -1 for none.
 *   out         dev (T, ldo) of out_dtype; columns past D are left as they were.
 *   status_dev  dev int32 or NULL; zeroed on `stream`, then DLRM_FLAG_INDEX_OOB
 *               is OR-ed in if an id lies outside [0, rows). Such an id reads
 *               nothing and its row of Y is zero, with or without a status word.
 * ldw, ldo >= D. Pointers are aligned to their element size; rows whose base
 * and pitch are multiples of 16 bytes use 128-bit accesses, others those of two
 * elements or one, with the same results.
 */
DLRM_API int dlrm_embedding_lookup(const void* table, int table_dtype, int64_t ldw, int64_t rows,
                                   int64_t D, const int32_t* ids, int64_t T, float scale,
                                   int64_t padding_idx, void* out, int out_dtype, int64_t ldo,
                                   int32_t* status_dev, dlrm_stream_t stream);

/* Bytes of scratch that dlrm_embedding_grad needs for these sizes (0 for few
 * tokens into a small table, else a multiple
 * of 16), or a negative dlrm_status_t for sizes that it refuses. */
DLRM_API int64_t dlrm_embedding_grad_scratch_bytes(int64_t T, int64_t rows, int64_t D);

/*
 * dlrm_embedding_grad -- out[r, :] = scale * sum_{t: ids[t] == r} grad[t / L, :].
 * The tokens are sorted by id (stable), and the rows of equal ids are summed in
 * f32 in an order that the sizes, types and alignments fix: equal calls give
 * equal bits.
 *   grad        dev (T / L, ldg) of grad_dtype; columns [0, D) are used. May be
 *               NULL iff T == 0.
 *   ids         dev int32 (T,); may be NULL iff T == 0.
 *   L           ids for each row of grad, >= 1; T must be a multiple of it.
 *   rows        rows of the table, 1 .. 2^31 - 2.
 *   scale       multiplied into each finished sum, in f32.
 *   padding_idx an id whose tokens are left out, or -1 for none.
 *   out         dev (rows, ldo) of out_dtype; columns past D are left as they were.
 *   accumulate  0: out is written; rows that no token names become zero.
 *               1: the sums are added to out in f32 and rounded once; rows that
 *               no token names are neither read nor written (with scale = -lr
 *               and out the table itself: one sparse SGD step).
 *   scratch     dev, 16-byte aligned, of at least
 *               dlrm_embedding_grad_scratch_bytes(T, rows, D) bytes
 *               (DLRM_ERR_SCRATCH otherwise; NULL if that is 0); its contents
 *               need not be set. Calls
 *               whose work overlaps on the GPU must not share it.
 *   status_dev  as for dlrm_embedding_lookup; an id outside [0, rows) adds
 *               nothing.
 */
DLRM_API int dlrm_embedding_grad(const void* grad, int grad_dtype, int64_t ldg, const int32_t* ids,
                                 int64_t T, int64_t L, int64_t rows, int64_t D, float scale,
                                 int64_t padding_idx, void* out, int out_dtype, int64_t ldo,
                                 int accumulate, void* scratch, int64_t scratch_bytes,
                                 int32_t* status_dev, dlrm_stream_t stream);

/* cudaError_t of the last failing CUDA call made by this thread in this library. */
DLRM_API int dlrm_tokens_last_cuda_error(void);

/* Number of kernels this library has launched in this process (all threads). */
DLRM_API int64_t dlrm_tokens_launch_count(void);

#ifdef __cplusplus
}
#endif

#endif /* DLRM_TOKENS_H */
