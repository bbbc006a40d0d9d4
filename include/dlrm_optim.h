/*
 * dlrm_optim.h -- C ABI of the optimiser step on B200: one AdamW step over many
 * tensors at once, with moments in 32 or in 8 bits.
 *
 * It stands beside the sparse SGD step of dlrm_embedding_grad(accumulate) and
 * trains what that does not reach: the layers of dlrm_mlp.h, and tables by a dense
 * gradient.
 *
 * For an element with weight p and gradient G, at step t:
 *
 *   g = grad_scale * G
 *   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr decay) - lr / (1 - beta1^t) * m / (sqrt(v / (1 - beta2^t)) + eps)
 *
 * Moments lie in one flat buffer (the arena): tensor i's elements start where
 * those before it end, rounded up to a multiple of 256 elements. Elements behind a
 * tensor's end, up to that multiple, belong to no tensor; they start as zeros and
 * stay so.
 *
 * In 8 bits, 256 elements of the arena share one f32 scale for each moment. The
 * first is e4m3 (finite codes, sign in the top bit) times its scale, which puts the
 * block's largest at 448. Of the second the root is held: e = code >> 4, f = code & 15
 * stand for 2^(e - 15) (1 + f / 16), and for 2^-14 f / 16 where e = 0, times a scale
 * that puts the largest at 1.9375. Both are rounded up or down at random, in proportion
 * to what is left over, so that small changes of every step are kept on average
 * (to nearest, beta2 = 0.999 would hold the second moment where it is). A root that is
 * not zero is not stored as zero. A block that holds a NaN or an infinity
 * gets the scale NaN and codes 0: the moments of the block's elements are NaN from the
 * next step on. First moments of a block whose largest is below 448 * 2^-126 are dropped,
 * and second moments below 2^-126 are zero.
 *
 * The random bits are a hash of `seed`, the step and the element's place in the
 * arena: equal calls give equal bits.
 *
 * The library (libdlrm_narrow.so, with the calls of dlrm_fp4.h) follows the
 * conventions of dlrm_sparse.h: "dev" pointers are device pointers on the current
 * device, the caller owns every buffer, nothing is allocated or kept between calls,
 * calls are asynchronous on `stream` and can be captured into CUDA graphs, a negative
 * return is a dlrm_status_t, and host-side checks run before anything is enqueued.
 */
#ifndef DLRM_OPTIM_H
#define DLRM_OPTIM_H

#include <stdint.h>

#include "dlrm_sparse.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Elements that share a scale; every tensor starts at a multiple of it. */
#define DLRM_ADAMW_BLOCK 256

/*
 * dlrm_adamw_step -- one step over n tensors (n >= 0; with none only the step is counted).
 *   params, grads  host arrays of n dev pointers; elements contiguous, types
 *                  param_dtypes[i] and grad_dtypes[i] (dlrm_table_dtype_t). Pointers of
 *                  empty tensors are not read. No parameter overlaps another one or a
 *                  gradient.
 *   counts         host array, elements of each tensor, >= 0; the arena has fewer than
 *                  2^40 elements.
 *   decays         host array of n weight decays (f32, finite), or NULL for none.
 *   bits           32: m and v are dev f32 arenas, m_scale and v_scale NULL.
 *                  8: m and v are dev byte arenas, m_scale and v_scale dev f32, one
 *                  for each block.
 *   master         dev f32 arena, or NULL. With it, a bf16 parameter's weight is the one
 *                  in the arena, and the parameter gets it rounded to nearest (its old
 *                  value is not read); f32 parameters do not use theirs. Without it a
 *                  bf16 parameter is rounded at random, as the moments are.
 *   step           dev int32[2]: steps taken so far (>= 0), and a word of the call's own, in which
 *                  its CTAs count what they take. t = step[0] + 1; the call writes it back,
 *                  and the word to 0. The word may hold anything above -2^30 before a call:
 *                  both numbers may be set to a count, or counted up or down.
 *   lr             learning rate, finite; lr_dev (dev f32) is taken instead if it is not NULL.
 *   beta1, beta2   in [0, 1); eps: a normal positive number of f32.
 *   grad_scale_dev dev f32 that every gradient is multiplied with (a clipping
 *                  coefficient), or NULL for 1.
 * The arenas and the parameters of one call must not be used by another call at the same
 * time. Pointers are aligned to their elements (the arenas and scales to 16 bytes);
 * parameters and gradients that start on 16 bytes take 128-bit accesses.
 */
DLRM_API int dlrm_adamw_step(int64_t n, void* const* params, const void* const* grads,
                             const int64_t* counts, const int32_t* param_dtypes,
                             const int32_t* grad_dtypes, const float* decays, int bits, void* m,
                             void* v, float* m_scale, float* v_scale, float* master,
                             int32_t* step, double lr, const float* lr_dev, double beta1,
                             double beta2, double eps, const float* grad_scale_dev, uint32_t seed,
                             dlrm_stream_t stream);

/* dlrm_adamw_moments -- the 8-bit moments of `count` arena elements (a multiple of
 * DLRM_ADAMW_BLOCK) as values of dtype: m_out and v_out dev, 32-byte aligned. The first is a code
 * times its scale and the second the square of such a product, each product rounded to f32, as a
 * step reads them; both are then rounded to dtype. */
DLRM_API int dlrm_adamw_moments(int64_t count, const void* m, const void* v, const float* m_scale,
                                const float* v_scale, void* m_out, void* v_out, int dtype,
                                dlrm_stream_t stream);

/* cudaError_t of the last failing CUDA call made by this thread in this library. */
DLRM_API int dlrm_narrow_last_cuda_error(void);

/* Number of kernels this library has launched in this process (all threads). */
DLRM_API int64_t dlrm_narrow_launch_count(void);

#ifdef __cplusplus
}
#endif

#endif /* DLRM_OPTIM_H */
