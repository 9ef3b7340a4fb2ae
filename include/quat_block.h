/*
 * quat_block.h -- C ABI of the operators of a residual block around the sequence
 * mixer: layer norm over a row, and dropout from a counter-based generator.
 *
 * Conventions are those of quat_cumprod.h: plain device pointers on the current
 * device, caller-owned; `stream` is a cudaStream_t; every call validates its
 * arguments, enqueues its work on `stream` and returns; scratch is the library's
 * workspace of the (device, stream); outputs must not overlap inputs.  Status
 * codes are quat_cumprod.h's.  Pointers need the alignment of their elements
 * only; 16-byte alignment (of pointers, rows and row distances) is faster.
 *
 * Element types: QS_F32 or QS_BF16 (quat_mixer.h).  Sums, means and weights are
 * fp32; an output in bfloat16 is rounded to nearest even once, when stored.
 */
#ifndef QUAT_BLOCK_H
#define QUAT_BLOCK_H

#include <stdint.h>

#include "quat_cumprod.h"
#include "quat_mixer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Longest row of quat_layer_norm_*. */
#define QS_NORM_MAX_D 16384

/*
 * Layer norm of R rows of D values, row r at x + r * ld:
 *
 *     y = (x - mean(x)) * (mean((x - mean(x))^2) + eps)^(-1/2) * w + b
 *
 * with w, b fp32 [D] (NULL: 1 and 0).  y is contiguous [R, D].  ld >= 0 (0: one
 * row R times).  eps >= 0; with eps = 0 a row of equal values gives NaN.
 */
int quat_layer_norm_fwd(int dtype, float eps, const void *x, const float *w, const float *b, void *y,
                        int64_t R, int64_t D, int64_t ld, void *stream);

/*
 * Its vector-Jacobian product for a cotangent d_y (contiguous [R, D]), recomputed
 * from x: d_x (contiguous, `dtype`) and, where not NULL, d_w and d_b (fp32 [D], the
 * sums over all rows, in a fixed order; zeros without rows).
 */
int quat_layer_norm_bwd(int dtype, float eps, const void *x, const float *w, const void *d_y, void *d_x,
                        float *d_w, float *d_b, int64_t R, int64_t D, int64_t ld, void *stream);

/*
 * Dropout of n contiguous values, added on a residual (NULL: none):
 *
 *     y_i = residual_i + (word_i >= floor(p 2^32) ? x_i / (1 - p) : 0)
 *
 * word_i is word i % 4 of Philox4x32-10 (Salmon, Moraes, Dror, Shaw: Parallel random
 * numbers: as easy as 1, 2, 3, 2011) for the counter (i / 4, offset), 64 bits each, low
 * halves first, under the 64-bit key `seed`.  key: {seed, offset} in device memory,
 * read when the work runs: a captured graph draws anew when the program counts the
 * offset up between replays.  0 <= p <= 1; with p = 1 every value is dropped.
 */
int quat_dropout_fwd(int dtype, double p, const int64_t *key, const void *x, const void *residual, void *y,
                     int64_t n, void *stream);

/* Its vector-Jacobian product: d_x_i = word_i >= floor(p 2^32) ? d_y_i / (1 - p) : 0, the same words again. */
int quat_dropout_bwd(int dtype, double p, const int64_t *key, const void *d_y, void *d_x, int64_t n, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QUAT_BLOCK_H */
