/*
 * pgemm block operators -- what stands around the products of a model's
 * feed-forward block, on the same library and with the conventions of
 * pgemm_layers.h (row-major matrices, weights in either order, types, overlap,
 * workspaces, capture, determinism, sizes, statuses).
 */
#ifndef PGEMM_BLOCKS_H
#define PGEMM_BLOCKS_H

#include <stddef.h>

#include "pgemm_layers.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Layer norm of m rows of n features:
 *   mean = the row's mean, rstd = 1 / sqrt(its variance + eps),
 *   Y = (X - mean) * rstd * weight + bias.
 *   arguments: 1 dtype (of X, weight, bias and Y), 2 m, 3 n, 4 X, 5 weight (n, or
 *   NULL: ones), 6 bias (n, or NULL: zeros), 7 eps (at least 0), 8 mean (m, fp32,
 *   or NULL: not kept), 9 rstd (the same), 10 Y, 11 stream.
 * m == 0 or n == 0: nothing is touched.  The variance is the mean square of what
 * is left of the mean (not the difference of two sums).
 */
int pgemm_layer_norm(int dtype, int m, int n, pgemm_rows X, const void *weight, const void *bias,
                     float eps, float *mean, float *rstd, pgemm_rows Y, void *stream);

/*
 * Its gradients: with h = (X - mean) * rstd and g = dY * weight,
 *   dX = rstd * (g - mean of g - h * mean of g h) + residual,
 *   dweight = the sum over rows of dY * h, dbias = the sum of dY's rows.
 *   arguments: 1 dtype (of dY, X, weight, residual and dX), 2 out_dtype (of dweight
 *   and dbias: dtype or PGEMM_F32), 3 m, 4 n, 5 dY, 6 X, 7 mean, 8 rstd (m, fp32,
 *   as pgemm_layer_norm kept them), 9 weight (or NULL: ones), 10 residual (the
 *   gradient that reaches X past the norm; data NULL: none; may be dX itself),
 *   11 dX (data NULL: not wanted), 12 dweight (or NULL), 13 dbias (or NULL),
 *   14 workspace, 15 workspace_bytes, 16 stream.
 * m == 0 gives a zero dweight and dbias.  The workspace must have
 * pgemm_layer_norm_backward_workspace bytes where dweight or dbias is wanted
 * (partial sums).
 */
int pgemm_layer_norm_backward(int dtype, int out_dtype, int m, int n, pgemm_rows dY, pgemm_rows X,
                              const float *mean, const float *rstd, const void *weight,
                              pgemm_rows residual, pgemm_rows dX, void *dweight, void *dbias,
                              void *workspace, size_t workspace_bytes, void *stream);
size_t pgemm_layer_norm_backward_workspace(int m, int n);

/*
 * For bindings: a call with all its arguments in one struct, in the order and
 * types of the function's parameters (each at its natural alignment, the
 * stream last).  Returns the function's status, or -1 for an unknown op.
 */
enum {
  PGEMM_OP_LAYER_NORM = 0,
  PGEMM_OP_LAYER_NORM_BACKWARD = 1
};
int pgemm_block_call(int op, const void *args);

#ifdef __cplusplus
}
#endif

#endif /* PGEMM_BLOCKS_H */
