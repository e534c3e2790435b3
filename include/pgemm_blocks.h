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
 * is left of the mean (not the difference of two sums), in 64 bits for rows whose
 * squares leave fp32's range.
 */
int pgemm_layer_norm(int dtype, int m, int n, pgemm_rows X, const void *weight, const void *bias,
                     float eps, float *mean, float *rstd, pgemm_rows Y, void *stream);

/*
 * Its gradients: with h = (X - mean) * rstd and g = dY * weight,
 *   dX = rstd * (g - mean of g - h * mean of g h) + residual,
 *   dweight = the sum over rows of dY * h, dbias = the sum of dY's rows.
 *   arguments: 1 kind (dtype of dY, X, weight, residual and dX; out_dtype of dweight
 *   and dbias; act none), 2 m, 3 n, 4 dY, 5 X, 6 mean, 7 rstd (m, fp32, as
 *   pgemm_layer_norm kept them), 8 weight (or NULL: ones), 9 residual (the gradient
 *   that reaches X past the norm; data NULL: none; may be dX itself), 10 dX (data
 *   NULL: not wanted), 11 dweight (or NULL), 12 dbias (or NULL), 13 workspace,
 *   14 workspace_bytes, 15 stream.
 * m == 0 gives a zero dweight and dbias.  X - mean and h are fp32.  The workspace must
 * have pgemm_layer_norm_backward_workspace bytes where dweight or dbias is wanted
 * (partial sums).
 */
int pgemm_layer_norm_backward(pgemm_kind kind, int m, int n, pgemm_rows dY, pgemm_rows X,
                              const float *mean, const float *rstd, const void *weight,
                              pgemm_rows residual, pgemm_rows dX, void *dweight, void *dbias,
                              void *workspace, size_t workspace_bytes, void *stream);
size_t pgemm_layer_norm_backward_workspace(int m, int n);

/* The two weights of a gated product, both in one order and with one ld (their stride
 * is not used), and what belongs to each. */
typedef struct {
  pgemm_weight gate, up;
} pgemm_gate_weights;
typedef struct {
  pgemm_rows gate, up;
} pgemm_gate_rows;
typedef struct {
  void *gate, *up;
} pgemm_gate_bias;

/*
 * Y(m x n) = act(Zg) * Zu with Zg = X(m x k) Wg(k x n) + bias g and Zu = X Wu + bias u,
 * in one kernel.
 *   arguments: 1 kind, 2 m, 3 n (at most 2^30 - 4096), 4 k, 5 X, 6 W, 7 bias (n each,
 *   or NULL), 8 Z (data NULL: not kept), 9 Y, 10 workspace (or NULL),
 *   11 workspace_bytes, 12 stream.
 * Activation and product see the fp32 sums; Z is those rounded to T.  m == 0 or n ==
 * 0: nothing is touched; k == 0: Z is the bias.  With a workspace of
 * pgemm_gated_linear_workspace bytes the summed index may be shared by several
 * workgroups, and operands whose rows are not whole chunks of 16 bytes may be copied
 * into rows that are; NULL or a smaller one never changes more than the order of the
 * sums.
 */
int pgemm_gated_linear(pgemm_kind kind, int m, int n, int k, pgemm_rows X, pgemm_gate_weights W,
                       pgemm_gate_bias bias, pgemm_gate_rows Z, pgemm_rows Y, void *workspace,
                       size_t workspace_bytes, void *stream);
size_t pgemm_gated_linear_workspace(int dtype, int m, int n, int k);

/*
 * Its gradients: with dZg = dY * Zu * act'(Zg) and dZu = dY * act(Zg),
 *   dX = dZg Wg^T + dZu Wu^T (summed in fp32, rounded once), dW = X^T dZ of each,
 *   dbias = the sum of dZ's rows of each.
 *   arguments: 1 kind, 2 m, 3 n (as above), 4 k, 5 dY (T), 6 Z (T, as
 *   pgemm_gated_linear kept them), 7 X, 8 W, 9 dX (T; data NULL: not wanted), 10 dW
 *   (out_dtype, each in its own order; data NULL: not wanted), 11 dbias (out_dtype,
 *   or NULL), 12 workspace, 13 workspace_bytes, 14 stream.
 * W is read only for dX and X only for dW; m == 0 gives zero dW and dbias.  dZ is
 * rounded to T before the products, as pgemm_linear_backward's.
 * Where a kept Z is infinite (fp16 sums beyond 65504), act and act' have their limits,
 * and a product with an exact 0 (of dY, act or act') is 0; a NaN stays one.
 * The workspace must have pgemm_gated_linear_backward_workspace bytes (it holds dZ
 * of both, partial sums, and copies of X and W where n or k is not a multiple of 16
 * bytes' elements).
 */
int pgemm_gated_linear_backward(pgemm_kind kind, int m, int n, int k, pgemm_rows dY,
                                pgemm_gate_rows Z, pgemm_rows X, pgemm_gate_weights W,
                                pgemm_rows dX, pgemm_gate_weights dW, pgemm_gate_bias dbias,
                                void *workspace, size_t workspace_bytes, void *stream);
size_t pgemm_gated_linear_backward_workspace(pgemm_kind kind, int m, int n, int k);

/* 8-bit floating point: e4m3 without infinities (largest 448), e5m2 (largest 57344). */
enum { PGEMM_E4M3 = 0, PGEMM_E5M2 = 1 };
/* Scales of the blocks of 128 columns: of block b of row i (rows == 1) or of rows
 * 128 i .. 128 i + 127 (rows == 128) at data[i * row_stride + b * block_stride]. */
typedef struct {
  float *data;
  long long row_stride, block_stride;
  int rows;
} pgemm_scales;

/*
 * Blocks of 128 columns to 8 bits: with F the type's largest number,
 *   scale = max(the block's largest |x| / F, 2^-126),  Q = x / scale, rounded to
 *   nearest even,
 * so that Q * scale stands for x.  A block that holds an infinity or a NaN gets NaN
 * for its scale and its values.  The last block of a row may have fewer columns.
 *   arguments: 1 dtype (of X), 2 type (of Q), 3 r, 4 c, 5 X (r x c, in either
 *   order: PGEMM_KN with rows contiguous, PGEMM_NK with columns), 6 Q (r x c, rows of
 *   ld bytes), 7 scales (written; strides that do not overlap), 8 stream.
 * r == 0 or c == 0: nothing is touched.
 */
int pgemm_quantize(int dtype, int type, int r, int c, pgemm_weight X, pgemm_rows Q,
                   pgemm_scales scales, void *stream);

/*
 * Product of 8-bit operands with a scale for each block of 128 of the summed index:
 *   Z = sum over blocks B of x_scale[i, B] w_scale[j, B] (sum over k in B of
 *       X[i, k] W[j, k]) + bias,  Y(m x n) = act(Z) + residual.
 *   arguments: 1 kind, 2 m, 3 n, 4 k, 5 X (m x k, rows of ld bytes), 6 x_scales
 *   (rows 1), 7 W (n x k, rows of ld bytes: a weight kept as n x k), 8 w_scales
 *   (rows 1 or 128), 9 bias (n, or NULL), 10 residual (data NULL: none), 11 Z (data
 *   NULL: not kept), 12 Y, 13 workspace (or NULL), 14 workspace_bytes, 15 stream.
 * bias, residual, Z and Y have kind.out_dtype.  The products are exact, the sums of
 * blocks and their scaling fp32; a product of two scales should be a normal fp32
 * number.  For fp32 results the sums within a block are fp32 too; for 16-bit results
 * the matrix cores' 8-bit instructions form them, which add eight products at a
 * time, each cut off 13 bits below the largest (far below a 16-bit rounding).
 * Scales are read only and may have strides of 0.  m == 0 or n == 0: nothing is
 * touched; k == 0: Z is the bias.  With a workspace of pgemm_linear_fp8_workspace
 * bytes the summed index may be shared by several workgroups; NULL or a smaller one
 * never changes more than the order of the sums.
 */
typedef struct {
  int x_type, w_type;     /* PGEMM_E4M3 or PGEMM_E5M2 */
  int out_dtype, act;
} pgemm_fp8_kind;
int pgemm_linear_fp8(pgemm_fp8_kind kind, int m, int n, int k, pgemm_rows X, pgemm_scales x_scales,
                     pgemm_rows W, pgemm_scales w_scales, const void *bias, pgemm_rows residual,
                     pgemm_rows Z, pgemm_rows Y, void *workspace, size_t workspace_bytes,
                     void *stream);
size_t pgemm_linear_fp8_workspace(int m, int n, int k);

/*
 * For bindings: a call with all its arguments in one struct, in the order and
 * types of the function's parameters (each at its natural alignment, the
 * stream last).  Returns the function's status, or -1 for an unknown op.
 */
enum {
  PGEMM_OP_LAYER_NORM = 0,
  PGEMM_OP_LAYER_NORM_BACKWARD = 1,
  PGEMM_OP_QUANTIZE = 2,
  PGEMM_OP_LINEAR_FP8 = 3,
  PGEMM_OP_GATED_LINEAR = 4,
  PGEMM_OP_GATED_LINEAR_BACKWARD = 5
};
int pgemm_block_call(int op, const void *args);

#ifdef __cplusplus
}
#endif

#endif /* PGEMM_BLOCKS_H */
