/*
 * pgemm layer operators -- the matrix products of a model's layers, on the
 * same library and conventions as pgemm.h (device pointers on the current HIP
 * device, an opaque HIP stream, asynchronous calls, 0 or a negative status,
 * -p for a bad argument p, checked before any HIP call).
 *
 * Layout.  Matrices here are ROW-major with rows of `ld` elements: element
 *   (i, j) of X is X.data[i * X.ld + j], ld >= the number of columns.  Weights
 *   alone come in either order (PGEMM_KN: k x n with rows contiguous;
 *   PGEMM_NK: element (i, j) at data[j * ld + i], a weight kept as n x k).
 * Types.  dtype names the element type T of X, W, bias and Z: PGEMM_F32,
 *   PGEMM_F16, PGEMM_BF16.  out_dtype names that of the result (and of a
 *   residual): T or PGEMM_F32.  Sums are fp32 whatever T is; each result is
 *   rounded once.
 * Overlap.  Results must not overlap inputs, except that the residual may be
 *   the result itself (same data and ld).
 * Workspaces are device scratch, 16-byte aligned, owned by the caller; their
 *   content on entry is ignored.  Calls that share one must be ordered.
 * Capture.  Every call only launches kernels (no allocation, memset or
 *   synchronization), so it can be captured into a HIP graph.
 * Determinism.  Identical inputs give identical bits.
 * Sizes are at most 2^31 - 4096 each.  A product of more tiles than one launch takes (2^32 threads: 2^24 tiles
 *   of 64 x 64 to 128 x 128, 2^23 of 256 x 256) is refused as argument 2,
 *   before any launch of its call.
 * Reads.  Rows of a matrix may be read up to 16 bytes past their end where that
 *   is still before the end of its last row (such values reach no result).
 */
#ifndef PGEMM_LAYERS_H
#define PGEMM_LAYERS_H

#include <stddef.h>

#include "pgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { PGEMM_F32 = 0, PGEMM_F16 = 1, PGEMM_BF16 = 2 };
enum { PGEMM_KN = 0, PGEMM_NK = 1 };
/* gelu is z Phi(z); gelu_tanh 0.5 z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3)));
 * silu z / (1 + exp(-z)).  A NaN stays NaN under each. */
enum {
  PGEMM_ACT_NONE = 0,
  PGEMM_ACT_RELU = 1,
  PGEMM_ACT_GELU = 2,
  PGEMM_ACT_GELU_TANH = 3,
  PGEMM_ACT_SILU = 4
};
enum { PGEMM_SOFTMAX = 0, PGEMM_SIGMOID = 1 };

typedef struct {
  void *data;
  long long ld;
} pgemm_rows;

typedef struct {
  const void *data;
  long long ld;
  int order;              /* PGEMM_KN or PGEMM_NK */
  long long stride;       /* elements between experts' weights (0 if there is one) */
} pgemm_weight;

typedef struct {
  int dtype, out_dtype;   /* of T; of the result */
  int act;
} pgemm_kind;

/*
 * Y(m x n) = act(X(m x k) W(k x n) + bias) + residual; Z = X W + bias.
 *   arguments: 1 kind, 2 m, 3 n, 4 k, 5 X, 6 W, 7 bias (n, or NULL),
 *   8 residual (data NULL: none), 9 Z (data NULL: not kept), 10 Y,
 *   11 workspace (or NULL), 12 workspace_bytes, 13 stream.
 * m == 0 or n == 0: nothing is touched.  k == 0: X W is zero, X and W are not
 * read.  The activation sees the fp32 sum; Z is that sum rounded to T.
 * With a workspace of pgemm_linear_workspace bytes the summed index may be
 * shared by several workgroups (few rows, long k); NULL or a smaller one
 * never changes more than the order of the sums.
 */
int pgemm_linear(pgemm_kind kind, int m, int n, int k, pgemm_rows X, pgemm_weight W,
                 const void *bias, pgemm_rows residual, pgemm_rows Z, pgemm_rows Y,
                 void *workspace, size_t workspace_bytes, void *stream);
size_t pgemm_linear_workspace(int dtype, int m, int n, int k);

/*
 * Gradients of pgemm_linear: with dZ = dY * act'(Z),
 *   dX(m x k) = dZ W^T,  dW(k x n) = X^T dZ,  dbias(n) = the sum of dZ's rows
 * (the residual's gradient is dY itself).
 *   arguments: 1 kind, 2 m, 3 n, 4 k, 5 dY (T), 6 Z (T, as pgemm_linear kept
 *   it; data NULL if act is none), 7 X, 8 W, 9 dX (T; data NULL: not wanted),
 *   10 dW (out_dtype, its own order; data NULL: not wanted), 11 dbias
 *   (out_dtype, or NULL), 12 workspace, 13 workspace_bytes, 14 stream.
 * W is read only for dX and X only for dW; m == 0 gives a zero dW and dbias.
 * dZ is rounded to T before the products, so that they run on the matrix
 * cores at T's rate: an error of half a unit of T's last place per element,
 * like that of the results themselves.
 * The workspace must have pgemm_linear_backward_workspace bytes (it holds dZ
 * unless act is none, and partial sums).
 */
int pgemm_linear_backward(pgemm_kind kind, int m, int n, int k, pgemm_rows dY, pgemm_rows Z,
                          pgemm_rows X, pgemm_weight W, pgemm_rows dX, pgemm_weight dW,
                          void *dbias, void *workspace, size_t workspace_bytes, void *stream);
size_t pgemm_linear_backward_workspace(pgemm_kind kind, int m, int n, int k);

/*
 * Routing: the `top` best of `experts` experts for each of m tokens, their
 * weights, and the plan by which expert products read them.
 *   scores: softmax over the experts, or the sigmoid, of the logits (m x
 *   experts, of dtype).  A logit of -inf or of the type's lowest value is
 *   masked, and so is NaN: such an expert has score 0 and is never chosen.
 *   +inf counts as the largest fp32 number.
 *   key: score + bias (fp32, or NULL; a bias that is not finite, or beyond
 *   3e38, masks its expert); with neither bias nor groups the logit
 *   itself (the scores' own order, also where they underflow).  Keys are
 *   compared in 64 bits; ties go to the lower index.
 *   groups: the experts in `groups` equal ranges; only the top_groups with the
 *   largest sum of their two largest keys (of one, if one is left) take part.
 *   weights (m x top, fp32, contiguous): the chosen scores, divided by their
 *   sum if renorm, times scale.  Best key first.
 *   expert_index (m x top, int32): -1 with weight 0 where too few experts are
 *   left (a token whose logits are all masked is not routed at all).
 *   offsets (experts + 1): rows [offsets[e], offsets[e+1]) belong to expert e;
 *   tokens: the token of each row, in token order within an expert (m * top
 *   entries; those behind offsets[experts] are left as they were);
 *   slots (m x top): the row of each choice, -1 for none.
 *   arguments: 1 dtype, 2 m, 3 experts (1..1024), 4 top (1..32, at most the
 *   experts of top_groups groups), 5 score, 6 groups, 7 top_groups, 8 renorm,
 *   9 scale, 10 logits, 11 bias, 12 out, 13 workspace
 *   (pgemm_route_workspace bytes), 14 workspace_bytes, 15 stream.
 */
typedef struct {
  float *weights;
  int *expert_index, *offsets, *tokens, *slots;
} pgemm_route_out;
int pgemm_route(int dtype, int m, int experts, int top, int score, int groups, int top_groups,
                int renorm, float scale, pgemm_rows logits, const float *bias, pgemm_route_out out,
                void *workspace, size_t workspace_bytes, void *stream);
size_t pgemm_route_workspace(int m, int experts, int top);

/*
 * Gradient of the weights with respect to the logits (the choice itself has
 * none; the bias enters only the choice).  Indices outside 0..experts-1 (-1)
 * take no part.  Masked logits get 0.
 *   arguments: 1 dtype, 2 m, 3 experts, 4 top, 5 score, 6 renorm, 7 scale,
 *   8 dweights (m x top), 9 logits, 10 expert_index (m x top), 11 dlogits (of
 *   dtype), 12 stream.
 */
int pgemm_route_backward(int dtype, int m, int experts, int top, int score, int renorm,
                         float scale, const float *dweights, pgemm_rows logits,
                         const int *expert_index, pgemm_rows dlogits, void *stream);

/*
 * The plan of an expert product: row bounds by expert (experts + 1) and the
 * row of X of each row (NULL: the row itself), of which there are x_rows (at
 * least one with tokens, at least as many as rows without).
 */
typedef struct {
  int experts;            /* 1..1024 */
  const int *offsets, *tokens;
  int x_rows;
} pgemm_plan;

/*
 * Each expert's rows through its own weight:
 *   Y[r] = act(X[src(r)] W_e + bias_e), rows r in [offsets[e], offsets[e+1]).
 * src(r) is tokens[r], or r itself if tokens is NULL.  Rows of Y and Z behind
 * offsets[experts] are left as they were.  Row bounds are read on the device
 * and clamped to [0, rows], tokens to [0, x_rows).
 *   arguments: 1 kind, 2 rows (capacity of Y), 3 n, 4 k, 5 plan, 6 X, 7 W,
 *   8 bias (experts x n, contiguous, or NULL), 9 Z, 10 Y, 11 stream.
 */
int pgemm_expert_linear(pgemm_kind kind, int rows, int n, int k, pgemm_plan plan, pgemm_rows X,
                        pgemm_weight W, const void *bias, pgemm_rows Z, pgemm_rows Y,
                        void *stream);

/*
 * Its gradients: dX[r] = dZ[r] W_e^T per row (not summed over a token's rows;
 * pgemm_combine does that), dW_e = sum of X[src(r)]^T dZ[r], dbias_e = sum of
 * dZ[r].  An expert without rows gets zeros.
 *   arguments: 1 kind, 2 rows, 3 n, 4 k, 5 plan, 6 dY, 7 Z, 8 X, 9 W, 10 dX,
 *   11 dW, 12 dbias, 13 workspace, 14 workspace_bytes, 15 stream.
 */
int pgemm_expert_linear_backward(pgemm_kind kind, int rows, int n, int k, pgemm_plan plan,
                                 pgemm_rows dY, pgemm_rows Z, pgemm_rows X, pgemm_weight W,
                                 pgemm_rows dX, pgemm_weight dW, void *dbias, void *workspace,
                                 size_t workspace_bytes, void *stream);
size_t pgemm_expert_linear_backward_workspace(pgemm_kind kind, int rows, int n, int k,
                                              int experts);

/*
 * The experts' rows back to their tokens:
 *   out[t] = residual[t] + sum over j of weights[t, j] * Y[slots[t, j]].
 * A slot outside [0, rows) takes no part.  weights NULL: all 1.
 *   arguments: 1 dtype (of Y, residual and out), 2 m, 3 n, 4 top (1..32), 5 rows,
 *   6 Y, 7 slots (m x top), 8 weights (m x top), 9 residual, 10 out, 11 stream.
 */
int pgemm_combine(int dtype, int m, int n, int top, int rows, pgemm_rows Y, const int *slots,
                  const float *weights, pgemm_rows residual, pgemm_rows out, void *stream);

/*
 * Its gradients: dY[slots[t, j]] = weights[t, j] * dout[t] (rows that no slot
 * names are left as they were), dweights[t, j] = <dout[t], Y[slots[t, j]]> (0
 * without a row).  A row belongs to one (token, choice) at most.
 *   arguments: 1 dtype, 2 m, 3 n, 4 top, 5 rows, 6 dout, 7 Y (data NULL if
 *   dweights is), 8 slots, 9 weights, 10 dY (data NULL: not wanted),
 *   11 dweights (or NULL), 12 stream.
 */
int pgemm_combine_backward(int dtype, int m, int n, int top, int rows, pgemm_rows dout,
                           pgemm_rows Y, const int *slots, const float *weights, pgemm_rows dY,
                           float *dweights, void *stream);

/*
 * For bindings: a call with all its arguments in one struct, in the order and
 * types of the function's parameters (each at its natural alignment, the
 * stream last).  Returns the function's status, or -1 for an unknown op.
 */
enum {
  PGEMM_OP_LINEAR = 0,
  PGEMM_OP_LINEAR_BACKWARD = 1,
  PGEMM_OP_ROUTE = 2,
  PGEMM_OP_ROUTE_BACKWARD = 3,
  PGEMM_OP_EXPERT_LINEAR = 4,
  PGEMM_OP_EXPERT_LINEAR_BACKWARD = 5,
  PGEMM_OP_COMBINE = 6,
  PGEMM_OP_COMBINE_BACKWARD = 7
};
int pgemm_layer_call(int op, const void *args);

#ifdef __cplusplus
}
#endif

#endif /* PGEMM_LAYERS_H */
