// C ABI of the block operators: argument checks, the choice of kernels and
// their launches.  Declarations and the contract are in pgemm_blocks.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../layers/plan.hpp"
#include "ops.hpp"
#include "pgemm_blocks.h"

namespace pgemm {
namespace blocks {
namespace {

using namespace layers;

int status(hipError_t e) { return e == hipSuccess ? PGEMM_OK : PGEMM_EHIP; }

// Workgroups along the rows of a norm's gradients.  Each writes its column sums
// (8 n bytes) once, so that it should have a few rows; and each thread adds its
// rows one after the other, so that it should not have too many (as far as a launch
// of norm_sums_kernel goes: 2^24 workgroups).
int norm_groups(int m, int n) {
  const long long few = ceil_div(m, 4), long_sum = ceil_div(m, 1024);
  long long g = few < 2 * kUnits ? few : 2 * kUnits;
  if (g < long_sum) g = long_sum;
  const long long most = (1LL << 23) / ceil_div(n, 512);
  if (g > most) g = most;
  return g < 1 ? 1 : (int)g;
}

bool fp8_ok(int type) { return type == PGEMM_E4M3 || type == PGEMM_E5M2; }

bool scales_ok(const pgemm_scales& s, bool need) {
  if (s.rows != 1 && s.rows != kScaleBlock) return false;
  return vector_ok(s.data, 4, need) && s.row_stride >= 0 && s.block_stride >= 0;
}

}  // namespace
}  // namespace blocks
}  // namespace pgemm

using namespace pgemm::layers;
using namespace pgemm::blocks;

extern "C" {

int pgemm_layer_norm(int dtype, int m, int n, pgemm_rows X, const void* weight, const void* bias,
                     float eps, float* mean, float* rstd, pgemm_rows Y, void* stream) {
  if (!known(dtype)) return -1;
  if (!size_ok(m)) return -2;
  if (!size_ok(n)) return -3;
  const bool touch = m > 0 && n > 0;
  const int size = size_of(dtype);
  if (!rows_ok(X, n, size, touch)) return -4;
  if (!vector_ok(weight, size, false)) return -5;
  if (!vector_ok(bias, size, false)) return -6;
  if (!(eps >= 0.0f)) return -7;
  if (!vector_ok(mean, 4, false)) return -8;
  if (!vector_ok(rstd, 4, false)) return -9;
  if (!rows_ok(Y, n, size, touch)) return -10;
  if (!touch) return PGEMM_OK;
  NormArgs a{};
  a.X = X.data;
  a.W = weight;
  a.B = bias;
  a.Y = Y.data;
  a.mean = mean;
  a.rstd = rstd;
  a.ldx = X.ld;
  a.ldy = Y.ld;
  a.m = m;
  a.n = n;
  a.eps = eps;
  return status(norm_ops(dtype).norm(a, static_cast<hipStream_t>(stream)));
}

int pgemm_layer_norm_backward(int dtype, int out_dtype, int m, int n, pgemm_rows dY, pgemm_rows X,
                              const float* mean, const float* rstd, const void* weight,
                              pgemm_rows residual, pgemm_rows dX, void* dweight, void* dbias,
                              void* workspace, size_t workspace_bytes, void* stream) {
  if (!known(dtype)) return -1;
  if (out_dtype != dtype && out_dtype != PGEMM_F32) return -2;
  if (!size_ok(m)) return -3;
  if (!size_ok(n)) return -4;
  const bool touch = m > 0 && n > 0, sums = dweight != nullptr || dbias != nullptr;
  const int size = size_of(dtype), osize = size_of(out_dtype);
  if (!rows_ok(dY, n, size, touch)) return -5;
  if (!rows_ok(X, n, size, touch)) return -6;
  if (!vector_ok(mean, 4, touch)) return -7;
  if (!vector_ok(rstd, 4, touch)) return -8;
  if (!vector_ok(weight, size, false)) return -9;
  if (!rows_ok(residual, n, size, false)) return -10;
  if (!rows_ok(dX, n, size, false)) return -11;
  if (!vector_ok(dweight, osize, false)) return -12;
  if (!vector_ok(dbias, osize, false)) return -13;
  if (sums && n > 0) {
    if (workspace == nullptr || !aligned_to(workspace, 16)) return -14;
    if (workspace_bytes < pgemm_layer_norm_backward_workspace(m, n)) return -15;
  }
  if (n == 0) return PGEMM_OK;
  const NormOps& ops = norm_ops(dtype);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  NormBackArgs a{};
  a.dY = dY.data;
  a.X = X.data;
  a.mean = mean;
  a.rstd = rstd;
  a.W = weight;
  a.R = residual.data;
  a.dX = dX.data;
  a.ldy = dY.ld;
  a.ldx = X.ld;
  a.ldr = residual.ld;
  a.ldd = dX.ld;
  a.m = m;
  a.n = n;
  a.groups = norm_groups(m, n);
  float* partial = sums ? static_cast<float*>(workspace) : nullptr;
  if (dX.data != nullptr && m > 0) {
    if (n <= kSumMost) a.partial = partial;
    const hipError_t e = ops.norm_back(a, s);
    if (e != hipSuccess) return PGEMM_EHIP;
  }
  if (!sums) return PGEMM_OK;
  if (a.partial == nullptr) {      // (no rows: zeros)
    a.partial = partial;
    const hipError_t e = ops.norm_sums(a, s);
    if (e != hipSuccess) return PGEMM_EHIP;
  }
  const NormColumnArgs c = {partial, dweight, dbias, n, a.groups, out_dtype == PGEMM_F32};
  return status(ops.norm_columns(c, s));
}

size_t pgemm_layer_norm_backward_workspace(int m, int n) {
  if (m < 0 || n <= 0) return 0;
  return align256((size_t)norm_groups(m, n) * 2 * (size_t)n * 4);
}

int pgemm_quantize(int dtype, int type, int r, int c, pgemm_weight X, pgemm_rows Q,
                   pgemm_scales scales, void* stream) {
  if (!known(dtype)) return -1;
  if (!fp8_ok(type)) return -2;
  if (!size_ok(r)) return -3;
  if (!size_ok(c)) return -4;
  const bool touch = r > 0 && c > 0;
  if (!weight_ok(X, r, c, size_of(dtype), touch, 1)) return -5;
  if (!rows_ok(Q, c, 1, touch)) return -6;
  if (!scales_ok(scales, touch)) return -7;
  if (!touch) return PGEMM_OK;
  const long long blocks = ceil_div(c, kScaleBlock), high = ceil_div(r, scales.rows);
  const bool apart = (blocks == 1 || scales.block_stride >= 1) && (high == 1 || scales.row_stride >= 1) &&
                     (blocks == 1 || high == 1 || scales.row_stride >= blocks * scales.block_stride ||
                      scales.block_stride >= high * scales.row_stride);
  if (!apart) return -7;
  QuantizeArgs a{};
  a.X = X.data;
  a.Q = static_cast<uint8_t*>(Q.data);
  a.scales = scales.data;
  a.ldx = X.ld;
  a.ldq = Q.ld;
  a.srow = scales.row_stride;
  a.sblock = scales.block_stride;
  a.r = r;
  a.c = c;
  a.blocks = (int)blocks;
  a.together = scales.rows == kScaleBlock;
  return status(quantize_op(a, dtype, type, X.order == PGEMM_NK, static_cast<hipStream_t>(stream)));
}

int pgemm_linear_fp8(pgemm_fp8_kind kind, int m, int n, int k, pgemm_rows X, pgemm_scales x_scales,
                     pgemm_rows W, pgemm_scales w_scales, const void* bias, pgemm_rows residual,
                     pgemm_rows Z, pgemm_rows Y, void* workspace, size_t workspace_bytes,
                     void* stream) {
  if (!fp8_ok(kind.x_type) || !fp8_ok(kind.w_type) ||
      !kind_ok({kind.out_dtype, kind.out_dtype, kind.act}))
    return -1;
  if (!size_ok(m)) return -2;
  if (!size_ok(n)) return -3;
  if (!size_ok(k)) return -4;
  const bool touch = m > 0 && n > 0, read = touch && k > 0;
  const int osize = size_of(kind.out_dtype);
  if (!rows_ok(X, k, 1, read)) return -5;
  if (!scales_ok(x_scales, read) || x_scales.rows != 1) return -6;
  if (!rows_ok(W, k, 1, read)) return -7;
  if (!scales_ok(w_scales, read)) return -8;
  if (!vector_ok(bias, osize, false)) return -9;
  if (!rows_ok(residual, n, osize, false)) return -10;
  if (!rows_ok(Z, n, osize, false)) return -11;
  if (!rows_ok(Y, n, osize, touch)) return -12;
  if (workspace != nullptr && !aligned_to(workspace, 16)) return -13;
  if (!touch) return PGEMM_OK;
  Prod8Args args{};
  ProdArgs& a = args.p;
  a.A = X.data;
  a.lda = X.ld;
  a.B = W.data;
  a.ldb = W.ld;
  a.D = Y.data;
  a.ldd = Y.ld;
  a.M = m;
  a.N = n;
  a.K = k;
  a.bias = bias;
  a.R = residual.data;
  a.ldr = residual.ld;
  a.Z = Z.data;
  a.ldz = Z.ld;
  a.act = kind.act;
  a.out32 = kind.out_dtype == PGEMM_F32;
  args.type = kind.out_dtype;
  args.sx = x_scales.data;
  args.sx_row = x_scales.row_stride;
  args.sx_block = x_scales.block_stride;
  args.sw = w_scales.data;
  args.sw_row = w_scales.row_stride;
  args.sw_block = w_scales.block_stride;
  args.w_shift = w_scales.rows == 1 ? 0 : 7;
  const bool direct = operand_loading(X.data, X.ld, 1, k, 0) == kDirect &&
                      operand_loading(W.data, W.ld, 1, k, 0) == kDirect;
  const bool wide = kind.out_dtype == PGEMM_F32;
  // (kThrough: no tiles of 256 x 256)
  const Plan plan = plan_product(1, kInner, kDense, m, 0, n, k, direct && !wide ? kDirect : kThrough,
                                 workspace == nullptr ? 0 : workspace_bytes, false);
  if (plan.kernel < 0) return -2;
  a.splits = plan.splits;
  a.k_split = plan.k_split;
  a.partial = static_cast<float*>(workspace);
  set_tiles(&a, plan.kernel, kDense, m);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const Prod8 prod = kind.x_type == PGEMM_E4M3 ? (wide ? prod8_e4m3_wide : prod8_e4m3)
                                               : (wide ? prod8_e5m2_wide : prod8_e5m2);
  return status(prod(args, kind.w_type, plan.kernel, direct, s));
}

size_t pgemm_linear_fp8_workspace(int m, int n, int k) {
  if (m <= 0 || n <= 0 || k <= 0) return 0;
  return split_bytes(1, kInner, kDense, m, 1, n, k);
}

namespace {

struct LayerNormCall {
  int dtype, m, n;
  pgemm_rows X;
  const void* weight;
  const void* bias;
  float eps;
  float* mean;
  float* rstd;
  pgemm_rows Y;
  void* stream;
};
struct LayerNormBackwardCall {
  int dtype, out_dtype, m, n;
  pgemm_rows dY, X;
  const float* mean;
  const float* rstd;
  const void* weight;
  pgemm_rows residual, dX;
  void* dweight;
  void* dbias;
  void* workspace;
  size_t workspace_bytes;
  void* stream;
};

struct QuantizeCall {
  int dtype, type, r, c;
  pgemm_weight X;
  pgemm_rows Q;
  pgemm_scales scales;
  void* stream;
};
struct LinearFp8Call {
  pgemm_fp8_kind kind;
  int m, n, k;
  pgemm_rows X;
  pgemm_scales x_scales;
  pgemm_rows W;
  pgemm_scales w_scales;
  const void* bias;
  pgemm_rows residual, Z, Y;
  void* workspace;
  size_t workspace_bytes;
  void* stream;
};

}  // namespace

int pgemm_block_call(int op, const void* args) {
  if (args == nullptr) return -2;
  switch (op) {
    case PGEMM_OP_LAYER_NORM: {
      const LayerNormCall& c = *static_cast<const LayerNormCall*>(args);
      return pgemm_layer_norm(c.dtype, c.m, c.n, c.X, c.weight, c.bias, c.eps, c.mean, c.rstd, c.Y,
                              c.stream);
    }
    case PGEMM_OP_LAYER_NORM_BACKWARD: {
      const LayerNormBackwardCall& c = *static_cast<const LayerNormBackwardCall*>(args);
      return pgemm_layer_norm_backward(c.dtype, c.out_dtype, c.m, c.n, c.dY, c.X, c.mean, c.rstd,
                                       c.weight, c.residual, c.dX, c.dweight, c.dbias, c.workspace,
                                       c.workspace_bytes, c.stream);
    }
    case PGEMM_OP_QUANTIZE: {
      const QuantizeCall& c = *static_cast<const QuantizeCall*>(args);
      return pgemm_quantize(c.dtype, c.type, c.r, c.c, c.X, c.Q, c.scales, c.stream);
    }
    case PGEMM_OP_LINEAR_FP8: {
      const LinearFp8Call& c = *static_cast<const LinearFp8Call*>(args);
      return pgemm_linear_fp8(c.kind, c.m, c.n, c.k, c.X, c.x_scales, c.W, c.w_scales, c.bias,
                              c.residual, c.Z, c.Y, c.workspace, c.workspace_bytes, c.stream);
    }
    default: return -1;
  }
}

}  // extern "C"
