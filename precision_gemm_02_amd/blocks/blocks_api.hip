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
    default: return -1;
  }
}

}  // extern "C"
