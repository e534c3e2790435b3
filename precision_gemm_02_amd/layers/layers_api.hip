// C ABI of the layer operators: argument checks, the choice of kernels and
// their launches.  Declarations and the contract are in pgemm_layers.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.hpp"
#include "pgemm_layers.h"
#include "plan.hpp"

namespace pgemm {
namespace layers {
namespace {

// The parts of a backward call's workspace: dZ, then partial sums (column sums
// of the bias gradient, then the products' splits, one after the other in
// stream order).
struct BackSpace {
  size_t dz = 0, rest = 0;
  long long ldz = 0;
  int chunks = 1;
  size_t total() const { return dz + rest; }
};

BackSpace back_space(const pgemm_kind& kind, int rows, int n, int k, int groups, bool grouped) {
  BackSpace b;
  const int size = size_of(kind.dtype);
  b.ldz = round_up(n, 8);
  if (kind.act != PGEMM_ACT_NONE) b.dz = align256((size_t)rows * (size_t)b.ldz * (size_t)size);
  if (rows < 1) rows = 1;
  b.chunks = slope_chunks(rows, groups, n);
  b.rest = (size_t)groups * (size_t)b.chunks * (size_t)n * 4;
  const int r = (int)rows, mode = grouped ? kSums : kDense;
  const size_t parts[3] = {grouped ? 0 : split_bytes(size, kInner, kDense, r, 1, k, n),
                           split_bytes(size, kOuter, mode, k, groups, n, r),
                           split_bytes(size, kOuter, mode, n, groups, k, r)};
  for (const size_t x : parts)
    if (x > b.rest) b.rest = x;
  b.rest = align256(b.rest);
  return b;
}

// dZ (or dY itself) and the bias gradient, then the two products.
struct BackArgs {
  pgemm_kind kind;
  int rows, n, k, groups;
  const int* offsets;
  const int* tokens;
  int x_rows;
  pgemm_rows dY, Z, X, dX;
  pgemm_weight W, dW;
  void* dbias;
};

// All of the call is planned before any of it is launched.
int run_backward(const BackArgs& b, void* ws, const BackSpace& space, hipStream_t s) {
  const TypeOps& ops = ops_of(b.kind.dtype);
  const bool grouped = b.offsets != nullptr;
  char* base = static_cast<char*>(ws);
  void* rest = base + space.dz;
  const void* dz = b.dY.data;
  long long ldz = b.dY.ld;
  const bool act = b.kind.act != PGEMM_ACT_NONE;
  const bool slope = (act && (b.dX.data != nullptr || b.dW.data != nullptr)) || b.dbias != nullptr;
  const bool out32 = b.kind.out_dtype == PGEMM_F32;
  if (slope && act) {
    dz = base;
    ldz = space.ldz;
  }
  const bool want_dx = b.dX.data != nullptr && b.rows > 0 && b.k > 0;
  const bool want_dw = b.dW.data != nullptr && b.k > 0 && b.n > 0;
  Product dx{}, dw{};
  if (want_dx) {
    ProdArgs& a = dx.a;
    a.A = dz;
    a.lda = ldz;
    a.B = b.W.data;
    a.ldb = b.W.ld;
    a.strideB = b.W.stride;
    a.D = b.dX.data;
    a.ldd = b.dX.ld;
    a.out32 = b.kind.dtype == PGEMM_F32;
    a.M = b.rows;
    a.N = b.k;
    a.K = b.n;
    a.offsets = b.offsets;
    a.groups = grouped ? b.groups : 0;
    a.rows = b.rows;
    dx.dtype = b.kind.dtype;
    dx.la = kInner;
    dx.lb = b.W.order == PGEMM_KN ? kInner : kOuter;
    dx.mode = grouped ? kRows : kDense;
    if (!plan_call(&dx, b.rows, rest, space.rest)) return -2;
  }
  if (want_dw) {
    ProdArgs& a = dw.a;
    const bool kn = b.dW.order == PGEMM_KN;
    a.A = kn ? b.X.data : dz;
    a.lda = kn ? b.X.ld : ldz;
    a.B = kn ? dz : b.X.data;
    a.ldb = kn ? ldz : b.X.ld;
    a.gather = kn ? b.tokens : nullptr;
    a.gather_b = kn ? nullptr : b.tokens;
    a.gather_rows = b.x_rows;
    a.D = const_cast<void*>(b.dW.data);
    a.ldd = b.dW.ld;
    a.strideD = b.dW.stride;
    a.out32 = out32;
    a.M = kn ? b.k : b.n;
    a.N = kn ? b.n : b.k;
    a.K = b.rows;
    a.offsets = b.offsets;
    a.groups = grouped ? b.groups : 0;
    a.rows = b.rows;
    dw.dtype = b.kind.dtype;
    dw.la = dw.lb = kOuter;
    dw.mode = grouped ? kSums : kDense;
    if (!plan_call(&dw, a.M, rest, space.rest)) return -2;
  }
  if (slope) {
    SlopeArgs a{};
    a.dY = b.dY.data;
    a.ldy = b.dY.ld;
    if (act) {
      a.Z = b.Z.data;
      a.ldz = b.Z.ld;
      a.dZ = base;
      a.ldd = space.ldz;
    }
    a.n = b.n;
    a.act = b.kind.act;
    a.offsets = b.offsets;
    a.rows = b.rows;
    a.chunks = space.chunks;
    a.tpr = threads_per_row(b.n, 64);
    a.partial = b.dbias != nullptr ? static_cast<float*>(rest) : nullptr;
    a.sums32 = b.dbias != nullptr && out32;
    if (ops.slope(a, b.groups, s) != hipSuccess) return PGEMM_EHIP;
    if (b.dbias != nullptr &&
        ops.column_sum(a.partial, b.dbias, b.n, b.groups, a.chunks, out32, s) != hipSuccess)
      return PGEMM_EHIP;
  }
  if (want_dx) {
    const int st = launch_product(dx, s);
    if (st != PGEMM_OK) return st;
  }
  return want_dw ? launch_product(dw, s) : PGEMM_OK;
}

}  // namespace
}  // namespace layers
}  // namespace pgemm

using namespace pgemm::layers;

extern "C" {

int pgemm_linear(pgemm_kind kind, int m, int n, int k, pgemm_rows X, pgemm_weight W,
                 const void* bias, pgemm_rows residual, pgemm_rows Z, pgemm_rows Y,
                 void* workspace, size_t workspace_bytes, void* stream) {
  if (!kind_ok(kind)) return -1;
  if (!size_ok(m)) return -2;
  if (!size_ok(n)) return -3;
  if (!size_ok(k)) return -4;
  const bool touch = m > 0 && n > 0, read = touch && k > 0;
  const int size = size_of(kind.dtype), osize = size_of(kind.out_dtype);
  if (!rows_ok(X, k, size, read)) return -5;
  if (!weight_ok(W, k, n, size, read, 1)) return -6;
  if (!vector_ok(bias, size, false)) return -7;
  if (!rows_ok(residual, n, osize, false)) return -8;
  if (!rows_ok(Z, n, size, false)) return -9;
  if (!rows_ok(Y, n, osize, touch)) return -10;
  if (workspace != nullptr && !aligned_to(workspace, 16)) return -11;
  if (!touch) return PGEMM_OK;
  Product p{};
  ProdArgs& a = p.a;
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
  p.dtype = kind.dtype;
  p.la = kInner;
  p.lb = W.order == PGEMM_KN ? kOuter : kInner;
  p.mode = kDense;
  if (!plan_call(&p, m, workspace, workspace_bytes)) return -2;
  return launch_product(p, static_cast<hipStream_t>(stream));
}

size_t pgemm_linear_workspace(int dtype, int m, int n, int k) {
  if (!known(dtype) || m <= 0 || n <= 0 || k <= 0) return 0;
  return split_bytes(size_of(dtype), kInner, kDense, m, 1, n, k);
}

int pgemm_linear_backward(pgemm_kind kind, int m, int n, int k, pgemm_rows dY, pgemm_rows Z,
                          pgemm_rows X, pgemm_weight W, pgemm_rows dX, pgemm_weight dW,
                          void* dbias, void* workspace, size_t workspace_bytes, void* stream) {
  if (!kind_ok(kind)) return -1;
  if (!size_ok(m)) return -2;
  if (!size_ok(n)) return -3;
  if (!size_ok(k)) return -4;
  const int size = size_of(kind.dtype), osize = size_of(kind.out_dtype);
  const bool read = m > 0 && n > 0;
  if (!rows_ok(dY, n, size, read)) return -5;
  if (!rows_ok(Z, n, size, read && kind.act != PGEMM_ACT_NONE)) return -6;
  if (!rows_ok(X, k, size, read && k > 0 && dW.data != nullptr)) return -7;
  if (!weight_ok(W, k, n, size, read && k > 0 && dX.data != nullptr, 1)) return -8;
  if (!rows_ok(dX, k, size, false)) return -9;
  if (!weight_ok(dW, k, n, osize, false, 1)) return -10;
  if (!vector_ok(dbias, osize, false)) return -11;
  const BackSpace space = back_space(kind, m, n, k, 1, false);
  if (space.total() > 0 && (workspace == nullptr || !aligned_to(workspace, 16))) return -12;
  if (workspace_bytes < space.total()) return -13;
  if (n == 0) {
    // no columns: dX is a sum of nothing
    if (dX.data == nullptr || m == 0 || k == 0) return PGEMM_OK;
  }
  BackArgs b{kind, m, n, k, 1, nullptr, nullptr, 0, dY, Z, X, dX, W, dW, n > 0 ? dbias : nullptr};
  if (n == 0) b.kind.act = PGEMM_ACT_NONE;
  return run_backward(b, workspace, space, static_cast<hipStream_t>(stream));
}

size_t pgemm_linear_backward_workspace(pgemm_kind kind, int m, int n, int k) {
  if (!kind_ok(kind) || m < 0 || n <= 0 || k < 0) return 0;
  return back_space(kind, m, n, k, 1, false).total();
}

int pgemm_route(int dtype, int m, int experts, int top, int score, int groups, int top_groups,
                int renorm, float scale, pgemm_rows logits, const float* bias, pgemm_route_out out,
                void* workspace, size_t workspace_bytes, void* stream) {
  if (!known(dtype)) return -1;
  if (m < 0 || m > (1 << 30) / kMaxTop) return -2;
  if (experts < 1 || experts > kMaxExperts) return -3;
  if (top < 1 || top > kMaxTop || top > experts) return -4;
  if (score != PGEMM_SOFTMAX && score != PGEMM_SIGMOID) return -5;
  if (groups < 1 || groups > 64 || experts % groups != 0) return -6;
  if (top_groups < 1 || top_groups > groups) return -7;
  if (top > experts / groups * top_groups) return -4;
  if (!rows_ok(logits, experts, size_of(dtype), m > 0)) return -10;
  if (!vector_ok(bias, 4, false)) return -11;
  if (!vector_ok(out.offsets, 4, true)) return -12;
  if (!vector_ok(out.weights, 4, m > 0) || !vector_ok(out.expert_index, 4, m > 0) ||
      !vector_ok(out.tokens, 4, m > 0) || !vector_ok(out.slots, 4, m > 0))
    return -12;
  const size_t need = pgemm_route_workspace(m, experts, top);
  if (need > 0 && (workspace == nullptr || !aligned_to(workspace, 16))) return -13;
  if (workspace_bytes < need) return -14;
  RouteArgs a{};
  a.logits = logits.data;
  a.ld = logits.ld;
  a.bias = bias;
  a.m = m;
  a.experts = experts;
  a.top = top;
  a.score = score;
  a.groups = groups;
  a.top_groups = top_groups;
  a.renorm = renorm != 0;
  a.scale = scale;
  a.weights = out.weights;
  a.index = out.expert_index;
  a.offsets = out.offsets;
  a.tokens = out.tokens;
  a.slots = out.slots;
  a.blocks = m > 0 ? (int)ceil_div(m, kRouteTokens) : 1;
  a.counts = static_cast<int*>(workspace);
  a.totals = a.counts == nullptr ? nullptr : a.counts + (size_t)experts * (size_t)a.blocks;
  return ops_of(dtype).route(a, static_cast<hipStream_t>(stream)) == hipSuccess ? PGEMM_OK
                                                                             : PGEMM_EHIP;
}

size_t pgemm_route_workspace(int m, int experts, int top) {
  (void)top;
  if (m <= kRouteTokens || experts < 1) return 0;
  return align256((size_t)experts * (size_t)(ceil_div(m, kRouteTokens) + 1) * 4);
}

int pgemm_route_backward(int dtype, int m, int experts, int top, int score, int renorm,
                         float scale, const float* dweights, pgemm_rows logits,
                         const int* expert_index, pgemm_rows dlogits, void* stream) {
  if (!known(dtype)) return -1;
  if (m < 0 || m > (1 << 30) / kMaxTop) return -2;
  if (experts < 1 || experts > kMaxExperts) return -3;
  if (top < 1 || top > kMaxTop) return -4;
  if (score != PGEMM_SOFTMAX && score != PGEMM_SIGMOID) return -5;
  if (!vector_ok(dweights, 4, m > 0)) return -8;
  if (!rows_ok(logits, experts, size_of(dtype), m > 0)) return -9;
  if (!vector_ok(expert_index, 4, m > 0)) return -10;
  if (!rows_ok(dlogits, experts, size_of(dtype), m > 0)) return -11;
  if (m == 0) return PGEMM_OK;
  RouteBackArgs a{};
  a.dweights = dweights;
  a.logits = logits.data;
  a.ld = logits.ld;
  a.index = expert_index;
  a.dlogits = dlogits.data;
  a.ldd = dlogits.ld;
  a.m = m;
  a.experts = experts;
  a.top = top;
  a.score = score;
  a.renorm = renorm != 0;
  a.scale = scale;
  return ops_of(dtype).route_back(a, static_cast<hipStream_t>(stream)) == hipSuccess ? PGEMM_OK
                                                                                  : PGEMM_EHIP;
}

int pgemm_expert_linear(pgemm_kind kind, int rows, int n, int k, pgemm_plan plan, pgemm_rows X,
                        pgemm_weight W, const void* bias, pgemm_rows Z, pgemm_rows Y,
                        void* stream) {
  if (!kind_ok(kind)) return -1;
  if (!size_ok(rows)) return -2;
  if (!size_ok(n)) return -3;
  if (!size_ok(k)) return -4;
  const bool touch = rows > 0 && n > 0, read = touch && k > 0;
  const int size = size_of(kind.dtype), osize = size_of(kind.out_dtype);
  if (!plan_ok(plan, rows, touch)) return -5;
  if (!rows_ok(X, k, size, read)) return -6;
  if (!weight_ok(W, k, n, size, read, plan.experts)) return -7;
  if (!vector_ok(bias, size, false)) return -8;
  if (!rows_ok(Z, n, size, false)) return -9;
  if (!rows_ok(Y, n, osize, touch)) return -10;
  if (!touch) return PGEMM_OK;
  Product p{};
  ProdArgs& a = p.a;
  a.A = X.data;
  a.lda = X.ld;
  a.B = W.data;
  a.ldb = W.ld;
  a.strideB = W.stride;
  a.D = Y.data;
  a.ldd = Y.ld;
  a.M = rows;
  a.N = n;
  a.K = k;
  a.bias = bias;
  a.strideBias = n;
  a.Z = Z.data;
  a.ldz = Z.ld;
  a.act = kind.act;
  a.out32 = kind.out_dtype == PGEMM_F32;
  a.offsets = plan.offsets;
  a.groups = plan.experts;
  a.rows = rows;
  a.gather = plan.tokens;
  a.gather_rows = plan.x_rows;
  p.dtype = kind.dtype;
  p.la = kInner;
  p.lb = W.order == PGEMM_KN ? kOuter : kInner;
  p.mode = kRows;
  if (!plan_call(&p, rows, nullptr, 0)) return -2;
  return launch_product(p, static_cast<hipStream_t>(stream));
}

int pgemm_expert_linear_backward(pgemm_kind kind, int rows, int n, int k, pgemm_plan plan,
                                 pgemm_rows dY, pgemm_rows Z, pgemm_rows X, pgemm_weight W,
                                 pgemm_rows dX, pgemm_weight dW, void* dbias, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  if (!kind_ok(kind)) return -1;
  if (!size_ok(rows)) return -2;
  if (!size_ok(n)) return -3;
  if (!size_ok(k)) return -4;
  const int size = size_of(kind.dtype), osize = size_of(kind.out_dtype);
  const bool read = rows > 0 && n > 0;
  if (!plan_ok(plan, rows, true)) return -5;
  if (!rows_ok(dY, n, size, read)) return -6;
  if (!rows_ok(Z, n, size, read && kind.act != PGEMM_ACT_NONE)) return -7;
  if (!rows_ok(X, k, size, read && k > 0 && dW.data != nullptr)) return -8;
  if (!weight_ok(W, k, n, size, read && k > 0 && dX.data != nullptr, plan.experts)) return -9;
  if (!rows_ok(dX, k, size, false)) return -10;
  if (!weight_ok(dW, k, n, osize, false, plan.experts)) return -11;
  if (!vector_ok(dbias, osize, false)) return -12;
  const int experts = plan.experts;
  const BackSpace space = back_space(kind, rows, n, k, experts, true);
  if (space.total() > 0 && (workspace == nullptr || !aligned_to(workspace, 16))) return -13;
  if (workspace_bytes < space.total()) return -14;
  BackArgs b{kind, rows, n, k, experts, plan.offsets, plan.tokens, plan.x_rows,
             dY,   Z,    X, dX, W,      dW,           n > 0 ? dbias : nullptr};
  if (n == 0) b.kind.act = PGEMM_ACT_NONE;
  return run_backward(b, workspace, space, static_cast<hipStream_t>(stream));
}

size_t pgemm_expert_linear_backward_workspace(pgemm_kind kind, int rows, int n, int k,
                                              int experts) {
  if (!kind_ok(kind) || rows < 0 || n <= 0 || k < 0 || experts < 1) return 0;
  return back_space(kind, rows, n, k, experts, true).total();
}

int pgemm_combine(int dtype, int m, int n, int top, int rows, pgemm_rows Y, const int* slots,
                  const float* weights, pgemm_rows residual, pgemm_rows out, void* stream) {
  if (!known(dtype)) return -1;
  if (m < 0 || m > (1 << 30) / kMaxTop) return -2;
  if (!size_ok(n)) return -3;
  if (top < 1 || top > kMaxTop) return -4;
  if (rows < 0) return -5;
  const bool touch = m > 0 && n > 0;
  const int size = size_of(dtype);
  if (!rows_ok(Y, n, size, touch && rows > 0)) return -6;
  if (!vector_ok(slots, 4, touch)) return -7;
  if (!vector_ok(weights, 4, false)) return -8;
  if (!rows_ok(residual, n, size, false)) return -9;
  if (!rows_ok(out, n, size, touch)) return -10;
  if (!touch) return PGEMM_OK;
  CombineArgs a{};
  a.Y = Y.data;
  a.slots = slots;
  a.weights = weights;
  a.R = residual.data;
  a.out = out.data;
  a.ldy = Y.ld;
  a.ldr = residual.ld;
  a.ldo = out.ld;
  a.m = m;
  a.n = n;
  a.top = top;
  a.rows = rows;
  a.tpr = threads_per_row(n, 256);
  return ops_of(dtype).combine(a, static_cast<hipStream_t>(stream)) == hipSuccess ? PGEMM_OK
                                                                               : PGEMM_EHIP;
}

int pgemm_combine_backward(int dtype, int m, int n, int top, int rows, pgemm_rows dout,
                           pgemm_rows Y, const int* slots, const float* weights, pgemm_rows dY,
                           float* dweights, void* stream) {
  if (!known(dtype)) return -1;
  if (m < 0 || m > (1 << 30) / kMaxTop) return -2;
  if (!size_ok(n)) return -3;
  if (top < 1 || top > kMaxTop) return -4;
  if (rows < 0) return -5;
  const int size = size_of(dtype);
  const bool read = m > 0 && n > 0;
  if (!rows_ok(dout, n, size, read)) return -6;
  if (!rows_ok(Y, n, size, read && rows > 0 && dweights != nullptr)) return -7;
  if (!vector_ok(slots, 4, m > 0)) return -8;
  if (!vector_ok(weights, 4, false)) return -9;
  if (!rows_ok(dY, n, size, false)) return -10;
  if (!vector_ok(dweights, 4, false)) return -11;
  if (m == 0 || (dY.data == nullptr && dweights == nullptr)) return PGEMM_OK;
  CombineBackArgs a{};
  a.dout = dout.data;
  a.Y = Y.data;
  a.slots = slots;
  a.weights = weights;
  a.dY = dY.data;
  a.dweights = dweights;
  a.ldo = dout.ld;
  a.ldy = Y.ld;
  a.ldd = dY.ld;
  a.m = m;
  a.n = n;
  a.top = top;
  a.rows = rows;
  return ops_of(dtype).combine_back(a, static_cast<hipStream_t>(stream)) == hipSuccess
             ? PGEMM_OK
             : PGEMM_EHIP;
}

namespace {

struct LinearCall {
  pgemm_kind kind;
  int m, n, k;
  pgemm_rows X;
  pgemm_weight W;
  const void* bias;
  pgemm_rows residual, Z, Y;
  void* workspace;
  size_t workspace_bytes;
  void* stream;
};
struct LinearBackwardCall {
  pgemm_kind kind;
  int m, n, k;
  pgemm_rows dY, Z, X;
  pgemm_weight W;
  pgemm_rows dX;
  pgemm_weight dW;
  void* dbias;
  void* workspace;
  size_t workspace_bytes;
  void* stream;
};
struct RouteCall {
  int dtype, m, experts, top, score, groups, top_groups, renorm;
  float scale;
  pgemm_rows logits;
  const float* bias;
  pgemm_route_out out;
  void* workspace;
  size_t workspace_bytes;
  void* stream;
};
struct RouteBackwardCall {
  int dtype, m, experts, top, score, renorm;
  float scale;
  const float* dweights;
  pgemm_rows logits;
  const int* expert_index;
  pgemm_rows dlogits;
  void* stream;
};
struct ExpertLinearCall {
  pgemm_kind kind;
  int rows, n, k;
  pgemm_plan plan;
  pgemm_rows X;
  pgemm_weight W;
  const void* bias;
  pgemm_rows Z, Y;
  void* stream;
};
struct ExpertLinearBackwardCall {
  pgemm_kind kind;
  int rows, n, k;
  pgemm_plan plan;
  pgemm_rows dY, Z, X;
  pgemm_weight W;
  pgemm_rows dX;
  pgemm_weight dW;
  void* dbias;
  void* workspace;
  size_t workspace_bytes;
  void* stream;
};
struct CombineCall {
  int dtype, m, n, top, rows;
  pgemm_rows Y;
  const int* slots;
  const float* weights;
  pgemm_rows residual, out;
  void* stream;
};
struct CombineBackwardCall {
  int dtype, m, n, top, rows;
  pgemm_rows dout, Y;
  const int* slots;
  const float* weights;
  pgemm_rows dY;
  float* dweights;
  void* stream;
};

}  // namespace

int pgemm_layer_call(int op, const void* args) {
  if (args == nullptr) return -2;
  switch (op) {
    case PGEMM_OP_LINEAR: {
      const LinearCall& c = *static_cast<const LinearCall*>(args);
      return pgemm_linear(c.kind, c.m, c.n, c.k, c.X, c.W, c.bias, c.residual, c.Z, c.Y,
                          c.workspace, c.workspace_bytes, c.stream);
    }
    case PGEMM_OP_LINEAR_BACKWARD: {
      const LinearBackwardCall& c = *static_cast<const LinearBackwardCall*>(args);
      return pgemm_linear_backward(c.kind, c.m, c.n, c.k, c.dY, c.Z, c.X, c.W, c.dX, c.dW,
                                   c.dbias, c.workspace, c.workspace_bytes, c.stream);
    }
    case PGEMM_OP_ROUTE: {
      const RouteCall& c = *static_cast<const RouteCall*>(args);
      return pgemm_route(c.dtype, c.m, c.experts, c.top, c.score, c.groups, c.top_groups,
                         c.renorm, c.scale, c.logits, c.bias, c.out, c.workspace,
                         c.workspace_bytes, c.stream);
    }
    case PGEMM_OP_ROUTE_BACKWARD: {
      const RouteBackwardCall& c = *static_cast<const RouteBackwardCall*>(args);
      return pgemm_route_backward(c.dtype, c.m, c.experts, c.top, c.score, c.renorm, c.scale,
                                  c.dweights, c.logits, c.expert_index, c.dlogits, c.stream);
    }
    case PGEMM_OP_EXPERT_LINEAR: {
      const ExpertLinearCall& c = *static_cast<const ExpertLinearCall*>(args);
      return pgemm_expert_linear(c.kind, c.rows, c.n, c.k, c.plan, c.X, c.W, c.bias, c.Z, c.Y,
                                 c.stream);
    }
    case PGEMM_OP_EXPERT_LINEAR_BACKWARD: {
      const ExpertLinearBackwardCall& c = *static_cast<const ExpertLinearBackwardCall*>(args);
      return pgemm_expert_linear_backward(c.kind, c.rows, c.n, c.k, c.plan, c.dY, c.Z, c.X, c.W,
                                          c.dX, c.dW, c.dbias, c.workspace, c.workspace_bytes,
                                          c.stream);
    }
    case PGEMM_OP_COMBINE: {
      const CombineCall& c = *static_cast<const CombineCall*>(args);
      return pgemm_combine(c.dtype, c.m, c.n, c.top, c.rows, c.Y, c.slots, c.weights, c.residual,
                           c.out, c.stream);
    }
    case PGEMM_OP_COMBINE_BACKWARD: {
      const CombineBackwardCall& c = *static_cast<const CombineBackwardCall*>(args);
      return pgemm_combine_backward(c.dtype, c.m, c.n, c.top, c.rows, c.dout, c.Y, c.slots,
                                    c.weights, c.dY, c.dweights, c.stream);
    }
    default: return -1;
  }
}

}  // extern "C"
