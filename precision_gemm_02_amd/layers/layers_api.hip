// C ABI of the layer operators: argument checks, the choice of kernels and
// their launches.  Declarations and the contract are in pgemm_layers.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.hpp"
#include "pgemm_layers.h"

namespace pgemm {
namespace layers {
namespace {

constexpr int kUnits = 256;                       // compute units of an MI355X
// The kernels step past a size by a few tiles, in 32 bits.
constexpr int kMaxSize = 0x7fffffff - 4095;
constexpr long long kMaxThreads = 0xffffffffLL;   // of a launch, along x

int size_of(int dtype) { return dtype == PGEMM_F32 ? 4 : 2; }
bool known(int dtype) { return dtype == PGEMM_F32 || dtype == PGEMM_F16 || dtype == PGEMM_BF16; }

const TypeOps& ops_of(int dtype) {
  return dtype == PGEMM_F32 ? ops_f32() : dtype == PGEMM_F16 ? ops_f16() : ops_bf16();
}

bool kind_ok(const pgemm_kind& k) {
  return known(k.dtype) && (k.out_dtype == k.dtype || k.out_dtype == PGEMM_F32) &&
         k.act >= PGEMM_ACT_NONE && k.act <= PGEMM_ACT_SILU;
}

bool size_ok(int v) { return v >= 0 && v <= kMaxSize; }

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }
long long round_up(long long a, long long b) { return ceil_div(a, b) * b; }
size_t align256(size_t b) { return (b + 255) & ~(size_t)255; }

bool aligned_to(const void* p, int bytes) {
  return reinterpret_cast<uintptr_t>(p) % (unsigned)bytes == 0;
}

// A matrix of `cols` columns that the call touches (need) or may touch.
bool rows_ok(const pgemm_rows& x, int cols, int size, bool need) {
  if (x.data == nullptr) return !need;
  return aligned_to(x.data, size) && x.ld >= (cols > 1 ? cols : 1);
}
bool weight_ok(const pgemm_weight& w, int k, int n, int size, bool need, int experts) {
  if (w.data == nullptr) return !need;
  if (w.order != PGEMM_KN && w.order != PGEMM_NK) return false;
  const int cols = w.order == PGEMM_KN ? n : k, rows = w.order == PGEMM_KN ? k : n;
  if (!aligned_to(w.data, size) || w.ld < (cols > 1 ? cols : 1)) return false;
  if (experts <= 1) return true;
  return w.stride >= (rows > 0 ? (long long)(rows - 1) * w.ld + cols : 0);
}
bool vector_ok(const void* p, int size, bool need) {
  return p == nullptr ? !need : aligned_to(p, size);
}

// offsets are read by a call that touches anything (need).
bool plan_ok(const pgemm_plan& p, int rows, bool need) {
  return p.experts >= 1 && p.experts <= kMaxExperts && vector_ok(p.offsets, 4, need) &&
         vector_ok(p.tokens, 4, false) && p.x_rows >= 0 &&
         (p.tokens != nullptr ? p.x_rows > 0 || rows == 0 : p.x_rows >= rows);
}

// ---- the choice of a product's kernel ----------------------------------------

struct Plan {
  int kernel = -1;         // (-1: none, the product has more tiles than a launch takes)
  int splits = 1;
  int k_split = 0;
  int loading = kThrough;
};

// The loading that an operand allows: `inner` is its contiguous extent.
int operand_loading(const void* p, long long ld, int size, int inner, long long stride) {
  const int v = 16 / size;
  if (aligned_to(p, 16) && ld % v == 0 && inner % v == 0 && stride % v == 0) return kDirect;
  // fp32 goes through registers instead: 4098 x 3002 x 1022 k x n 230 us, with
  // kRagged 247 (bf16 78 us through registers, 57 so)
  return size == 2 && aligned_to(p, 4) && ld % 2 == 0 && stride % 2 == 0 ? kRagged : kThrough;
}

// A tile class's time, fitted to 15 dense shapes in both weight orders (64 to
// 8192 rows) and 5 expert shapes, every class timed on each: the flop rate of
// `together` workgroups that share a compute unit, the share of it that fewer
// of them reach, and the fixed time of each such group (prologue, epilogue).
struct ClassTime {
  double rate;             // of the whole chip
  double fixed;            // seconds
  int together;
  double part[4];          // by workgroups left over (0: unused)
};
ClassTime class_time(int kernel, int size) {
  static const ClassTime t16[3] = {{1.35e15, 10e-6, 1, {0, 0, 0, 0}},
                                   {1.10e15, 7e-6, 2, {0, 0.7, 0, 0}},
                                   {0.60e15, 3.5e-6, 4, {0, 0.5, 0.75, 0.9}}};
  static const ClassTime t32[3] = {{142e12, 6e-6, 1, {0, 0, 0, 0}},
                                   {130e12, 4e-6, 2, {0, 0.93, 0, 0}},
                                   {119e12, 3e-6, 4, {0, 0.8, 0.9, 0.95}}};
  return (size == 2 ? t16 : t32)[kernel];
}

double tiles_time(const ClassTime& c, double tiles, double tile_flops) {
  const long long whole = (long long)tiles;
  const long long per = ceil_div(whole + (tiles > (double)whole ? 1 : 0), kUnits);
  const double one = tile_flops / (c.rate / kUnits);
  const long long full = per / c.together, left = per % c.together;
  double t = (double)full * (c.together * one + c.fixed);
  if (left > 0) t += (double)left * one / c.part[left] + c.fixed;
  return t;
}

// Bytes of a plan's partial sums.
size_t split_space(const Plan& p, int mode, long long rows, int groups, int n) {
  if (p.splits <= 1) return 0;
  return (size_t)p.splits * (size_t)rows * (size_t)n * 4 * (size_t)(mode == kSums ? groups : 1);
}

// The tiles of a product.  `rows` as in plan_product.
void set_tiles(ProdArgs* a, int kernel, int mode, long long rows) {
  if (kernel >= kFew16) {
    a->tiles_m = 1;
    a->tiles_n = (int)ceil_div(a->N, few_columns(kernel));
    return;
  }
  long long tm = ceil_div(rows, kShape[kernel].bm);
  if (mode == kRows) tm += a->groups < rows ? a->groups : rows;   // partly filled tiles
  a->tiles_m = (int)tm;
  a->tiles_n = (int)ceil_div(a->N, kShape[kernel].bn);
}

// Whether one launch takes all of them.
bool launch_fits(int kernel, int mode, long long rows, int groups, int n) {
  ProdArgs a{};
  a.N = n;
  a.groups = groups;
  a.rows = (int)rows;
  a.splits = 1;
  set_tiles(&a, kernel, mode, rows);
  return prod_grid(a, mode, kernel).x <= kMaxThreads / prod_threads(kernel);
}

// rows: the rows of D over all groups (how they are distributed is not known
// here; any distribution is correct).  may_split: the summed index may be
// shared by workgroups, through partial sums in `ws_bytes` bytes (any_ws: as
// many as it takes).
Plan plan_product(int size, int la, int mode, long long rows, int groups, int n, int k,
                  int loading, size_t ws_bytes, bool any_ws, bool may_split = true) {
  Plan p;
  p.loading = loading;
  const int bk = 128 / size;
  if (mode == kRows) may_split = false;
  if (mode == kRows && groups > rows) groups = (int)rows;
  const double per = mode == kRows ? (double)rows / groups : (double)rows;
  // Few rows: B is read once, the rest is latency.  The few-rows kernel
  // takes 16 or 32 rows per pass and never needs a tile of operands.
  const long long wide = ceil_div(n, 64) * (mode == kRows ? groups : 1);
  const int few = wide >= 2 * kUnits ? (per <= 16 ? kFew16Wide : kFew32Wide)
                                     : (per <= 16 ? kFew16 : kFew32);
  if (la == kInner && per <= 32 && launch_fits(few, mode, rows, groups, n)) {
    p.kernel = few;
    if (may_split && n > 0) {   // (no columns: the size of a workspace that is not used)
      // one split per free compute unit, each of 16 units of 128 bytes at least
      long long s = kUnits / ceil_div(n, few_columns(p.kernel));
      if (s > k / (16 * bk)) s = k / (16 * bk);
      p.splits = s < 1 ? 1 : s > 64 ? 64 : (int)s;
    }
  } else {
    double best = 0;
    for (int c = 0; c < 3; ++c) {
      if (c == kTile256 && loading != kDirect) continue;
      if (!launch_fits(c, mode, rows, groups, n)) continue;
      const int bm = kShape[c].bm, bn = kShape[c].bn;
      // tiles that are half empty waste the loads too (512 tokens, top 8 of
      // 64 experts, 1024 x 1024: 39 us with 64-row tiles, 45 with 128)
      if (mode == kRows && c != kTile64 && 2 * per <= bm &&
          launch_fits(kTile64, mode, rows, groups, n))
        continue;
      double tiles = (double)ceil_div(n, bn);
      if (mode == kRows) tiles *= groups * (per / bm > 0.5 ? per / bm + 0.5 : 1.0);
      else tiles *= (double)ceil_div(rows, bm) * (mode == kSums ? groups : 1);
      const double depth = mode == kSums ? (double)k / groups : (double)k;
      const ClassTime ct = class_time(c, size);
      const double matrix = (double)rows * n * (mode == kSums ? groups : 1);
      for (const int s : {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 24, 32, 48, 64}) {
        // (beyond 16 pieces per compute unit nothing is left to balance)
        if (s > 1 && (!may_split || depth / s < 4 * bk || tiles * s > 16.0 * kUnits)) break;
        // the partial sums' traffic, and the launch that adds them
        const double split = s > 1 ? 4e-6 + s * matrix * 8 / 6e12 : 0;
        const double t = tiles_time(ct, tiles * s, 2.0 * bm * bn * depth / s) + split;
        if (best == 0 || t < best) {
          best = t;
          p.kernel = c;
          p.splits = s;
        }
      }
    }
  }
  if (p.splits > 1) {
    if (mode == kDense) {
      p.k_split = (int)round_up(ceil_div(k, p.splits), bk);
      p.splits = (int)ceil_div(k, p.k_split);
    }
    const size_t need = split_space(p, mode, rows, groups, n);
    if (!any_ws && ws_bytes < need)   // the best plan that needs no space
      return plan_product(size, la, mode, rows, groups, n, k, loading, 0, false, false);
  }
  return p;
}

// Workspace that plan_product may use for a product, over any alignment.
size_t split_bytes(int size, int la, int mode, long long rows, int groups, int n, int k) {
  size_t most = 0;
  for (const int loading : {kThrough, kDirect}) {
    const Plan p = plan_product(size, la, mode, rows, groups, n, k, loading, 0, true);
    const size_t b = split_space(p, mode, rows, groups, n);
    if (b > most) most = b;
  }
  return most;
}

// A product with its plan, ready to be launched.
struct Product {
  ProdArgs a;
  int dtype, la, lb, mode;
  Plan plan;
};

// Fill in what depends on the plan; false if no launch takes the product.
// `rows` as in plan_product.
bool plan_call(Product* p, long long rows, void* ws, size_t ws_bytes) {
  ProdArgs& a = p->a;
  const int size = size_of(p->dtype), la = p->la, lb = p->lb, mode = p->mode;
  const int al = operand_loading(a.A, a.lda, size,
                                 la == kInner ? (mode == kSums ? 0 : a.K) : a.M, 0);
  const int bl = operand_loading(a.B, a.ldb, size, lb == kInner ? a.K : a.N,
                                 mode == kRows ? a.strideB : 0);
  int loading = al == kDirect && bl == kDirect       ? kDirect
                : al != kThrough && bl != kThrough   ? kRagged
                                                     : kThrough;
  if (mode == kSums && loading == kRagged) loading = kThrough;   // see Loader
  p->plan = plan_product(size, la, mode, rows, a.groups, a.N, mode == kSums ? a.rows : a.K,
                         loading, ws == nullptr ? 0 : ws_bytes, false);
  if (p->plan.kernel < 0) return false;
  a.splits = p->plan.splits;
  a.k_split = p->plan.k_split;
  a.partial = static_cast<float*>(ws);
  set_tiles(&a, p->plan.kernel, mode, rows);
  return true;
}

int launch_product(const Product& p, hipStream_t s) {
  return ops_of(p.dtype).prod(p.a, p.la, p.lb, p.mode, p.plan.kernel, p.plan.loading, s) ==
                 hipSuccess
             ? PGEMM_OK
             : PGEMM_EHIP;
}

// Threads per row of a row-wise kernel with 8 columns per thread.
int threads_per_row(int n, int most) {
  int t = 1;
  while (t < most && t * 8 < n) t *= 2;
  return t;
}

// Row chunks per group of the slope kernel: enough workgroups for every
// compute unit, at least 16 rows of an average group each.
int slope_chunks(long long rows, int groups, int n) {
  if (n < 1) return 1;
  const long long cols = ceil_div(n, threads_per_row(n, 64) * 8);
  long long c = 4 * kUnits / (cols * groups);
  const long long most = ceil_div(ceil_div(rows, groups), 16);
  if (c > most) c = most;
  return c < 1 ? 1 : (int)c;
}

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
