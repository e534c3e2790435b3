// Internal: argument checks of the operators' entry points, and the choice of a
// product's kernel and its launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.hpp"
#include "pgemm_layers.h"

namespace pgemm {
namespace layers {

constexpr int kUnits = 256;                       // compute units of an MI355X
// The kernels step past a size by a few tiles, in 32 bits.
constexpr int kMaxSize = 0x7fffffff - 4095;
constexpr long long kMaxThreads = 0xffffffffLL;   // of a launch, along x

inline int size_of(int dtype) { return dtype == PGEMM_F32 ? 4 : 2; }
inline bool known(int dtype) { return dtype == PGEMM_F32 || dtype == PGEMM_F16 || dtype == PGEMM_BF16; }

inline const TypeOps& ops_of(int dtype) {
  return dtype == PGEMM_F32 ? ops_f32() : dtype == PGEMM_F16 ? ops_f16() : ops_bf16();
}

inline bool kind_ok(const pgemm_kind& k) {
  return known(k.dtype) && (k.out_dtype == k.dtype || k.out_dtype == PGEMM_F32) &&
         k.act >= PGEMM_ACT_NONE && k.act <= PGEMM_ACT_SILU;
}

inline bool size_ok(int v) { return v >= 0 && v <= kMaxSize; }

inline long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }
inline long long round_up(long long a, long long b) { return ceil_div(a, b) * b; }
inline size_t align256(size_t b) { return (b + 255) & ~(size_t)255; }

inline bool aligned_to(const void* p, int bytes) {
  return reinterpret_cast<uintptr_t>(p) % (unsigned)bytes == 0;
}

// A matrix of `cols` columns that the call touches (need) or may touch.
inline bool rows_ok(const pgemm_rows& x, int cols, int size, bool need) {
  if (x.data == nullptr) return !need;
  return aligned_to(x.data, size) && x.ld >= (cols > 1 ? cols : 1);
}
inline bool weight_ok(const pgemm_weight& w, int k, int n, int size, bool need, int experts) {
  if (w.data == nullptr) return !need;
  if (w.order != PGEMM_KN && w.order != PGEMM_NK) return false;
  const int cols = w.order == PGEMM_KN ? n : k, rows = w.order == PGEMM_KN ? k : n;
  if (!aligned_to(w.data, size) || w.ld < (cols > 1 ? cols : 1)) return false;
  if (experts <= 1) return true;
  return w.stride >= (rows > 0 ? (long long)(rows - 1) * w.ld + cols : 0);
}
inline bool vector_ok(const void* p, int size, bool need) {
  return p == nullptr ? !need : aligned_to(p, size);
}

// offsets are read by a call that touches anything (need).
inline bool plan_ok(const pgemm_plan& p, int rows, bool need) {
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
inline int operand_loading(const void* p, long long ld, int size, int inner, long long stride) {
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
// The three classes', and what a split adds: its launch, and the partial sums' traffic.
struct ClassTimes {
  ClassTime of[3];
  double reduce, bandwidth;
};
inline const ClassTimes& class_times(int size) {
  static const ClassTimes t16 = {{{1.35e15, 10e-6, 1, {0, 0, 0, 0}},
                                  {1.10e15, 7e-6, 2, {0, 0.7, 0, 0}},
                                  {0.60e15, 3.5e-6, 4, {0, 0.5, 0.75, 0.9}}}, 4e-6, 6e12};
  static const ClassTimes t32 = {{{142e12, 6e-6, 1, {0, 0, 0, 0}},
                                  {130e12, 4e-6, 2, {0, 0.93, 0, 0}},
                                  {119e12, 3e-6, 4, {0, 0.8, 0.9, 0.95}}}, 4e-6, 6e12};
  return size == 2 ? t16 : t32;
}

inline double tiles_time(const ClassTime& c, double tiles, double tile_flops) {
  const long long whole = (long long)tiles;
  const long long per = ceil_div(whole + (tiles > (double)whole ? 1 : 0), kUnits);
  const double one = tile_flops / (c.rate / kUnits);
  const long long full = per / c.together, left = per % c.together;
  double t = (double)full * (c.together * one + c.fixed);
  if (left > 0) t += (double)left * one / c.part[left] + c.fixed;
  return t;
}

// Bytes of a plan's partial sums.
inline size_t split_space(const Plan& p, int mode, long long rows, int groups, int n) {
  if (p.splits <= 1) return 0;
  return (size_t)p.splits * (size_t)rows * (size_t)n * 4 * (size_t)(mode == kSums ? groups : 1);
}

// The tiles of a product.  `rows` as in plan_product.
inline void set_tiles(ProdArgs* a, int kernel, int mode, long long rows) {
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
inline bool launch_fits(int kernel, int mode, long long rows, int groups, int n) {
  ProdArgs a{};
  a.N = n;
  a.groups = groups;
  a.rows = (int)rows;
  a.splits = 1;
  set_tiles(&a, kernel, mode, rows);
  return prod_grid(a, mode, kernel).x <= kMaxThreads / prod_threads(kernel);
}

// Shares k summed indices between p->splits workgroups, in whole steps of bk: as many as have
// work, the last of whose ends, rounded up, has to stay within the kernels' 32 bits.
inline void share_inner(Plan* p, int k, int bk) {
  for (int s = p->splits; ; --s) {
    const long long each = round_up(ceil_div(k, s), bk), n = ceil_div(k, each);
    if (s > 1 && n * each > 0x7fffffffLL) continue;
    p->k_split = (int)each;
    p->splits = (int)n;
    return;
  }
}

// rows: the rows of D over all groups (how they are distributed is not known
// here; any distribution is correct).  may_split: the summed index may be
// shared by workgroups, through partial sums in `ws_bytes` bytes (any_ws: as
// many as it takes).  may_few: the few-rows kernels may be chosen.  times: of the kernels
// that take the product (nullptr: the layer operators').
inline Plan plan_product(int size, int la, int mode, long long rows, int groups, int n, int k,
                         int loading, size_t ws_bytes, bool any_ws, bool may_split = true,
                         bool may_few = true, const ClassTimes* times = nullptr) {
  if (times == nullptr) times = &class_times(size);
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
  if (may_few && la == kInner && per <= 32 && launch_fits(few, mode, rows, groups, n)) {
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
      const ClassTime& ct = times->of[c];
      const double matrix = (double)rows * n * (mode == kSums ? groups : 1);
      for (const int s : {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 24, 32, 48, 64}) {
        // (beyond 16 pieces per compute unit nothing is left to balance)
        if (s > 1 && (!may_split || depth / s < 4 * bk || tiles * s > 16.0 * kUnits)) break;
        const double split = s > 1 ? times->reduce + s * matrix * 8 / times->bandwidth : 0;
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
    if (mode == kDense) share_inner(&p, k, bk);
    const size_t need = split_space(p, mode, rows, groups, n);
    if (!any_ws && ws_bytes < need)   // the best plan that needs no space
      return plan_product(size, la, mode, rows, groups, n, k, loading, 0, false, false, may_few,
                          times);
  }
  return p;
}

// Workspace that plan_product may use for a product, over any alignment.
inline size_t split_bytes(int size, int la, int mode, long long rows, int groups, int n, int k) {
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
inline bool plan_call(Product* p, long long rows, void* ws, size_t ws_bytes) {
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

inline int launch_product(const Product& p, hipStream_t s) {
  return ops_of(p.dtype).prod(p.a, p.la, p.lb, p.mode, p.plan.kernel, p.plan.loading, s) ==
                 hipSuccess
             ? PGEMM_OK
             : PGEMM_EHIP;
}

// Threads per row of a row-wise kernel with 8 columns per thread.
inline int threads_per_row(int n, int most) {
  int t = 1;
  while (t < most && t * 8 < n) t *= 2;
  return t;
}

// Row chunks per group of the slope kernel: enough workgroups for every
// compute unit, at least 16 rows of an average group each.
inline int slope_chunks(long long rows, int groups, int n) {
  if (n < 1) return 1;
  const long long cols = ceil_div(n, threads_per_row(n, 64) * 8);
  long long c = 4 * kUnits / (cols * groups);
  const long long most = ceil_div(ceil_div(rows, groups), 16);
  if (c > most) c = most;
  return c < 1 ? 1 : (int)c;
}

}  // namespace layers
}  // namespace pgemm
