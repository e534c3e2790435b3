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
// (8 n bytes) once, so that it should have a few rows, and one of 1024 threads on
// each compute unit is enough (8192 x 4096 bf16: 256 of them 51 us, 512 of 512 threads
// 52, 1024 of 256 threads 78); and each thread adds its rows one after the other, so
// that it should not have too many (as far as a launch of norm_sums_kernel goes: 2^24
// workgroups).
int norm_groups(int m, int n) {
  const long long few = ceil_div(m, 2), long_sum = ceil_div(m, 1024);
  const long long cap = n <= 2048 ? 2 * kUnits : kUnits;
  long long g = few < cap ? few : cap;
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

// ---- gated products ------------------------------------------------------------

constexpr int kMaxGated = (1 << 30) - 4096;      // columns: both weights' together fit

bool gate_weights_ok(const pgemm_gate_weights& w, int k, int n, int size, bool need) {
  if (!weight_ok(w.gate, k, n, size, need, 1) || !weight_ok(w.up, k, n, size, need, 1)) return false;
  return !need || (w.gate.order == w.up.order && w.gate.ld == w.up.ld);
}

// Columns of each weight that a workgroup takes.
int gate_columns(int kernel) {
  if (kernel >= kFew16) return kernel >= kFew16Wide ? 32 : 16;
  return kShape[kernel].bn / 2;
}

// The plan of a few-rows kernel (of 16 or 32, which is all that the kernels take), whose
// workgroups take `wide` columns where that gives every compute unit one, else 16.
// `results`: partial sums of a row and split.  (No kernel if one launch does not take them.)
Plan few_plan(int size, int m, int n, int wide, int results, int k, int loading, size_t ws_bytes,
              bool any_ws) {
  Plan p;
  p.loading = loading;
  const bool is_wide = ceil_div(n, wide) >= kUnits;
  if (m > 32 || ceil_div(n, is_wide ? wide : 16) > kMaxThreads / prod_threads(kFew16)) return p;
  p.kernel = is_wide ? (m <= 16 ? kFew16Wide : kFew32Wide) : (m <= 16 ? kFew16 : kFew32);
  const int bk = 128 / size;
  // one split per free compute unit, each of 16 units of 128 bytes at least
  long long s = kUnits / ceil_div(n, is_wide ? wide : 16);
  if (s > k / (16 * bk)) s = k / (16 * bk);
  if (s > 64) s = 64;
  if (s > 1) {
    p.splits = (int)s;
    share_inner(&p, k, bk);
    if (!any_ws && ws_bytes < split_space(p, kDense, m, 1, results)) p.splits = 1;
  }
  return p;
}

// The times of this file's tile kernels (see ClassTimes), fitted to 24 shapes of 64 to 8192
// rows, every class timed on each alone and split 2, 4 and 8 ways.  The class and split that
// they choose take 1.00 to 1.01 times the best one's time in the mean; with the layer
// operators' times it was 1.05 for whole 16-bit tiles (1000 x 2048 x 1024: 15.4 us, now
// 12.4), 1.03 for 8 bits (128 x 2048 x 2048: 12.4 us, now 9.4).
const ClassTimes* pair_times(int size, int loading) {
  static const ClassTimes whole16 = {{{1.98e15, 10.5e-6, 1, {0, 0, 0, 0}},
                                      {1.26e15, 5e-6, 2, {0, 1.0, 0, 0}},
                                      {0.73e15, 3.5e-6, 4, {0, 0.57, 0.92, 0.92}}}, 6.4e-6, 8.1e12};
  static const ClassTimes through16 = {{{0, 0, 1, {0, 0, 0, 0}},        // (has no largest tiles)
                                        {0.82e15, 5.3e-6, 2, {0, 0.79, 0, 0}},
                                        {0.43e15, 3.3e-6, 4, {0, 0.75, 0.93, 1.0}}}, 3.8e-6, 6.4e12};
  static const ClassTimes any32 = {{{150e12, 2.9e-6, 1, {0, 0, 0, 0}},
                                    {160e12, 5.3e-6, 2, {0, 0.89, 0, 0}},
                                    {155e12, 5.2e-6, 4, {0, 0.965, 0.994, 0.994}}}, 4.3e-6, 5.9e12};
  return size == 4 ? &any32 : loading == kDirect ? &whole16 : &through16;
}

// The 8-bit tile kernels' times (whole8 and wide8 fitted so too).  wide8, of fp32 results,
// serves 16-bit results of rows that are not whole chunks too: of 10 shapes with either kind of
// scales the choice took 1.00 to 1.07 times the best class's time.  Of such rows with fp32
// results it took up to 1.79 times (8191 x 8192 x 4095 in tiles of 128 2130 us, of 64 1255;
// 4096^2 x 4095 534 and 320; 2000 x 2048 x 4095 137 and 84), hence odd32.
const ClassTimes* times8(bool direct, bool wide) {
  static const ClassTimes whole8 = {{{2.77e15, 12.2e-6, 1, {0, 0, 0, 0}},
                                     {2.19e15, 8.7e-6, 2, {0, 0.92, 0, 0}},
                                     {1.39e15, 6.6e-6, 4, {0, 0.84, 0.84, 1.0}}}, 3.8e-6, 8.5e12};
  static const ClassTimes wide8 = {{{0, 0, 1, {0, 0, 0, 0}},            // (have no largest tiles)
                                    {1.20e15, 9.5e-6, 2, {0, 0.70, 0, 0}},
                                    {0.81e15, 7.5e-6, 4, {0, 0.92, 0.92, 0.98}}}, 2e-6, 7.6e12};
  static const ClassTimes odd32 = {{{0, 0, 1, {0, 0, 0, 0}},
                                    {0.26e15, 2e-6, 2, {0, 0.99, 0, 0}},
                                    {0.46e15, 6e-6, 4, {0, 0.45, 0.67, 0.9}}}, 2e-6, 7.6e12};
  if (!direct && wide) return &odd32;
  return direct && !wide ? &whole8 : &wide8;
}

// A plan that takes none of the layer operators' kernels.
Plan plan_pair(int size, int la, int rows, int n, int k, int loading, size_t ws_bytes, bool any_ws) {
  return plan_product(size, la, kDense, rows, 1, n, k, loading, ws_bytes, any_ws, true, false,
                      pair_times(size, loading));
}

// The plan of a gated product: a product with 2 n columns, but for few rows.  Workspace as in
// plan_product.
Plan gate_plan(int size, int m, int n, int k, int loading, size_t ws_bytes, bool any_ws) {
  const Plan p = few_plan(size, m, n, gate_columns(kFew16Wide), 2 * n, k, loading, ws_bytes, any_ws);
  if (p.kernel >= 0) return p;
  return plan_pair(size, kInner, m, 2 * n, k, loading, ws_bytes, any_ws);
}

// The plan of a product in 8 bits, of rows in whole chunks (direct) or not, with fp32 results
// (wide) or 16-bit ones; only 16-bit results of whole chunks have tiles of 256 x 256.
constexpr int kFewWide8 = 32;                     // columns of its wide few-rows kernels
Plan plan8(int m, int n, int k, bool direct, bool wide, size_t ws_bytes, bool any_ws) {
  const int loading = direct && !wide ? kDirect : kThrough;
  const Plan p = few_plan(1, m, n, kFewWide8, n, k, loading, ws_bytes, any_ws);
  if (p.kernel >= 0) return p;
  return plan_product(1, kInner, kDense, m, 1, n, k, loading, ws_bytes, any_ws, true, false,
                      times8(direct, wide));
}

int pair_loading(const pgemm_gate_weights& w, int size, int inner) {
  const int g = operand_loading(w.gate.data, w.gate.ld, size, inner, 0);
  const int u = operand_loading(w.up.data, w.up.ld, size, inner, 0);
  return g == u ? g : g == kThrough || u == kThrough ? kThrough : kRagged;
}
int both_loading(int a, int b) {
  return a == kDirect && b == kDirect ? kDirect : a != kThrough && b != kThrough ? kRagged : kThrough;
}

// Rows of a gated backward call from which operands whose rows are not whole chunks of 16
// bytes are copied into rows that are, for the whole-tile kernels, rather than taken through
// registers (us, bf16 and fp32; k x n weights).  X, which also brings both weights' gradients
// into one launch: 64 rows of 1001 x 1001 27.9 and 28 (fp32 38.6, 38), 128 of 501 x 500 30.6
// and 24.8, 1000 of 1001 x 1001 60 and 42.  The weights, whose copy does not shrink with the
// rows: beside X's 300 rows of 1001 x 1001 30.1 and 33.9 (fp32 54.2, 52.5), 512 of 2047 x 2047
// 61 and 58 (fp32 181, 163), 4000 of them 177 and 159; in a launch of their own 512 of 1024 x
// 2047 37 and 40 (fp32 100, 93), 2000 68 and 65.
constexpr int kPadRows = 64;
int pad_weight_rows(int size, bool beside) {
  if (size == 4) return beside ? 256 : 512;
  return beside ? 512 : 2048;
}

// Bytes of a copy of X (m x k), and of one weight in either order, into whole chunks; 0 where
// sizes alone do not ask for one.
size_t pad_bytes(int size, int height, int width) {
  return width % (16 / size) ? align256((size_t)height * (size_t)round_up(width, 8) * (size_t)size) : 0;
}
size_t pad_weight_bytes(int size, int k, int n) {
  const size_t kn = pad_bytes(size, k, n), nk = pad_bytes(size, n, k);
  return kn > nk ? kn : nk;
}

// The copies that a call makes before its products.
struct Copies {
  PadRowsArgs args{};
  int count = 0;
  void add(const void** at, long long* ld, int height, int width, char* to) {
    const long long wide = round_up(width, 8);
    args.of[count++] = {*at, to, *ld, wide, height, width, threads_per_row((int)wide, 256)};
    *at = to;
    *ld = wide;
  }
};

// The parts of a gated backward call's workspace: dZ of both weights, partial sums (of the
// bias gradients, then of the products, in stream order), padded copies of X and the weights.
struct GateSpace {
  size_t dz = 0, rest = 0, x = 0, w = 0;
  int half = 0, chunks = 1;
  size_t total() const { return dz + rest + x + 2 * w; }
};

// Row chunks of the slope kernel (its grid's y): two workgroups for every compute unit's four,
// at least 8 rows each; and as norm_groups has it, no thread should add more than 1024 rows one
// after the other.
int gate_chunks(int rows, int half) {
  if (half < 1) return 1;
  const int tpr = threads_per_row(half, 64);
  long long c = 8 * kUnits / ceil_div(half, tpr * 8);
  const long long most = ceil_div(rows, 8), long_sum = ceil_div(rows, 1024LL * (256 / tpr));
  if (c > most) c = most;
  if (c < long_sum) c = long_sum;
  return c < 1 ? 1 : c > 65535 ? 65535 : (int)c;
}

// The copies of a forward call, behind its partial sums.  Through registers k x n weights of odd
// rows cost most (us, bf16 and fp32: 64 rows of 1001 x 1001 15.0 and with copies 15.6, fp32 19.3
// and 22.8; 128 of 2047 x 2047 25.8, 25.2 and 51, 39; 300 of 1001 x 1000 18.3, 11.4 and 38, 24;
// 4000 of 2047 x 2047 113, 69), n x k weights least (512 of 2047 x 2047 23.4, 27.4 and 81, 79;
// 2000 of 1001 x 1001 21.1, 23.9; 1000 of 2047 x 2047 34.7, 29.6 and 142, 138; 4000 105, 68).
// The rule for k x n weights goes by the rows alone.  From about 500 x 500 on the copies win (128
// rows of 501 x 501 11.6, 10.2 and 21.4, 15.8); in smaller ones they are a launch too many (130
// rows of 129 x 64 4.5, 9.6 and 8.1, 9.0; 130 to 8000 rows of 33 x 33 8.3, 9.9 in either; 1000
// of 257 x 257 8.8, 10.1 and 14.4, 12.9): there a call without the workspace is faster.
struct GateCopies {
  size_t x = 0, w = 0;
  size_t total() const { return x + 2 * w; }
};
GateCopies gate_copies(int size, int m, int n, int k, bool kn) {
  GateCopies c;
  const double items = (double)m * n * k;
  if (n < 1 || k < 1 || (kn ? m < 128 : size != 2 || m < 512 || items < 3e9)) return c;
  c.x = pad_bytes(size, m, k);
  c.w = kn ? pad_bytes(size, k, n) : pad_bytes(size, n, k);
  return c;
}

GateSpace gate_space(const pgemm_kind& kind, int m, int n, int k) {
  GateSpace g;
  const int size = size_of(kind.dtype);
  g.half = (int)round_up(n, 128 / size);       // whole steps of the kernels
  g.dz = align256((size_t)m * 2 * (size_t)g.half * (size_t)size);
  const int rows = m < 1 ? 1 : m;
  g.chunks = gate_chunks(rows, g.half);
  g.rest = 2 * (size_t)g.chunks * (size_t)n * 4;
  const int both = 2LL * k <= kMaxSize ? 2 * k : k;
  auto pair = [&](int la, int height, int width, int along, int loading) {
    return split_space(plan_pair(size, la, height, width, along, loading, 0, true), kDense, height, 1,
                       width);
  };
  const size_t parts[] = {pair(kInner, rows, k, 2 * g.half, kThrough),
                          pair(kInner, rows, k, 2 * g.half, kDirect),
                          pair(kOuter, k, n, rows, kDirect),
                          pair(kOuter, n, k, rows, kDirect),
                          pair(kOuter, k, 2 * n, rows, kDirect),
                          pair(kOuter, n, both, rows, kDirect),
                          split_bytes(size, kOuter, kDense, k, 1, n, rows),
                          split_bytes(size, kOuter, kDense, n, 1, k, rows)};
  for (const size_t x : parts)
    if (x > g.rest) g.rest = x;
  g.rest = align256(g.rest);
  const int per = 16 / size;
  if (m >= kPadRows && n > 0 && k > 0) {
    g.x = pad_bytes(size, m, k);
    if (m >= pad_weight_rows(size, k % per != 0)) g.w = pad_weight_bytes(size, k, n);
  }
  return g;
}

// Whether pair_whole_kernel takes operands whose loads are direct: offsets within a tile
// of at most 256 rows fit 31 bits.
bool whole_tiles(int size, long long lda, long long ldb) {
  const long long most = 0x7fffffffLL / (256 * size) - 16;
  return lda < most && ldb < most;
}

// The products for the weights' gradients, dW = X^T dZ of each: one launch for both
// where pair_whole_kernel takes them, else one of `one` for each that is wanted.
struct WeightGradients {
  bool whole = false;
  PairArgs args{};
  int kernel = -1;
  int count = 0;
  Product one[2] = {};
};

bool plan_weights(WeightGradients* g, const pgemm_kind& kind, int m, int n, int k,
                  const pgemm_rows& X, const void* const* dz, long long ldz,
                  const pgemm_gate_weights& dW, int x_cols, void* ws, size_t ws_bytes) {
  const int size = size_of(kind.dtype);
  const pgemm_weight* const to[2] = {&dW.gate, &dW.up};
  const pgemm_weight* first = nullptr;
  bool alike = true;
  for (int w = 0; w < 2; ++w) {
    if (to[w]->data == nullptr) continue;
    const bool kn = to[w]->order == PGEMM_KN;
    if (first == nullptr) first = to[w];
    alike = alike && to[w]->order == first->order && to[w]->ld == first->ld;
    ProdArgs& a = g->one[g->count++].a;
    a.A = kn ? X.data : dz[w];
    a.lda = kn ? X.ld : ldz;
    a.B = kn ? dz[w] : X.data;
    a.ldb = kn ? ldz : X.ld;
    a.D = const_cast<void*>(to[w]->data);
    a.ldd = to[w]->ld;
    a.out32 = kind.out_dtype == PGEMM_F32;
    a.M = kn ? k : n;
    a.N = kn ? n : k;
    a.K = m;
  }
  // dZ's rows go on behind column n (see gate_slope_kernel): its loads are direct
  if (alike && whole_tiles(size, X.ld, ldz) &&
      operand_loading(X.data, X.ld, size, x_cols, 0) == kDirect) {
    g->args.p = g->one[0].a;
    g->args.count = g->count;
    g->args.A2 = g->one[g->count - 1].a.A;
    g->args.B2 = g->one[g->count - 1].a.B;
    g->args.D2 = g->one[g->count - 1].a.D;
    ProdArgs& a = g->args.p;
    const long long columns = (long long)a.N * g->count;
    if (columns <= kMaxSize) {
      const Plan p = plan_pair(size, kOuter, a.M, (int)columns, m, kDirect, ws_bytes, false);
      if (p.kernel >= 0) {
        a.splits = p.splits;
        a.k_split = p.k_split;
        a.partial = static_cast<float*>(ws);
        set_tiles(&a, p.kernel, kDense, a.M);
        g->kernel = p.kernel;
        g->whole = (long long)a.tiles_m * a.tiles_n * g->count <= kMaxThreads / prod_threads(p.kernel);
      }
    }
  }
  if (g->whole) return true;
  for (int i = 0; i < g->count; ++i) {
    Product& p = g->one[i];
    p.dtype = kind.dtype;
    p.la = p.lb = kOuter;
    p.mode = kDense;
    if (!plan_call(&p, p.a.M, ws, ws_bytes)) return false;
  }
  return true;
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

int pgemm_layer_norm_backward(pgemm_kind kind, int m, int n, pgemm_rows dY, pgemm_rows X,
                              const float* mean, const float* rstd, const void* weight,
                              pgemm_rows residual, pgemm_rows dX, void* dweight, void* dbias,
                              void* workspace, size_t workspace_bytes, void* stream) {
  if (!kind_ok(kind) || kind.act != PGEMM_ACT_NONE) return -1;
  if (!size_ok(m)) return -2;
  if (!size_ok(n)) return -3;
  const bool touch = m > 0 && n > 0, sums = dweight != nullptr || dbias != nullptr;
  const int size = size_of(kind.dtype), osize = size_of(kind.out_dtype);
  if (!rows_ok(dY, n, size, touch)) return -4;
  if (!rows_ok(X, n, size, touch)) return -5;
  if (!vector_ok(mean, 4, touch)) return -6;
  if (!vector_ok(rstd, 4, touch)) return -7;
  if (!vector_ok(weight, size, false)) return -8;
  if (!rows_ok(residual, n, size, false)) return -9;
  if (!rows_ok(dX, n, size, false)) return -10;
  if (!vector_ok(dweight, osize, false)) return -11;
  if (!vector_ok(dbias, osize, false)) return -12;
  if (sums && n > 0) {
    if (workspace == nullptr || !aligned_to(workspace, 16)) return -13;
    if (workspace_bytes < pgemm_layer_norm_backward_workspace(m, n)) return -14;
  }
  if (n == 0) return PGEMM_OK;
  const NormOps& ops = norm_ops(kind.dtype);
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
    const int groups = a.groups;
    if (a.partial == nullptr) a.groups = m < 8 * kUnits ? m : 8 * kUnits;   // (no column sums)
    const hipError_t e = ops.norm_back(a, s);
    a.groups = groups;
    if (e != hipSuccess) return PGEMM_EHIP;
  }
  if (!sums) return PGEMM_OK;
  if (a.partial == nullptr) {      // (no rows: zeros)
    a.partial = partial;
    const hipError_t e = ops.norm_sums(a, s);
    if (e != hipSuccess) return PGEMM_EHIP;
  }
  const NormColumnArgs c = {partial, dweight, dbias, n, a.groups, kind.out_dtype == PGEMM_F32};
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
  const Plan plan = plan8(m, n, k, direct, wide, workspace == nullptr ? 0 : workspace_bytes, false);
  if (plan.kernel < 0) return -2;
  a.splits = plan.splits;
  a.k_split = plan.k_split;
  a.partial = static_cast<float*>(workspace);
  set_tiles(&a, plan.kernel, kDense, m);
  if (plan.kernel >= kFew16Wide) a.tiles_n = (int)ceil_div(n, kFewWide8);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const Prod8 prod = kind.x_type == PGEMM_E4M3 ? (wide ? prod8_e4m3_wide : prod8_e4m3)
                                               : (wide ? prod8_e5m2_wide : prod8_e5m2);
  const long long far = 0x7fffffffLL / (256 * 4);   // scales' offsets within a tile fit 32 bits
  const bool whole = direct && !wide && whole_tiles(1, X.ld, W.ld) && x_scales.row_stride < far &&
                     w_scales.row_stride < far;
  return status(prod(args, kind.w_type, plan.kernel, whole ? kWhole : direct ? kDirect : kThrough, s));
}

size_t pgemm_linear_fp8_workspace(int m, int n, int k) {
  if (m <= 0 || n <= 0 || k <= 0) return 0;
  size_t most = 0;
  for (const bool direct : {false, true})
    for (const bool wide : {false, true}) {
      const size_t b = split_space(plan8(m, n, k, direct, wide, 0, true), kDense, m, 1, n);
      if (b > most) most = b;
    }
  return most;
}

int pgemm_gated_linear(pgemm_kind kind, int m, int n, int k, pgemm_rows X, pgemm_gate_weights W,
                       pgemm_gate_bias bias, pgemm_gate_rows Z, pgemm_rows Y, void* workspace,
                       size_t workspace_bytes, void* stream) {
  if (!kind_ok(kind)) return -1;
  if (!size_ok(m)) return -2;
  if (n < 0 || n > kMaxGated) return -3;
  if (!size_ok(k)) return -4;
  const bool touch = m > 0 && n > 0, read = touch && k > 0;
  const int size = size_of(kind.dtype);
  if (!rows_ok(X, k, size, read)) return -5;
  if (!gate_weights_ok(W, k, n, size, read)) return -6;
  if (!vector_ok(bias.gate, size, false) || !vector_ok(bias.up, size, false)) return -7;
  if (!rows_ok(Z.gate, n, size, false) || !rows_ok(Z.up, n, size, false)) return -8;
  if (!rows_ok(Y, n, size_of(kind.out_dtype), touch)) return -9;
  if (workspace != nullptr && !aligned_to(workspace, 16)) return -10;
  if (!touch) return PGEMM_OK;
  const int lb = W.gate.order == PGEMM_KN ? kOuter : kInner;
  int x_cols = k, inner = lb == kInner ? k : n;          // columns that may be read
  Copies pads;
  size_t space = workspace == nullptr ? 0 : workspace_bytes;
  const GateCopies copies = gate_copies(size, m, n, k, lb == kOuter);
  const bool x_whole = operand_loading(X.data, X.ld, size, k, 0) == kDirect;
  const bool w_whole = pair_loading(W, size, inner) == kDirect;
  // (both operands have to become whole)
  if (copies.total() > 0 && (x_whole || copies.x > 0) && (w_whole || copies.w > 0) &&
      space >= pgemm_gated_linear_workspace(kind.dtype, m, n, k)) {
    space -= copies.total();
    char* const to = static_cast<char*>(workspace) + space / 16 * 16;
    if (!x_whole) {
      const void* at = X.data;
      pads.add(&at, &X.ld, m, k, to);
      X.data = const_cast<void*>(at);
      x_cols = (int)X.ld;
    }
    if (!w_whole) {
      pads.add(&W.gate.data, &W.gate.ld, lb == kInner ? n : k, inner, to + copies.x);
      pads.add(&W.up.data, &W.up.ld, lb == kInner ? n : k, inner, to + copies.x + copies.w);
      inner = (int)W.gate.ld;
    }
  }
  PairArgs args{};
  ProdArgs& a = args.p;
  a.A = X.data;
  a.lda = X.ld;
  a.B = W.gate.data;
  a.ldb = W.gate.ld;
  a.D = Y.data;
  a.ldd = Y.ld;
  a.M = m;
  a.N = n;
  a.K = k;
  a.bias = bias.gate;
  a.Z = Z.gate.data;
  a.ldz = Z.gate.ld;
  a.act = kind.act;
  a.out32 = kind.out_dtype == PGEMM_F32;
  args.B2 = W.up.data;
  args.bias2 = bias.up;
  args.Z2 = Z.up.data;
  args.ldz2 = Z.up.ld;
  const int loading = both_loading(operand_loading(X.data, X.ld, size, x_cols, 0),
                                   pair_loading(W, size, inner));
  const Plan plan = gate_plan(size, m, n, k, loading, space, false);
  if (plan.kernel < 0) return -2;
  a.splits = plan.splits;
  a.k_split = plan.k_split;
  a.partial = static_cast<float*>(workspace);
  a.tiles_m = plan.kernel >= kFew16 ? 1 : (int)ceil_div(m, kShape[plan.kernel].bm);
  a.tiles_n = (int)ceil_div(n, gate_columns(plan.kernel));
  const GateOps& ops = gate_ops(kind.dtype);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (pads.count > 0 && ops.pad(pads.args, pads.count, s) != hipSuccess) return PGEMM_EHIP;
  return status(ops.pair(args, lb, kColumns, plan.kernel, loading,
                         loading == kDirect && whole_tiles(size, X.ld, W.gate.ld), s));
}

size_t pgemm_gated_linear_workspace(int dtype, int m, int n, int k) {
  if (!known(dtype) || m <= 0 || n <= 0 || n > kMaxGated || k <= 0) return 0;
  size_t most = 0;
  for (const int loading : {kThrough, kDirect}) {
    const Plan p = gate_plan(size_of(dtype), m, n, k, loading, 0, true);
    const size_t b = split_space(p, kDense, m, 1, 2 * n);
    if (b > most) most = b;
  }
  const size_t kn = gate_copies(size_of(dtype), m, n, k, true).total();
  const size_t nk = gate_copies(size_of(dtype), m, n, k, false).total();
  return align256(most) + (kn > nk ? kn : nk);
}

int pgemm_gated_linear_backward(pgemm_kind kind, int m, int n, int k, pgemm_rows dY,
                                pgemm_gate_rows Z, pgemm_rows X, pgemm_gate_weights W,
                                pgemm_rows dX, pgemm_gate_weights dW, pgemm_gate_bias dbias,
                                void* workspace, size_t workspace_bytes, void* stream) {
  if (!kind_ok(kind)) return -1;
  if (!size_ok(m)) return -2;
  if (n < 0 || n > kMaxGated) return -3;
  if (!size_ok(k)) return -4;
  const bool read = m > 0 && n > 0;
  const int size = size_of(kind.dtype), osize = size_of(kind.out_dtype);
  const bool any_dw = dW.gate.data != nullptr || dW.up.data != nullptr;
  if (!rows_ok(dY, n, size, read)) return -5;
  if (!rows_ok(Z.gate, n, size, read) || !rows_ok(Z.up, n, size, read)) return -6;
  if (!rows_ok(X, k, size, read && k > 0 && any_dw)) return -7;
  if (!gate_weights_ok(W, k, n, size, read && k > 0 && dX.data != nullptr)) return -8;
  if (!rows_ok(dX, k, size, false)) return -9;
  if (!weight_ok(dW.gate, k, n, osize, false, 1) || !weight_ok(dW.up, k, n, osize, false, 1)) return -10;
  if (!vector_ok(dbias.gate, osize, false) || !vector_ok(dbias.up, osize, false)) return -11;
  const GateSpace space = gate_space(kind, m, n, k);
  if (space.total() > 0 && (workspace == nullptr || !aligned_to(workspace, 16))) return -12;
  if (workspace_bytes < space.total()) return -13;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const GateOps& ops = gate_ops(kind.dtype);
  const bool bias = n > 0 && (dbias.gate != nullptr || dbias.up != nullptr);
  const bool want_dx = dX.data != nullptr && m > 0 && k > 0;
  const bool want_dw = any_dw && k > 0 && n > 0;
  char* const dz = static_cast<char*>(workspace);
  void* const rest = dz + space.dz;
  const long long ldz = 2LL * space.half;
  const void* const dzs[2] = {dz, dz + (size_t)space.half * (size_t)size};

  // all of the call is planned before any of it is launched
  Copies pads;
  char* const copies = dz + space.dz + space.rest;
  const int per = 16 / size;
  const bool kn = W.gate.order == PGEMM_KN;
  int inner = kn ? n : k, x_cols = k;          // columns that may be read
  if (want_dx && n > 0 && m >= pad_weight_rows(size, k % per != 0)) {
    if (inner % per && pair_loading(W, size, inner) != kDirect) {
      pads.add(&W.gate.data, &W.gate.ld, kn ? k : n, inner, copies + space.x);
      pads.add(&W.up.data, &W.up.ld, kn ? k : n, inner, copies + space.x + space.w);
      inner = (int)W.gate.ld;
    }
  }
  if (want_dw && m >= kPadRows && k % per && operand_loading(X.data, X.ld, size, k, 0) != kDirect) {
    const void* at = X.data;
    pads.add(&at, &X.ld, m, k, copies);
    X.data = const_cast<void*>(at);
    x_cols = (int)X.ld;
  }
  PairArgs dx{};
  Plan dx_plan;
  int lb = kInner, loading = kThrough;
  if (want_dx) {
    ProdArgs& a = dx.p;
    a.A = dz;
    a.lda = ldz;
    a.B = W.gate.data;
    a.ldb = W.gate.ld;
    a.D = dX.data;
    a.ldd = dX.ld;
    a.M = m;
    a.N = k;
    a.K = (int)ldz;
    dx.B2 = W.up.data;
    dx.half = space.half;
    dx.inner = n;
    lb = kn ? kInner : kOuter;
    loading = both_loading(operand_loading(dz, ldz, size, (int)ldz, 0), pair_loading(W, size, inner));
    dx_plan = plan_pair(size, kInner, m, k, (int)ldz, loading, space.rest, false);
    if (dx_plan.kernel < 0) return -2;
    a.splits = dx_plan.splits;
    a.k_split = dx_plan.k_split;
    a.partial = static_cast<float*>(rest);
    set_tiles(&a, dx_plan.kernel, kDense, m);
  }
  WeightGradients dw;
  if (want_dw && !plan_weights(&dw, kind, m, n, k, X, dzs, ldz, dW, x_cols, rest, space.rest))
    return -2;

  if (pads.count > 0 && ops.pad(pads.args, pads.count, s) != hipSuccess) return PGEMM_EHIP;
  if (n > 0 && (want_dx || want_dw || bias)) {
    GateSlopeArgs a{};
    a.dY = dY.data;
    a.ldy = dY.ld;
    a.Zg = Z.gate.data;
    a.ldg = Z.gate.ld;
    a.Zu = Z.up.data;
    a.ldu = Z.up.ld;
    a.dZ = dz;
    a.ldd = ldz;
    a.n = n;
    a.half = space.half;
    a.act = kind.act;
    a.rows = m;
    a.chunks = space.chunks;
    a.tpr = threads_per_row(space.half, 64);
    a.partial = bias ? static_cast<float*>(rest) : nullptr;
    const bool out32 = kind.out_dtype == PGEMM_F32;
    if (ops.slope(a, bias && out32, s) != hipSuccess) return PGEMM_EHIP;
    if (bias) {
      const NormColumnArgs c = {a.partial, dbias.gate, dbias.up, n, a.chunks, out32};
      if (norm_ops(kind.dtype).norm_columns(c, s) != hipSuccess) return PGEMM_EHIP;
    }
  }
  if (want_dx && ops.pair(dx, lb, kHalves, dx_plan.kernel, loading,
                          loading == kDirect && whole_tiles(size, ldz, W.gate.ld), s) != hipSuccess)
    return PGEMM_EHIP;
  if (dw.whole) return status(ops.apart(dw.args, dw.kernel, s));
  for (int i = 0; i < dw.count; ++i) {
    const int st = launch_product(dw.one[i], s);
    if (st != PGEMM_OK) return st;
  }
  return PGEMM_OK;
}

size_t pgemm_gated_linear_backward_workspace(pgemm_kind kind, int m, int n, int k) {
  if (!kind_ok(kind) || !size_ok(m) || n <= 0 || n > kMaxGated || !size_ok(k)) return 0;
  return gate_space(kind, m, n, k).total();
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
  pgemm_kind kind;
  int m, n;
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

struct GatedLinearCall {
  pgemm_kind kind;
  int m, n, k;
  pgemm_rows X;
  pgemm_gate_weights W;
  pgemm_gate_bias bias;
  pgemm_gate_rows Z;
  pgemm_rows Y;
  void* workspace;
  size_t workspace_bytes;
  void* stream;
};
struct GatedLinearBackwardCall {
  pgemm_kind kind;
  int m, n, k;
  pgemm_rows dY;
  pgemm_gate_rows Z;
  pgemm_rows X;
  pgemm_gate_weights W;
  pgemm_rows dX;
  pgemm_gate_weights dW;
  pgemm_gate_bias dbias;
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
      return pgemm_layer_norm_backward(c.kind, c.m, c.n, c.dY, c.X, c.mean, c.rstd, c.weight,
                                       c.residual, c.dX, c.dweight, c.dbias, c.workspace,
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
    case PGEMM_OP_GATED_LINEAR: {
      const GatedLinearCall& c = *static_cast<const GatedLinearCall*>(args);
      return pgemm_gated_linear(c.kind, c.m, c.n, c.k, c.X, c.W, c.bias, c.Z, c.Y, c.workspace,
                                c.workspace_bytes, c.stream);
    }
    case PGEMM_OP_GATED_LINEAR_BACKWARD: {
      const GatedLinearBackwardCall& c = *static_cast<const GatedLinearBackwardCall*>(args);
      return pgemm_gated_linear_backward(c.kind, c.m, c.n, c.k, c.dY, c.Z, c.X, c.W, c.dX, c.dW,
                                         c.dbias, c.workspace, c.workspace_bytes, c.stream);
    }
    default: return -1;
  }
}

}  // extern "C"
