// Matrix products of the layer operators: D = epilogue(A B) on gfx950 for
// bf16, fp16 and fp32 with fp32 accumulation.
//
// D is M x N with its rows contiguous.  Either operand comes in one of two
// orders: "inner" (contiguous along the summed index: A row-major, B
// column-major) or "outer" (contiguous along its own output index: A
// column-major, B row-major).  The three pairs that the layers need are
// inner/inner and inner/outer (forward, and the gradient of the input) and
// outer/outer (the gradient of the weight, summed over tokens).
//
// Grouped forms take the tokens of many experts in one launch: ROWS groups
// the rows of D (each expert's rows against its own B), SUMS groups the
// summed index (each expert's own D).  Row bounds come from device memory.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace pgemm {
namespace layers {

enum Act { kNone = 0, kRelu = 1, kGelu = 2, kGeluTanh = 3, kSilu = 4 };
enum Order { kInner = 0, kOuter = 1 };
enum Mode { kDense = 0, kRows = 1, kSums = 2 };
// How a tile's operands reach LDS (see Loader).
enum Loading { kThrough = 0, kDirect = 1, kRagged = 2 };

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// 16 bytes at an address aligned to the element only (gfx950 global memory
// accesses need no more).
struct __attribute__((packed, aligned(2))) Bytes16 {
  u32x4 v;
};

__device__ __forceinline__ u32x4 load16(const void* p) {
  return static_cast<const Bytes16*>(p)->v;
}
__device__ __forceinline__ void store16(void* p, u32x4 v) { static_cast<Bytes16*>(p)->v = v; }

// D(16 x 16) += A B: one 16-byte chunk of the summed index per lane.  Lane
// l = 16 g + i gives row i of A and column i of B, chunk g.  fp32 takes it in
// four instructions (lane group g: index 4 g + s at instruction s); both
// operands use the same order, so every product is formed once.  (32 x 32
// blocks were 2 to 4 % slower in the large tiles on random data.)
template <typename T>
struct Elem;
template <>
struct Elem<__bf16> {
  static constexpr int kMfmas = 1;
  static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
};
template <>
struct Elem<_Float16> {
  static constexpr int kMfmas = 1;
  static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
};
template <>
struct Elem<float> {
  static constexpr int kMfmas = 4;
  static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[s], y[s], c, 0, 0, 0);
    return c;
  }
};

struct ProdArgs {
  const void* A;
  const void* B;
  void* D;                // M x N; T, or fp32 when out32
  long long lda, ldb, ldd;
  int M, N, K;
  const void* bias;       // N, of T (nullptr: none)
  const void* R;          // residual of D's type (nullptr: none)
  void* Z;                // pre-activations, T (nullptr: not kept)
  long long ldr, ldz;
  int act;
  int out32;
  // groups (kRows, kSums): offsets[0..groups], each expert's own B or D
  const int* offsets;
  int groups;
  int rows;               // row capacity (R); offsets are clamped to it
  const int* gather;      // source row of A of each sorted row (nullptr: itself)
  const int* gather_b;    // the same for B (kSums)
  int gather_rows;        // valid source rows; others read as zeros
  long long strideB, strideD, strideBias;
  // the summed index over several workgroups: partial sums (fp32) of split s
  // at partial + s * M * N; the reduction runs the epilogue
  float* partial;
  int splits;
  int k_split;            // inner indices per split
  int tiles_m, tiles_n;
};

// ---- the epilogue ------------------------------------------------------------

// Activations in fp32.  tanh and the logistic function go through one exp and
// one division; the exp's argument is such that overflow gives the limit.  By the
// results' type, not the inputs':
//  * kFast, for results of 16 bits: the hardware's exp2 and reciprocal, off by
//    about |z| + 2 units of 2^-24 (of the tanh form, by its argument's), far below
//    half a step of the result (2^-8 of bf16, 2^-11 of fp16).
//  * kFine, for fp32 results of 16-bit inputs: the library's exp and the hardware's
//    reciprocal (one unit of the last place).
//  * kExact, for fp32 throughout.
enum Forms { kFast, kFine, kExact };

template <int F>
__device__ __forceinline__ float logistic(float z) {
  if constexpr (F == kFast) return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
  else if constexpr (F == kFine) return __builtin_amdgcn_rcpf(1.0f + expf(-z));
  else return 1.0f / (1.0f + expf(-z));
}

// The normal distribution function Phi and exp(-z^2/2).  The lower tail is
// computed as such: 1 + erf would cancel there.  kFast and kFine: Phi(-|z|)
// exp(z^2/2) as a polynomial in t = 1/(1 + c |z|), fitted for the least relative
// error over |z| <= 14.5 (where every result of 16 bits has become 0).  kFast: 1.2e-6,
// 1.5e-6 with fp32 coefficients; its exp adds 1.25 z^2 + 4 units of 2^-24 (its
// argument's roundings), so that Phi is off by at most 1.5e-5 of itself at z = -13.
// kFine: 1.9e-8, 8 units of 2^-24 as evaluated, and z^2/2 from the exp's argument.
// Results below the smallest normal fp32 value may be 0.
template <int F>
__device__ __forceinline__ float normal_cdf(float z, float* bell) {
  if constexpr (F == kExact) {
    *bell = expf(-0.5f * z * z);
    return 0.5f * erfcf(-0.70710678118654752f * z);
  } else {
    float e, p;
    if constexpr (F == kFast) {
      e = __builtin_amdgcn_exp2f(z * z * -0.72134752044f);   // log2(e) / 2
      const float t = __builtin_amdgcn_rcpf(1.0f + 0.26f * fabsf(z));
      p = -0.07180302f;
      p = p * t + 0.22505027f;
      p = p * t - 0.101182476f;
      p = p * t + 0.16286214f;
      p = p * t + 0.07458985f;
      p = p * t + 0.10695134f;
      p = (p * t + 0.103532486f) * t;
    } else {
      e = expf(-0.5f * z * z);
      const float t = __builtin_amdgcn_rcpf(1.0f + 0.21f * fabsf(z));
      p = -0.07129451f;
      p = p * t + 0.28180316f;
      p = p * t - 0.3264904f;
      p = p * t + 0.34498343f;
      p = p * t - 0.09077039f;
      p = p * t + 0.12347116f;
      p = p * t + 0.06956999f;
      p = p * t + 0.085012406f;
      p = (p * t + 0.08371515f) * t;
    }
    const float q = p * e;
    *bell = e;
    return z > 0.0f ? 1.0f - q : q;
  }
}

template <int F>
__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case kRelu: return z > 0.0f ? z : (z != z ? z : 0.0f);
    case kGelu: {
      float bell;
      return z * normal_cdf<F>(z, &bell);
    }
    // 0.5 (1 + tanh u) = logistic(2 u)
    case kGeluTanh:
      return z * logistic<F>(1.5957691216057308f * (z + 0.044715f * z * z * z));
    case kSilu: return z * logistic<F>(z);
    default: return z;
  }
}

// Beside Phi and the logistic function, which have their limits at infinities (and
// keep a NaN), z is taken as the nearest of [-1e4, 1e4], where every slope has long
// reached its limit of 0 or 1: past 5e19 the products of the tanh form would be 0
// times infinity, and so would all three at an infinite z, which is what a
// pre-activation beyond fp16 becomes although its activation is finite.
template <int F>
__device__ __forceinline__ float act_slope(float z, int act) {
  const float c = __builtin_amdgcn_fmed3f(z, -1e4f, 1e4f);
  switch (act) {
    case kRelu: return z > 0.0f ? 1.0f : 0.0f;
    case kGelu: {
      float bell;
      const float phi = normal_cdf<F>(z, &bell);
      return phi + c * bell * 0.39894228040143268f;
    }
    case kGeluTanh: {
      const float q = logistic<F>(1.5957691216057308f * (z + 0.044715f * z * z * z));
      return q + c * q * (1.0f - q) * 1.5957691216057308f * (1.0f + 0.134145f * c * c);
    }
    case kSilu: {
      const float q = logistic<F>(z);
      return q * (1.0f + c * (1.0f - q));
    }
    default: return 1.0f;
  }
}

// 8 consecutive elements as fp32, and back (one rounding to nearest).
template <typename T>
__device__ __forceinline__ void get8(const void* base, long long at, float* v) {
  const T* p = static_cast<const T*>(base) + at;
  if constexpr (sizeof(T) == 4) {
    const f32x4 a = __builtin_bit_cast(f32x4, load16(p)), b = __builtin_bit_cast(f32x4, load16(p + 4));
#pragma unroll
    for (int j = 0; j < 4; ++j) { v[j] = a[j]; v[4 + j] = b[j]; }
  } else {
    typedef T t8 __attribute__((ext_vector_type(8)));
    const t8 a = __builtin_bit_cast(t8, load16(p));
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (float)a[j];
  }
}
template <typename T>
__device__ __forceinline__ void put8(void* base, long long at, const float* v) {
  T* p = static_cast<T*>(base) + at;
  if constexpr (sizeof(T) == 4) {
    f32x4 a, b;
#pragma unroll
    for (int j = 0; j < 4; ++j) { a[j] = v[j]; b[j] = v[4 + j]; }
    store16(p, __builtin_bit_cast(u32x4, a));
    store16(p + 4, __builtin_bit_cast(u32x4, b));
  } else {
    typedef T t8 __attribute__((ext_vector_type(8)));
    t8 a;
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = (T)v[j];
    store16(p, __builtin_bit_cast(u32x4, a));
  }
}

// Eight residual values as they are stored (16-bit types use the first half).
struct Raw8 {
  u32x4 lo, hi;
};
template <typename T>
__device__ __forceinline__ Raw8 load_residual(const ProdArgs& a, long long m, int n0) {
  Raw8 r;
  if (sizeof(T) == 4 || a.out32) {
    const float* p = static_cast<const float*>(a.R) + m * a.ldr + n0;
    r.lo = load16(p);
    r.hi = load16(p + 4);
  } else {
    r.lo = load16(static_cast<const T*>(a.R) + m * a.ldr + n0);
    r.hi = u32x4{0, 0, 0, 0};
  }
  return r;
}
template <typename T>
__device__ __forceinline__ void add_residual(const ProdArgs& a, const Raw8& r, float* v) {
  if (sizeof(T) == 4 || a.out32) {
    const f32x4 x = __builtin_bit_cast(f32x4, r.lo), y = __builtin_bit_cast(f32x4, r.hi);
#pragma unroll
    for (int j = 0; j < 4; ++j) { v[j] += x[j]; v[4 + j] += y[j]; }
  } else if constexpr (sizeof(T) == 2) {
    typedef T t8 __attribute__((ext_vector_type(8)));
    const t8 x = __builtin_bit_cast(t8, r.lo);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += (float)x[j];
  }
}

// The switch stands outside the loops: the kernels' code stays small.
template <int F>
__device__ __forceinline__ void act8(float* v, int act) {
  switch (act) {
    case kRelu:
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = act_value<F>(v[j], kRelu);
      break;
    case kGelu:
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = act_value<F>(v[j], kGelu);
      break;
    case kGeluTanh:
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = act_value<F>(v[j], kGeluTanh);
      break;
    case kSilu:
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = act_value<F>(v[j], kSilu);
      break;
    default: break;
  }
}

// The bias of columns n0 .. n0+7, zeros where there is none.
template <typename T>
__device__ __forceinline__ void load_bias(const ProdArgs& a, const void* bias, int n0, float* b) {
#pragma unroll
  for (int j = 0; j < 8; ++j) b[j] = 0.0f;
  if (bias == nullptr) return;
  if (n0 + 8 <= a.N) {
    get8<T>(bias, n0, b);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (n0 + j < a.N) b[j] = (float)static_cast<const T*>(bias)[n0 + j];
  }
}

// Row m, columns n0 .. n0+7 of D from v, the sums with the bias added.  The
// activation sees the fp32 value; Z and D are each rounded once from it.
// `residual` holds a.R's values if there is one and all eight columns exist.
template <typename T>
__device__ __forceinline__ void finish_row(const ProdArgs& a, void* D, long long m, int n0,
                                           float* v, const Raw8& residual) {
  constexpr int Whole = sizeof(T) == 4 ? kExact : kFine;   // fp32 results
  const bool fast = sizeof(T) == 2 && !a.out32;
  const int live = a.N - n0;
  if (live >= 8) {
    if (a.Z != nullptr) put8<T>(a.Z, m * a.ldz + n0, v);
    if (a.act != kNone) {
      if (fast) act8<kFast>(v, a.act);
      else act8<Whole>(v, a.act);
    }
    if (a.R != nullptr) add_residual<T>(a, residual, v);
    if (a.out32) put8<float>(D, m * a.ldd + n0, v);
    else put8<T>(D, m * a.ldd + n0, v);
    return;
  }
#pragma unroll 1
  for (int j = 0; j < live; ++j) {
    float x = 0.0f;
#pragma unroll
    for (int q = 0; q < 8; ++q) x = q == j ? v[q] : x;   // no indexed registers
    const int n = n0 + j;
    if (a.Z != nullptr) static_cast<T*>(a.Z)[m * a.ldz + n] = (T)x;
    x = fast ? act_value<kFast>(x, a.act) : act_value<Whole>(x, a.act);
    if (a.R != nullptr)
      x += a.out32 ? static_cast<const float*>(a.R)[m * a.ldr + n]
                   : (float)static_cast<const T*>(a.R)[m * a.ldr + n];
    if (a.out32) static_cast<float*>(D)[m * a.ldd + n] = x;
    else static_cast<T*>(D)[m * a.ldd + n] = (T)x;
  }
}

// The whole epilogue of eight sums.
template <typename T>
__device__ __forceinline__ void finish8(const ProdArgs& a, const void* bias, void* D, long long m,
                                        int n0, const float* sum) {
  float v[8];
  load_bias<T>(a, bias, n0, v);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] += sum[j];
  Raw8 r{};
  if (a.R != nullptr && n0 + 8 <= a.N) r = load_residual<T>(a, m, n0);
  finish_row<T>(a, D, m, n0, v, r);
}

// ---- groups ------------------------------------------------------------------

__device__ __forceinline__ int clamp_bound(int v, int rows) {
  return v < 0 ? 0 : (v > rows ? rows : v);
}

// Rows of group e, clamped so that wrong bounds stay inside the buffers.
__device__ __forceinline__ void group_bounds(const int* offsets, int e, int rows, int* lo, int* hi) {
  const int a = clamp_bound(offsets[e], rows), b = clamp_bound(offsets[e + 1], rows);
  *lo = a;
  *hi = b > a ? b : a;
}

// The group that holds row tile t when every group takes ceil(rows / bm)
// tiles (bm 0: one, if it has rows): its index (-1: t is past the last tile),
// first row and rows left.  Every lane of the calling wave takes part and gets
// the same answer.
__device__ __forceinline__ int find_group(const int* offsets, int groups, int rows, int bm, int t,
                                          int* row, int* left) {
  const int lane = threadIdx.x & 63;
  int base = 0;
  for (int e0 = 0; e0 < groups; e0 += 64) {
    const int e = e0 + lane;
    int lo = 0, hi = 0;
    if (e < groups) group_bounds(offsets, e, rows, &lo, &hi);
    const int n = bm == 0 ? (hi > lo ? 1 : 0) : (int)(((long long)(hi - lo) + bm - 1) / bm);
    int sum = n;   // inclusive prefix sum over the wave
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(sum, d);
      if (lane >= d) sum += o;
    }
    const bool mine = t >= base + sum - n && t < base + sum;
    const unsigned long long hit = __ballot(mine);
    if (hit != 0) {
      const int src = __ffsll((long long)hit) - 1;
      const int r = lo + (t - (base + sum - n)) * bm;
      *row = __builtin_amdgcn_readfirstlane(__shfl(r, src));
      *left = __builtin_amdgcn_readfirstlane(__shfl(hi - r, src));
      return e0 + src;
    }
    base += __shfl(sum, 63);
  }
  return -1;
}

}  // namespace layers
}  // namespace pgemm
