// Routing to experts: scores, choice, and the plan that sorts the chosen rows
// by expert.
//
// One wave per token, the experts over its lanes.  The choice is that of 64-bit
// keys, so that it does not depend on the order of a sum or on an exp's last
// bit; the weights are computed in 64 bits and rounded to fp32 once.
//
// The plan is a counting sort that keeps token order: a workgroup takes 64
// tokens and keeps one bit per (expert, token) in LDS; a row's rank among its
// workgroup's is the number of bits below its own.  With more than one
// workgroup, a second kernel sums each expert's counts over the workgroups and
// places the rows; with more than 512, where every workgroup's own sums would
// cost more than a launch, a kernel between them sums.
//
// Bound by latency and, above 64 experts, by registers: 16384 tokens of 192 experts
// 41 us a call, where their bytes would take 3.7; of 512 128 us, of 1024 1030.  The
// 64-bit decision that few tokens take lies in the same kernel, whose 128
// registers a lane (1024 threads) then spill: 48 bytes of scratch a lane at 192
// experts, 480 at 512, 2 KB at 1024.  4 tokens take 7.4 us, which is the launch.
#pragma once

#include "prod.hpp"

namespace pgemm {
namespace layers {

constexpr int kRouteTokens = 64;    // per workgroup: one 64-bit mask per expert
constexpr int kMaxExperts = 1024;
constexpr int kMaxTop = 32;

struct RouteArgs {
  const void* logits;
  long long ld;
  const float* bias;
  int m, experts, top, score, groups, top_groups, renorm;
  float scale;
  float* weights;
  int* index;
  int* offsets;
  int* tokens;
  int* slots;
  int* counts;            // [expert][workgroup], then the prefix sums
  int* totals;            // [expert]
  int blocks;
};

template <typename T>
__device__ __forceinline__ double lowest();
template <>
__device__ __forceinline__ double lowest<float>() { return -3.4028234663852886e38; }
template <>
__device__ __forceinline__ double lowest<_Float16>() { return -65504.0; }
template <>
__device__ __forceinline__ double lowest<__bf16>() { return -3.3895313892515355e38; }

// +inf counts as the largest fp32 number, whose differences are numbers: the
// scores are their limits.
constexpr float kMaxLogit = 3.4028234663852886e38f;
__device__ __forceinline__ float finite(float x) { return x < kMaxLogit ? x : kMaxLogit; }

// A logit in 64 bits; `live` is false for masked logits and NaN.
template <typename T>
__device__ __forceinline__ double logit(const void* base, long long at, bool* live) {
  const float x = (float)static_cast<const T*>(base)[at];
  *live = (double)x > lowest<T>();
  return (double)finite(x);
}

// Reductions over the wave by DPP moves (no LDS round trips): row_shr 1, 2, 4,
// 8 leave a row's result in its lane 15, row_bcast 15 and 31 the wave's in lane
// 63.  Sums take 0 from lanes outside and leave the rows that a broadcast
// does not reach.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_or_zero(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_or_zero(double v) {
  const u32x2 x = __builtin_bit_cast(u32x2, v);
  u32x2 y;
  y[0] = (uint32_t)dpp_or_zero<CTRL, ROWS>((int)x[0]);
  y[1] = (uint32_t)dpp_or_zero<CTRL, ROWS>((int)x[1]);
  return __builtin_bit_cast(double, y);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_or_zero(float v) {
  return __builtin_bit_cast(float, dpp_or_zero<CTRL, ROWS>(__builtin_bit_cast(int, v)));
}
template <typename V>
__device__ __forceinline__ V last_lane(V v) {
  if constexpr (sizeof(V) == 4) {
    return __builtin_bit_cast(V, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
  } else {
    const u32x2 x = __builtin_bit_cast(u32x2, v);
    u32x2 y;
    y[0] = (uint32_t)__builtin_amdgcn_readlane((int)x[0], 63);
    y[1] = (uint32_t)__builtin_amdgcn_readlane((int)x[1], 63);
    return __builtin_bit_cast(V, y);
  }
}
template <typename V>
__device__ __forceinline__ V wave_sum(V v) {
  v += dpp_or_zero<0x111, 0xf>(v);
  v += dpp_or_zero<0x112, 0xf>(v);
  v += dpp_or_zero<0x114, 0xf>(v);
  v += dpp_or_zero<0x118, 0xf>(v);
  v += dpp_or_zero<0x142, 0xa>(v);
  v += dpp_or_zero<0x143, 0xc>(v);
  return last_lane(v);
}
template <int CTRL>
__device__ __forceinline__ double dpp_larger(double v) {
  const u32x2 x = __builtin_bit_cast(u32x2, v);
  u32x2 y;
  y[0] = (uint32_t)__builtin_amdgcn_update_dpp((int)x[0], (int)x[0], CTRL, 0xf, 0xf, false);
  y[1] = (uint32_t)__builtin_amdgcn_update_dpp((int)x[1], (int)x[1], CTRL, 0xf, 0xf, false);
  const double o = __builtin_bit_cast(double, y);
  return o > v ? o : v;
}
__device__ __forceinline__ double wave_max(double v) {
  v = dpp_larger<0x111>(v);
  v = dpp_larger<0x112>(v);
  v = dpp_larger<0x114>(v);
  v = dpp_larger<0x118>(v);
  v = dpp_larger<0x142>(v);
  v = dpp_larger<0x143>(v);
  return last_lane(v);
}

// The lowest expert whose key is b (the lanes hold experts lane + 64 q).
template <int Q, typename K>
__device__ __forceinline__ int lowest_with(const K (&key)[Q], K b) {
  int at = kMaxExperts;
#pragma unroll
  for (int q = Q - 1; q >= 0; --q) {
    const unsigned long long has = __ballot(key[q] == b);
    if (has != 0) at = __ffsll((long long)has) - 1 + 64 * q;
  }
  return at;
}

// Exclusive prefix sum of v over the 1024 threads; *total receives the sum.
__device__ __forceinline__ int block_scan(int v, int* scratch, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int sum = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(sum, d);
    if (lane >= d) sum += o;
  }
  if (lane == 63) scratch[wave] = sum;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) {
    const int x = scratch[w];
    before += w < wave ? x : 0;
    all += x;
  }
  *total = all;
  return before + sum - v;
}

// The wave's largest value, in every lane.
__device__ __forceinline__ int wave_max_int(int v) {
#define PGEMM_DPP_MAX(ctrl)                                              \
  {                                                                     \
    const int o = __builtin_amdgcn_update_dpp(v, v, ctrl, 0xf, 0xf, false); \
    v = o > v ? o : v;                                                  \
  }
  PGEMM_DPP_MAX(0x111)
  PGEMM_DPP_MAX(0x112)
  PGEMM_DPP_MAX(0x114)
  PGEMM_DPP_MAX(0x118)
  PGEMM_DPP_MAX(0x142)
  PGEMM_DPP_MAX(0x143)
#undef PGEMM_DPP_MAX
  return __builtin_amdgcn_readlane(v, 63);
}

// A float as an integer of the same order (-0 as +0), and back.
__device__ __forceinline__ int ordered(float x) {
  const int i = __builtin_bit_cast(int, x + 0.0f);
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i) {
  return __builtin_bit_cast(float, i ^ ((i >> 31) & 0x7fffffff));
}

constexpr int kNoKey = -0x7fffffff - 1;

// exp(x) to about 1e-14, x within +-1000 (beyond, that of the limit): the
// series to degree 12 on |r| <= ln 2 / 2 (the next term is below 2e-16).
__device__ __forceinline__ double exp64(double x) {
  x = x < -1000.0 ? -1000.0 : (x > 1000.0 ? 1000.0 : x);
  const double n = __builtin_rint(x * 1.4426950408889634074);
  // ln 2 as its nearest 64-bit number and the rest; the fma forms n times the first
  // without a rounding, so that it need not be short
  double r = __builtin_fma(n, -0.6931471805599453, x);
  r = __builtin_fma(n, -2.3190468138462996e-17, r);
  double p = 1.0 / 479001600.0;
  p = __builtin_fma(p, r, 1.0 / 39916800.0);
  p = __builtin_fma(p, r, 1.0 / 3628800.0);
  p = __builtin_fma(p, r, 1.0 / 362880.0);
  p = __builtin_fma(p, r, 1.0 / 40320.0);
  p = __builtin_fma(p, r, 1.0 / 5040.0);
  p = __builtin_fma(p, r, 1.0 / 720.0);
  p = __builtin_fma(p, r, 1.0 / 120.0);
  p = __builtin_fma(p, r, 1.0 / 24.0);
  p = __builtin_fma(p, r, 1.0 / 6.0);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  p = __builtin_fma(p, r, 1.0);
  return __builtin_amdgcn_ldexp(p, (int)n);
}

// 1 / d for d in [1, 1e300]: the hardware's estimate and two Newton steps.
__device__ __forceinline__ double reciprocal64(double d) {
  double y = __builtin_amdgcn_rcp(d);
  y = __builtin_fma(y, __builtin_fma(-d, y, 1.0), y);
  return __builtin_fma(y, __builtin_fma(-d, y, 1.0), y);
}

// (that of -690, 1e-300, for all below)
__device__ __forceinline__ double sigmoid64(double x) {
  return reciprocal64(1.0 + exp64(x < -690.0 ? 690.0 : -x));
}

template <int CTRL>
__device__ __forceinline__ int dpp_move(int v) {
  return __builtin_amdgcn_update_dpp(v, v, CTRL, 0xf, 0xf, false);
}

// The two largest of two pairs, each largest first.
__device__ __forceinline__ void join(int& a1, int& a2, int b1, int b2) {
  const int lo = a1 < b1 ? a1 : b1, second = a2 > b2 ? a2 : b2;
  a1 = a1 > b1 ? a1 : b1;
  a2 = lo > second ? lo : second;
}

// A key as an integer; masked where it is not live, and so is a bias that
// makes it infinite, NaN or larger than 3e38.
__device__ __forceinline__ int to_key(double k, double per_unit, bool live) {
  return live && fabs(k) < (double)3.0e38f ? (int)__builtin_rint(k * per_unit) : kNoKey;
}

// One token's keys in 64 bits and its choice: lane j returns choice j (-1:
// none).  Taken where fp32 keys are too close to decide (see route_kernel).
template <typename T, int Q>
__device__ __forceinline__ int choose64(const RouteArgs& a, long long t) {
  const int lane = threadIdx.x & 63;
  const double none = -__builtin_inf();
  double key[Q], x[Q], top = none;
  bool live[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int e = lane + 64 * q;
    live[q] = false;
    x[q] = 0;
    if (e < a.experts) x[q] = logit<T>(a.logits, t * a.ld + e, &live[q]);
    if (live[q] && x[q] > top) top = x[q];
  }
  if (a.score == 0) {
    top = wave_max(top);
    double sum = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      key[q] = live[q] ? exp(x[q] - top) : 0.0;
      sum += key[q];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int q = 0; q < Q; ++q) key[q] = sum > 0 ? key[q] / sum : 0.0;
  } else {
#pragma unroll
    for (int q = 0; q < Q; ++q) key[q] = live[q] ? 1.0 / (1.0 + exp(-x[q])) : 0.0;
  }
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int e = lane + 64 * q;
    if (a.bias != nullptr && e < a.experts) key[q] += (double)a.bias[e];
    // (a bias that is infinite, NaN or beyond 3e38 masks its expert)
    if (!live[q] || !(fabs(key[q]) < (double)3.0e38f)) key[q] = none;
  }
  if (a.top_groups < a.groups) {
    const int size = a.experts / a.groups;
    double mine = none;       // lane g: the sum of group g's two best keys
    for (int g = 0; g < a.groups; ++g) {
      double in[Q], b1 = none, b2 = none;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        in[q] = (lane + 64 * q) / size == g ? key[q] : none;
        b1 = in[q] > b1 ? in[q] : b1;
      }
      b1 = wave_max(b1);
      const int i1 = lowest_with(in, b1);
#pragma unroll
      for (int q = 0; q < Q; ++q)
        if (lane + 64 * q != i1 && in[q] > b2) b2 = in[q];
      b2 = wave_max(b2);
      if (lane == g) mine = b2 > none ? b1 + b2 : b1;
    }
    unsigned long long keep = 0;
    for (int j = 0; j < a.top_groups; ++j) {
      const double b = wave_max(mine);
      if (!(b > none)) break;
      const int i = __ffsll((long long)__ballot(mine == b)) - 1;
      keep |= 1ull << i;
      if (lane == i) mine = none;
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int g = (lane + 64 * q) / size;
      if (g >= 64 || !((keep >> g) & 1)) key[q] = none;
    }
  }
  int pick = -1;
  for (int j = 0; j < a.top; ++j) {
    double b = none;
#pragma unroll
    for (int q = 0; q < Q; ++q) b = key[q] > b ? key[q] : b;
    b = wave_max(b);
    if (!(b > none)) break;
    const int i = lowest_with(key, b);
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (lane + 64 * q == i) key[q] = none;
    if (lane == j) pick = i;
  }
  return pick;
}

// Scores, choice, and the ranks within the workgroup's 64 tokens; the whole
// plan if there is only one workgroup.  Q: experts per lane.
//
// The choice is that of 64-bit keys, found in up to three ways.  Keys are
// compared as integers of 2^29 / (1 + the largest bias) per unit of key.
//  * From fp32 scores: off by less than 2e-6 (the exp's argument and result and
//    the sum, each a few 2^-24, |d| exp(d) < 0.37) and the bias's addition by
//    less than 1.2e-7 of the largest key.  Integers further apart than both
//    errors of two keys (`near`), or sums of two keys further than 3 of that,
//    are in the 64-bit order.
//  * Where two that are compared for the result (neighbours among the best
//    top + 1, or the last group in and the first one out) are closer: again
//    from 64-bit scores (to about 1e-13), integers off by half.
//  * Where those are still within 2 (sums: 6): by the 64-bit keys themselves.
// A key that is the logit itself is compared as the exact fp32 value.
// (16384 tokens of 192 experts in 6 groups: 64-bit comparisons throughout 89
// us; 64-bit scores throughout 53; from fp32 scores straight to 64-bit
// comparisons, which 0.2 % of the tokens then waited for, 58.  That is for fp32
// logits with a bias.  Equal logits without one have equal keys, which no integers
// tell apart: 16-bit logits of 256 experts in 8 groups take 119 us, with a bias 59.)
template <typename T, int Q>
__global__ __launch_bounds__(1024) void route_kernel(const RouteArgs a) {
  __shared__ unsigned int mask[2 * kMaxExperts];      // [half of the tokens][expert]
  __shared__ int chosen[kRouteTokens * kMaxTop];
  __shared__ int base[kMaxExperts];
  __shared__ int scratch[16];
  __shared__ int keys[16][64 * Q];                    // a wave's keys, by expert
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t0 = blockIdx.x * kRouteTokens;
  const bool logit_key = a.groups == 1 && a.bias == nullptr;
  const bool grouped = a.top_groups < a.groups;
  const int size = a.experts / a.groups;
  // lanes per group, a power of two
  int lpg = 1;
  while (lpg * 2 * a.groups <= 64) lpg *= 2;
  const int my_group = lane / lpg, my_sub = lane % lpg;
  int group_bit[Q];                                   // of the lane's experts
  float bias[Q], most_bias = 0.0f;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int e = lane + 64 * q;
    group_bit[q] = e < a.experts ? (e / size) * lpg : 0;
    bias[q] = a.bias != nullptr && e < a.experts ? a.bias[e] : 0.0f;
    // (an infinite or NaN bias masks its expert)
    const float m = fabsf(bias[q]);
    most_bias = m > most_bias && m < 3.0e38f ? m : most_bias;
  }
  most_bias = unordered(wave_max_int(ordered(most_bias)));
  const double per_unit = 536870912.0 / (1.0 + (double)most_bias);
  // see above: the sum of both fp32 errors, in integers
  const int coarse_near = 2 + (int)((4e-6 + 2.4e-7 * (1.0 + (double)most_bias)) * per_unit);

  for (int x = threadIdx.x; x < 2 * a.experts; x += 1024) mask[x] = 0;
  __syncthreads();

  const auto fetch = [&](int tt, T(&into)[Q]) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int e = lane + 64 * q;
      if (e < a.experts && tt < kRouteTokens && t0 + tt < a.m)
        into[q] = static_cast<const T*>(a.logits)[(long long)(t0 + tt) * a.ld + e];
    }
  };
  T next[Q];
  fetch(wave, next);
  for (int tt = wave; tt < kRouteTokens && t0 + tt < a.m; tt += 16) {
    const long long t = t0 + tt;
    float x[Q];
    int key[Q];                 // kNoKey: not to be chosen
    int top = kNoKey;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int e = lane + 64 * q;
      x[q] = 0;
      key[q] = kNoKey;
      if (e < a.experts) {
        x[q] = (float)next[q];
        if ((double)x[q] > lowest<T>()) {
          x[q] = finite(x[q]);
          key[q] = ordered(x[q]);
        }
      }
      top = key[q] > top ? key[q] : top;
    }
    fetch(tt + 16, next);       // the wave's next token, during this one
    unsigned live = 0;          // bit q: expert lane + 64 q is not masked
#pragma unroll
    for (int q = 0; q < Q; ++q) live |= key[q] != kNoKey ? 1u << q : 0u;
    // lane j: choice j and its logit
    int pick;
    float chosen_x;
    for (bool fine = false;; fine = true) {
      int near = 0;               // integers no further apart than this are not in order
      if (!logit_key) {
        if (!fine) {
          near = coarse_near;
          float score[Q];
          if (a.score == 0) {
            const float mx = unordered(wave_max_int(top));
            float sum = 0;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
              score[q] = (live >> q) & 1 ? __expf(x[q] - mx) : 0.0f;
              sum += score[q];
            }
            sum = wave_sum(sum);
            const float inv = sum > 0 ? 1.0f / sum : 0.0f;
#pragma unroll
            for (int q = 0; q < Q; ++q) score[q] *= inv;
          } else {
#pragma unroll
            for (int q = 0; q < Q; ++q) score[q] = logistic<kFast>(x[q]);
          }
#pragma unroll
          for (int q = 0; q < Q; ++q)
            key[q] = to_key((double)(score[q] + bias[q]), per_unit, (live >> q) & 1);
        } else {
          near = 2;
          double score[Q];
          if (a.score == 0) {
            const double mx = (double)unordered(wave_max_int(top));
            double sum = 0;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
              score[q] = (live >> q) & 1 ? exp64((double)x[q] - mx) : 0.0;
              sum += score[q];
            }
            sum = wave_sum(sum);
            const double inv = sum > 0 ? reciprocal64(sum) : 0.0;
#pragma unroll
            for (int q = 0; q < Q; ++q) score[q] *= inv;
          } else {
#pragma unroll
            for (int q = 0; q < Q; ++q) score[q] = sigmoid64((double)x[q]);
          }
#pragma unroll
          for (int q = 0; q < Q; ++q)
            key[q] = to_key(score[q] + (double)bias[q], per_unit, (live >> q) & 1);
        }
      }
      bool unclear = false;
      if (grouped) {
#pragma unroll
        for (int q = 0; q < Q; ++q) keys[wave][lane + 64 * q] = key[q];
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        int m1 = kNoKey, m2 = kNoKey;
        if (my_group < a.groups) {
          const int* from = keys[wave] + my_group * size;
          for (int i = my_sub; i < size; i += 4 * lpg) {
            int k[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int at = i + u * lpg;
              k[u] = from[at < size ? at : i];
              if (at >= size) k[u] = kNoKey;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) join(m1, m2, k[u], kNoKey);
          }
        }
        // over the group's lanes: neighbours, pairs, quads (mirrored within 8),
        // eights (mirrored within 16) by DPP, then through LDS
        if (lpg > 1) join(m1, m2, dpp_move<0xB1>(m1), dpp_move<0xB1>(m2));
        if (lpg > 2) join(m1, m2, dpp_move<0x4E>(m1), dpp_move<0x4E>(m2));
        if (lpg > 4) join(m1, m2, dpp_move<0x141>(m1), dpp_move<0x141>(m2));
        if (lpg > 8) join(m1, m2, dpp_move<0x140>(m1), dpp_move<0x140>(m2));
        if (lpg > 16) join(m1, m2, __shfl_xor(m1, 16), __shfl_xor(m2, 16));
        int sum = kNoKey;
        if (m1 != kNoKey) sum = m1 + (m2 == kNoKey ? 0 : m2);
        int rank = 0;
        for (int g = 0; g < a.groups; ++g) {
          const int o = __builtin_amdgcn_readlane(sum, g * lpg);
          rank += o > sum || (o == sum && g < my_group) ? 1 : 0;
        }
        const bool first = my_sub == 0 && my_group < a.groups;
        const unsigned long long keep = __ballot(first && sum != kNoKey && rank < a.top_groups);
        const unsigned long long in = __ballot(first && rank == a.top_groups - 1),
                                 out = __ballot(first && rank == a.top_groups);
        const int vi = __builtin_amdgcn_readlane(sum, __ffsll((long long)in) - 1),
                  vo = __builtin_amdgcn_readlane(sum, __ffsll((long long)out) - 1);
        // (vi >= vo; sums reach +-2^30, so that the difference needs 32 bits unsigned)
        unclear = vo != kNoKey && (unsigned)vi - (unsigned)vo <= 3u * (unsigned)near;
#pragma unroll
        for (int q = 0; q < Q; ++q)
          if (!((keep >> group_bit[q]) & 1)) key[q] = kNoKey;
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        __builtin_amdgcn_wave_barrier();
      }
      // the best `top` of them, best first; lane j keeps choice j.  One more
      // round checks that the next key is clearly behind.
      int last = kNoKey;
      pick = -1;
      chosen_x = -__builtin_inff();
      const int rounds = a.top + (logit_key ? 0 : 1);
      for (int j = 0; j < rounds; ++j) {
        int b = key[0];
#pragma unroll
        for (int q = 1; q < Q; ++q) b = key[q] > b ? key[q] : b;
        b = wave_max_int(b);
        if (b == kNoKey) break;
        // (logits as keys are exact, and their difference can pass 32 bits)
        if (!logit_key && j > 0 && last - b <= near) unclear = true;
        last = b;
        if (j == a.top) break;
        bool done = false;                       // the lowest index that has it
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const unsigned long long has = __ballot(key[q] == b);
          if (!done && has != 0) {
            const int src = __ffsll((long long)has) - 1;
            if (lane == src) key[q] = kNoKey;
            const float at = __builtin_bit_cast(
                float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x[q]), src));
            if (lane == j) {
              pick = src + 64 * q;
              chosen_x = at;
            }
            done = true;
          }
        }
      }
      if (!unclear) break;
      if (fine) {
        pick = choose64<T, Q>(a, t);
        bool in = false;
        chosen_x = pick >= 0 ? (float)logit<T>(a.logits, t * a.ld + pick, &in) : -__builtin_inff();
        break;
      }
    }

    // the chosen scores in 64 bits
    double w = 0;
    const double px = (double)chosen_x;
    if (a.score != 0) {
      // far below 0 the sigmoid is exp(x), whose ratios no shift changes: where all
      // scores would underflow, the largest logit is taken as -600
      double shift = 0;
      if (a.renorm && __ballot(pick >= 0 && chosen_x >= -600.0f) == 0)
        shift = (double)unordered(wave_max_int(ordered(chosen_x))) + 600.0;
      w = pick >= 0 ? sigmoid64(px - shift) : 0.0;
      if (a.renorm) {
        const double sum = wave_sum(w);
        w = sum > 0 ? w / sum : 0.0;
      }
    } else if (a.renorm) {                     // a softmax of the chosen logits
      const double mx = (double)unordered(wave_max_int(ordered(chosen_x)));
      w = pick >= 0 ? exp64(px - mx) : 0.0;
      const double sum = wave_sum(w);
      w = sum > 0 ? w / sum : 0.0;
    } else {
      const double mx = (double)unordered(wave_max_int(top));
      double sum = 0;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int e = lane + 64 * q;
        const bool in = e < a.experts && (double)x[q] > lowest<T>();
        if (in) sum += exp64((double)x[q] - mx);
      }
      sum = wave_sum(sum);
      w = pick >= 0 ? exp64(px - mx) / sum : 0.0;
    }
    if (lane < a.top) {
      a.weights[t * a.top + lane] = (float)(w * (double)a.scale);
      a.index[t * a.top + lane] = pick;
      chosen[tt * a.top + lane] = pick;
      if (pick >= 0) atomicOr(&mask[(tt >> 5) * a.experts + pick], 1u << (tt & 31));
    }
  }
  __syncthreads();

  // counts per expert; with one workgroup also the offsets
  const int e = threadIdx.x;
  const int count = e < a.experts ? __popc(mask[e]) + __popc(mask[a.experts + e]) : 0;
  if (a.blocks > 1) {
    if (e < a.experts) {
      a.counts[(long long)e * a.blocks + blockIdx.x] = count;
      base[e] = 0;
    }
  } else {
    int total;
    const int at = block_scan(count, scratch, &total);
    if (e < a.experts) {
      base[e] = at;
      a.offsets[e] = at;
    }
    if (e == 0) a.offsets[a.experts] = total;
  }
  __syncthreads();
  const int live_tokens = a.m - t0 < kRouteTokens ? a.m - t0 : kRouteTokens;
  for (int x = threadIdx.x; x < live_tokens * a.top; x += 1024) {
    const int tt = x / a.top, p = chosen[x];
    int slot = -1;
    if (p >= 0) {
      const unsigned below = (1u << (tt & 31)) - 1;
      slot = base[p] + (tt < 32 ? __popc(mask[p] & below)
                                : __popc(mask[p]) + __popc(mask[a.experts + p] & below));
      if (a.blocks == 1) a.tokens[slot] = t0 + tt;
    }
    a.slots[(long long)t0 * a.top + x] = slot;
  }
}

// Each expert's counts become its workgroups' first ranks: one wave per expert.
template <typename T>
__global__ __launch_bounds__(64) void route_sum_kernel(const RouteArgs a) {
  int* c = a.counts + (long long)blockIdx.x * a.blocks;
  const int lane = threadIdx.x;
  int base = 0;
  for (int b0 = 0; b0 < a.blocks; b0 += 64) {
    const int b = b0 + lane;
    const int v = b < a.blocks ? c[b] : 0;
    int sum = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(sum, d);
      if (lane >= d) sum += o;
    }
    if (b < a.blocks) c[b] = base + sum - v;
    base += __shfl(sum, 63);
  }
  if (lane == 0) a.totals[blockIdx.x] = base;
}

// Rows to their places.  Every workgroup scans the experts' totals itself,
// and (SUM) first sums each expert's counts, one wave per expert.
template <typename T, bool SUM>
__global__ __launch_bounds__(1024) void route_place_kernel(const RouteArgs a) {
  __shared__ int base[kMaxExperts], totals[kMaxExperts];
  __shared__ int scratch[16];
  const int e = threadIdx.x;
  if constexpr (SUM) {
    const int lane = threadIdx.x & 63;
    // four experts of a wave at once, for the latency of the reductions
    for (int x0 = (threadIdx.x >> 6) * 4; x0 < a.experts; x0 += 64) {
      int before[4] = {0, 0, 0, 0}, all[4] = {0, 0, 0, 0};
#pragma unroll 4
      for (int b = lane; b < a.blocks; b += 64) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int x = x0 + u < a.experts ? x0 + u : a.experts - 1;
          const int v = a.counts[(long long)x * a.blocks + b];
          all[u] += v;
          before[u] += b < (int)blockIdx.x ? v : 0;
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        all[u] = wave_sum(all[u]);
        before[u] = wave_sum(before[u]);
      }
      if (lane < 4 && x0 + lane < a.experts) {
        totals[x0 + lane] = lane == 0 ? all[0] : lane == 1 ? all[1] : lane == 2 ? all[2] : all[3];
        base[x0 + lane] =
            lane == 0 ? before[0] : lane == 1 ? before[1] : lane == 2 ? before[2] : before[3];
      }
    }
    __syncthreads();
  }
  int total;
  const int mine = e < a.experts ? (SUM ? totals[e] : a.totals[e]) : 0;
  const int at = block_scan(mine, scratch, &total);
  if (e < a.experts) {
    base[e] = at + (SUM ? base[e] : a.counts[(long long)e * a.blocks + blockIdx.x]);
    if (blockIdx.x == 0) a.offsets[e] = at;
  }
  if (e == 0 && blockIdx.x == 0) a.offsets[a.experts] = total;
  __syncthreads();
  const int t0 = blockIdx.x * kRouteTokens;
  const int live_tokens = a.m - t0 < kRouteTokens ? a.m - t0 : kRouteTokens;
  for (int x = threadIdx.x; x < live_tokens * a.top; x += 1024) {
    const long long i = (long long)t0 * a.top + x;
    const int p = a.index[i];
    if (p >= 0) {
      const int slot = base[p] + a.slots[i];
      a.slots[i] = slot;
      a.tokens[slot] = t0 + x / a.top;
    }
  }
}

struct RouteBackArgs {
  const float* dweights;
  const void* logits;
  const int* index;
  void* dlogits;
  long long ld, ldd;
  int m, experts, top, score, renorm;
  float scale;
};

// One wave per token.  With p the scores, P the chosen ones, g the weights'
// gradients times scale: renorm: ds_j = (g_j - sum_i g_i P_i / S) / S with
// S the sum of P, otherwise ds_j = g_j; then through the sigmoid,
// ds p (1 - p), or the softmax, p (ds - sum_i p_i ds_i).  The softmax
// renormalised is a softmax of the chosen logits alone, which is how it is
// computed, and the renormalised sigmoid likewise: no score underflows.
template <typename T, int Q>
__global__ __launch_bounds__(256) void route_back_kernel(const RouteBackArgs a) {
  const long long t = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= a.m) return;
  const int lane = threadIdx.x & 63;
  float x[Q], top = -__builtin_inff();
  bool live[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int e = lane + 64 * q;
    live[q] = false;
    x[q] = 0;
    if (e < a.experts) {
      const float l = (float)static_cast<const T*>(a.logits)[t * a.ld + e];
      live[q] = (double)l > lowest<T>();
      x[q] = finite(l);
    }
    if (live[q] && x[q] > top) top = x[q];
  }
  // lane j: choice j
  int pick = -1;
  float g = 0;
  if (lane < a.top) {
    pick = a.index[t * a.top + lane];
    g = a.dweights[t * a.top + lane] * a.scale;
    if ((unsigned)pick >= (unsigned)a.experts) pick = -1;
  }
  // the chosen logits
  float px = 0;
  bool plive = false;
  if (pick >= 0) {
    const float l = (float)static_cast<const T*>(a.logits)[t * a.ld + pick];
    plive = (double)l > lowest<T>();
    px = finite(l);
  }
  if (!plive) { pick = -1; g = 0; }

  float d;                      // lane j: what choice j adds to its logit
  float inner = 0, sum_all = 1, top_all = 0;
  auto wsum = [](float v) {
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) v += __shfl_xor(v, s);
    return v;
  };
  auto wmax = [](float v) {
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) v = fmaxf(v, __shfl_xor(v, s));
    return v;
  };
  if (a.score == 0 && a.renorm) {
    const float mx = wmax(plive ? px : -__builtin_inff());
    float p = plive ? expf(px - mx) : 0.0f;
    const float s = wsum(p);
    p = s > 0 ? p / s : 0.0f;
    d = p * (g - wsum(p * g));
  } else if (a.score == 0) {
    top_all = wmax(top);
    float s = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (live[q]) s += expf(x[q] - top_all);
    sum_all = wsum(s);
    const float p = plive ? expf(px - top_all) / sum_all : 0.0f;
    d = p * g;
    inner = wsum(d);
  } else {
    // 1 - p without cancellation
    const float not_p = plive ? 1.0f / (1.0f + expf(px)) : 0.0f;
    if (a.renorm) {
      // sigmoid(x) = exp(min(x, 0)) / (1 + exp(-|x|)): the sum's ratios keep with
      // the largest exp taken out of them, also where every score underflows
      const float low = fminf(px, 0.0f), c = wmax(plive ? low : -__builtin_inff());
      const float p = plive ? expf(low - c) / (1.0f + expf(-fabsf(px))) : 0.0f;
      const float s = wsum(p);
      const float r = s > 0 ? p / s : 0.0f;
      d = r * (g - wsum(r * g)) * not_p;
    } else {
      const float p = plive ? 1.0f / (1.0f + expf(-px)) : 0.0f;
      d = g * p * not_p;
    }
  }
  float out[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    out[q] = 0;
    if (a.score == 0 && !a.renorm && live[q]) out[q] = -inner * (expf(x[q] - top_all) / sum_all);
  }
  for (int j = 0; j < a.top; ++j) {
    const int e = __shfl(pick, j);
    const float v = __shfl(d, j);
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (e == lane + 64 * q) out[q] += v;
  }
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int e = lane + 64 * q;
    if (e < a.experts) static_cast<T*>(a.dlogits)[t * a.ldd + e] = (T)out[q];
  }
}

}  // namespace layers
}  // namespace pgemm
