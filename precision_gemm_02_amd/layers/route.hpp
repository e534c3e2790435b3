// Routing to experts: scores, choice, and the plan that sorts the chosen rows
// by expert.
//
// One wave per token, the experts over its lanes.  Scores and keys are
// computed in 64 bits, so that the choice does not depend on the order of a
// sum or on an exp's last bit; the weights are rounded to fp32 once.
//
// The plan is a counting sort that keeps token order: a workgroup takes 64
// tokens and keeps one bit per (expert, token) in LDS; a row's rank among its
// workgroup's is the number of bits below its own.  With more than one
// workgroup, a second kernel sums each expert's counts over the workgroups and
// a third places the rows.
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

// A logit in 64 bits, +inf as a large finite number (its score is then the
// limit); `live` is false for masked logits and NaN.
template <typename T>
__device__ __forceinline__ double logit(const void* base, long long at, bool* live) {
  const double x = (double)(float)static_cast<const T*>(base)[at];
  *live = x > lowest<T>();
  return x < 1e300 ? x : 1e300;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const double o = __shfl_xor(v, d);
    v = o > v ? o : v;
  }
  return v;
}

// The wave's largest (key, then lowest index).
__device__ __forceinline__ void wave_best(double* key, int* index) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const double k = __shfl_xor(*key, d);
    const int i = __shfl_xor(*index, d);
    const bool take = k > *key || (k == *key && i < *index);
    *key = take ? k : *key;
    *index = take ? i : *index;
  }
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

// Scores, choice, and the ranks within the workgroup's 64 tokens; the whole
// plan if there is only one workgroup.  Q: experts per lane.
template <typename T, int Q>
__global__ __launch_bounds__(1024) void route_kernel(const RouteArgs a) {
  __shared__ unsigned int mask[2 * kMaxExperts];      // [half of the tokens][expert]
  __shared__ int chosen[kRouteTokens * kMaxTop];
  __shared__ int base[kMaxExperts];
  __shared__ int scratch[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t0 = blockIdx.x * kRouteTokens;
  const double none = -__builtin_inf();

  for (int x = threadIdx.x; x < 2 * a.experts; x += 1024) mask[x] = 0;
  __syncthreads();

  for (int tt = wave; tt < kRouteTokens && t0 + tt < a.m; tt += 16) {
    const long long t = t0 + tt;
    double x[Q], key[Q], top = none;
    bool live[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int e = lane + 64 * q;
      live[q] = false;
      x[q] = 0;
      if (e < a.experts) x[q] = logit<T>(a.logits, t * a.ld + e, &live[q]);
      if (live[q] && x[q] > top) top = x[q];
    }
    // scores (0 where masked)
    double score[Q];
    if (a.score == 0) {
      top = wave_max(top);
      double sum = 0;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        score[q] = live[q] ? exp(x[q] - top) : 0.0;
        sum += score[q];
      }
      sum = wave_sum(sum);
#pragma unroll
      for (int q = 0; q < Q; ++q) score[q] = sum > 0 ? score[q] / sum : 0.0;
    } else {
#pragma unroll
      for (int q = 0; q < Q; ++q) score[q] = live[q] ? 1.0 / (1.0 + exp(-x[q])) : 0.0;
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int e = lane + 64 * q;
      double k = a.groups == 1 && a.bias == nullptr ? x[q] : score[q];
      if (a.bias != nullptr && e < a.experts) k += (double)a.bias[e];
      // a bias of -inf or NaN masks its expert too
      live[q] = live[q] && k > none;
      key[q] = live[q] ? k : none;
    }
    if (a.top_groups < a.groups) {
      // each group's two best keys, one group at a time
      const int size = a.experts / a.groups;
      double mine = none;       // lane g: group g's sum
      for (int g = 0; g < a.groups; ++g) {
        double b1 = none;
        int i1 = kMaxExperts;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const int e = lane + 64 * q;
          if (e / size == g && key[q] > b1) { b1 = key[q]; i1 = e; }
        }
        wave_best(&b1, &i1);
        double b2 = none;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const int e = lane + 64 * q;
          if (e / size == g && e != i1 && key[q] > b2) b2 = key[q];
        }
        b2 = wave_max(b2);
        if (lane == g) mine = b2 > none ? b1 + b2 : b1;
      }
      unsigned long long keep = 0;
      for (int j = 0; j < a.top_groups; ++j) {
        double b = mine;
        int i = lane;
        wave_best(&b, &i);
        if (b > none) keep |= 1ull << i;
        if (lane == i) mine = none;
      }
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int g = (lane + 64 * q) / size;
        if (g >= 64 || !((keep >> g) & 1)) key[q] = none;
      }
    }
    // the best `top` of them; lane j keeps choice j
    int pick = -1;
    double w = 0;
    for (int j = 0; j < a.top; ++j) {
      double b = none;
      int i = kMaxExperts;
#pragma unroll
      for (int q = 0; q < Q; ++q)
        if (key[q] > b) { b = key[q]; i = lane + 64 * q; }
      wave_best(&b, &i);
      double s = 0;
#pragma unroll
      for (int q = 0; q < Q; ++q)
        if (lane + 64 * q == i) { s = score[q]; key[q] = none; }
      s = __shfl(s, i & 63);
      if (lane == j && b > none) { pick = i; w = s; }
    }
    if (a.renorm) {
      const double sum = wave_sum(w);
      w = sum > 0 ? w / sum : 0.0;
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

// Rows to their places: every workgroup scans the experts' totals itself.
template <typename T>
__global__ __launch_bounds__(1024) void route_place_kernel(const RouteArgs a) {
  __shared__ int base[kMaxExperts];
  __shared__ int scratch[16];
  const int e = threadIdx.x;
  int total;
  const int at = block_scan(e < a.experts ? a.totals[e] : 0, scratch, &total);
  if (e < a.experts) {
    base[e] = at + a.counts[(long long)e * a.blocks + blockIdx.x];
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
// computed: no score underflows.
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
      x[q] = l < 3.0e38f ? l : 3.0e38f;
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
    px = l < 3.0e38f ? l : 3.0e38f;
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
    const float p = plive ? 1.0f / (1.0f + expf(-px)) : 0.0f;
    // 1 - p without cancellation
    const float not_p = plive ? 1.0f / (1.0f + expf(px)) : 0.0f;
    if (a.renorm) {
      const float s = wsum(p);
      const float r = s > 0 ? p / s : 0.0f;
      d = r * (g - wsum(r * g)) * not_p;
    } else {
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
