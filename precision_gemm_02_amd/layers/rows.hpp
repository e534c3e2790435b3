// Row-wise kernels of the layer operators: the activation's gradient with the
// bias gradient's column sums, and the experts' rows back to their tokens.
// All of them read and write each element once and are bound by memory.  bf16:
// dZ of 8192 x 4096 37 to 47 us (201 MB: 4.3 to 5.4 TB/s; 50 with an fp32 bias
// gradient's SiLU, 53 its GELU), combine of 8192 tokens'
// 8 rows of 2048 70 us (336 MB: 4.8), its gradients for 4095 tokens' 6 rows 49 us
// (36 in a trace; 218 MB: 4.5).
#pragma once

#include "prod.hpp"

namespace pgemm {
namespace layers {

// 8 consecutive elements of a row of n, zeros behind its end.
template <typename T>
__device__ __forceinline__ void get_row8(const void* base, long long row, int c, int n, float* v) {
  if (c + 8 <= n) {
    get8<T>(base, row + c, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = c + j < n ? (float)static_cast<const T*>(base)[row + c + j] : 0.0f;
  }
}
template <typename T>
__device__ __forceinline__ void put_row8(void* base, long long row, int c, int n, const float* v) {
  if (c + 8 <= n) {
    put8<T>(base, row + c, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < n) static_cast<T*>(base)[row + c + j] = (T)v[j];
  }
}

struct SlopeArgs {
  const void* dY;
  const void* Z;          // nullptr: dZ is dY itself
  void* dZ;
  long long ldy, ldz, ldd;
  int n, act;
  const int* offsets;     // nullptr: one group of `rows` rows
  int rows;
  int chunks;             // row chunks per group (grid y)
  int tpr;                // threads per row (a power of two, at most 64)
  float* partial;         // [group][chunk][n] column sums (nullptr: not wanted)
  bool sums32;            // their results are fp32 (see Forms)
};

// dZ = dY * act'(Z) for one group's rows, one chunk of them per workgroup and
// tpr * 8 columns, and the chunk's column sums: each thread sums its rows in
// order, the threads of one column are then added in order through LDS.
template <typename T, int F>
__global__ __launch_bounds__(256) void slope_kernel(const SlopeArgs a) {
  __shared__ float sums[256 * 8];
  const int e = blockIdx.z;
  int lo = 0, hi = a.rows;
  if (a.offsets != nullptr) group_bounds(a.offsets, e, a.rows, &lo, &hi);
  const long long len = hi - lo;
  const int r0 = lo + (int)(len * blockIdx.y / a.chunks);
  const int r1 = lo + (int)(len * (blockIdx.y + 1) / a.chunks);
  const int c = (blockIdx.x * a.tpr + threadIdx.x % a.tpr) * 8;
  const int rpb = 256 / a.tpr;
  float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (c < a.n) {
#pragma unroll 2
    for (int r = r0 + threadIdx.x / a.tpr; r < r1; r += rpb) {
      float d[8];
      get_row8<T>(a.dY, (long long)r * a.ldy, c, a.n, d);
      if (a.Z != nullptr) {
        float z[8];
        get_row8<T>(a.Z, (long long)r * a.ldz, c, a.n, z);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] *= act_slope<F>(z[j], a.act);
        put_row8<T>(a.dZ, (long long)r * a.ldd, c, a.n, d);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] += d[j];
    }
  }
  if (a.partial == nullptr) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) sums[threadIdx.x * 8 + j] = s[j];
  __syncthreads();
  const int width = a.tpr * 8;
  for (int x = threadIdx.x; x < width; x += 256) {
    const int n = blockIdx.x * width + x;
    if (n >= a.n) break;
    float v = 0.0f;
    for (int r = 0; r < rpb; ++r) v += sums[r * width + x];
    a.partial[((long long)e * a.chunks + blockIdx.y) * a.n + n] = v;
  }
}

// dbias from the chunks' column sums: 32 columns per workgroup, 8 threads per
// column that each add every eighth chunk in order, then their sums in order.
template <typename T>
__global__ __launch_bounds__(256) void column_sum_kernel(const float* partial, void* out, int n,
                                                         int chunks, int out32) {
  __shared__ float sums[8][32];
  const int c = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int x = blockIdx.x * 32 + c, e = blockIdx.y;
  float v = 0.0f;
  if (x < n) {
    const float* from = partial + (long long)e * chunks * n + x;
#pragma unroll 8
    for (int s = part; s < chunks; s += 8) v += from[(long long)s * n];
  }
  sums[part][c] = v;
  __syncthreads();
  if (part != 0 || x >= n) return;
#pragma unroll
  for (int p = 1; p < 8; ++p) v += sums[p][c];
  const long long at = (long long)e * n + x;
  if (out32) static_cast<float*>(out)[at] = v;
  else static_cast<T*>(out)[at] = (T)v;
}

struct CombineArgs {
  const void* Y;
  const int* slots;
  const float* weights;
  const void* R;
  void* out;
  long long ldy, ldr, ldo;
  int m, n, top, rows;
  int tpr;                // threads per token (a power of two, at most 256)
};

template <typename T>
__global__ __launch_bounds__(256) void combine_kernel(const CombineArgs a) {
  const int t = blockIdx.x * (256 / a.tpr) + threadIdx.x / a.tpr;
  const int c = (blockIdx.y * a.tpr + threadIdx.x % a.tpr) * 8;
  if (t >= a.m || c >= a.n) return;
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  const int* slots = a.slots + (long long)t * a.top;
  const float* w = a.weights + (long long)t * a.top;
#pragma unroll 4
  for (int j = 0; j < a.top; ++j) {
    const int s = slots[j];
    if ((unsigned)s < (unsigned)a.rows) {
      const float f = a.weights != nullptr ? w[j] : 1.0f;
      float y[8];
      get_row8<T>(a.Y, (long long)s * a.ldy, c, a.n, y);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] += f * y[q];
    }
  }
  if (a.R != nullptr) {
    float r[8];
    get_row8<T>(a.R, (long long)t * a.ldr, c, a.n, r);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] += r[q];
  }
  put_row8<T>(a.out, (long long)t * a.ldo, c, a.n, v);
}

struct CombineBackArgs {
  const void* dout;
  const void* Y;
  const int* slots;
  const float* weights;
  void* dY;
  float* dweights;
  long long ldo, ldy, ldd;
  int m, n, top, rows;
};

// One wave per (token, choice): dout's row is read once per choice, but from
// the caches (a workgroup's waves work on neighbouring choices).
template <typename T>
__global__ __launch_bounds__(256) void combine_back_kernel(const CombineBackArgs a) {
  const long long id = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (id >= (long long)a.m * a.top) return;
  const int lane = threadIdx.x & 63;
  const long long t = id / a.top;
  const int s = a.slots[id];
  float dot = 0.0f;
  if ((unsigned)s < (unsigned)a.rows) {
    const float w = a.weights != nullptr ? a.weights[id] : 1.0f;
#pragma unroll 4
    for (int c = lane * 8; c < a.n; c += 512) {
      float d[8];
      get_row8<T>(a.dout, t * a.ldo, c, a.n, d);
      if (a.dweights != nullptr) {
        float y[8];
        get_row8<T>(a.Y, (long long)s * a.ldy, c, a.n, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) dot += d[j] * y[j];
      }
      if (a.dY != nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] *= w;
        put_row8<T>(a.dY, (long long)s * a.ldd, c, a.n, d);
      }
    }
  }
  if (a.dweights != nullptr) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) dot += __shfl_xor(dot, d);
    if (lane == 0) a.dweights[id] = dot;
  }
}

}  // namespace layers
}  // namespace pgemm
