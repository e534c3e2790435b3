// Blocks of 128 columns, of one row or of 128 rows together, to 8 bits:
//
//   s = max(largest |x| of the block / F, 2^-126),  q = x / s rounded to nearest even,
//
// F the largest number of the 8-bit type.  Divisions are the correctly rounded
// ones.  The lower limit keeps blocks of zeros, and of numbers that an fp32 scale
// could not tell from 0, without a special case.  A block that holds an infinity or
// a NaN gets NaN for its scale and its values.
//
// Bound by memory: each element is read and written once.
#pragma once

#include "../layers/prod.hpp"
#include "../layers/rows.hpp"

namespace pgemm {
namespace blocks {

using layers::get_row8;
using layers::u32x2;
using layers::u32x4;

enum Fp8 { kE4M3 = 0, kE5M2 = 1 };
constexpr int kScaleBlock = 128;

struct QuantizeArgs {
  const void* X;          // (r, c): element (i, j) at i * ldx + j, or at j * ldx + i (outer)
  uint8_t* Q;             // (r, c), rows contiguous
  float* scales;          // of block (i, j) at i * srow + j * sblock
  long long ldx, ldq, srow, sblock;
  int r, c;
  int blocks;             // blocks of a row
  bool together;          // 128 rows share a scale
  long long first;        // the launch's first workgroup (of 128 x 128)
};

template <int F>
__device__ __forceinline__ float largest() {
  return F == kE4M3 ? 448.0f : 57344.0f;
}

// The larger magnitude, a NaN once there is one.
__device__ __forceinline__ float worse(float a, float b) { return a > b || a != a ? a : b; }

template <int F>
__device__ __forceinline__ float scale_of(float top) {
  if (!(top <= 3.402823466e38f)) return __builtin_nanf("");
  const float s = top / largest<F>();
  return s > 1.17549435e-38f ? s : 1.17549435e-38f;
}

// Four and eight values over their scale, rounded to 8 bits.
template <int F>
__device__ __forceinline__ uint32_t pack4(const float* v, float s) {
  int p = 0;
  if constexpr (F == kE4M3) {
    p = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] / s, v[1] / s, p, false);
    p = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] / s, v[3] / s, p, true);
  } else {
    p = __builtin_amdgcn_cvt_pk_bf8_f32(v[0] / s, v[1] / s, p, false);
    p = __builtin_amdgcn_cvt_pk_bf8_f32(v[2] / s, v[3] / s, p, true);
  }
  return (uint32_t)p;
}

struct __attribute__((packed, aligned(1))) Bytes8 {
  u32x2 v;
};
__device__ __forceinline__ void put_bytes8(uint8_t* row, long long c, int n, u32x2 v) {
  if (c + 8 <= n) {
    reinterpret_cast<Bytes8*>(row + c)->v = v;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < n) row[c + j] = (uint8_t)(v[j >> 2] >> (8 * (j & 3)));
  }
}

__device__ __forceinline__ float top8(const float* v) {
  float m = fabsf(v[0]);
#pragma unroll
  for (int j = 1; j < 8; ++j) m = worse(m, fabsf(v[j]));
  return m;
}

// X with its rows contiguous, a scale for each row's block: 16 lanes a block.
template <typename T, int F>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const QuantizeArgs a) {
  const long long total = (long long)a.r * a.blocks;
  for (long long id = (long long)blockIdx.x * 16 + (threadIdx.x >> 4); id < total;
       id += (long long)gridDim.x * 16) {
    const long long row = id / a.blocks;
    const int b = (int)(id - row * a.blocks), c = b * kScaleBlock + (threadIdx.x & 15) * 8;
    float v[8];
    get_row8<T>(a.X, row * a.ldx, c, a.c, v);
    float top = top8(v);
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) top = worse(top, __shfl_xor(top, d));
    const float s = scale_of<F>(top);
    if ((threadIdx.x & 15) == 0) a.scales[row * a.srow + b * a.sblock] = s;
    put_bytes8(a.Q + row * a.ldq, c, a.c, u32x2{pack4<F>(v, s), pack4<F>(v + 4, s)});
  }
}

// The largest of `top` over the workgroup's 256 threads.
__device__ __forceinline__ float workgroup_top(float top, float* lds) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) top = worse(top, __shfl_xor(top, d));
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = top;
  __syncthreads();
  return worse(worse(lds[0], lds[1]), worse(lds[2], lds[3]));
}

// The same with a scale for 128 rows together: a block per workgroup, in registers.
template <typename T, int F>
__global__ __launch_bounds__(256) void quantize_blocks_kernel(const QuantizeArgs a) {
  __shared__ float lds[4];
  const long long id = a.first + blockIdx.x;
  const int i = (int)(id / a.blocks), b = (int)(id - (long long)i * a.blocks);
  const int c = b * kScaleBlock + (threadIdx.x & 15) * 8;
  float v[8][8];
  float top = 0.0f;
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const long long row = (long long)i * kScaleBlock + p * 16 + (threadIdx.x >> 4);
    get_row8<T>(a.X, row * a.ldx, row < a.r ? c : a.c, a.c, v[p]);
    top = worse(top, top8(v[p]));
  }
  const float s = scale_of<F>(workgroup_top(top, lds));
  if (threadIdx.x == 0) a.scales[i * a.srow + b * a.sblock] = s;
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const long long row = (long long)i * kScaleBlock + p * 16 + (threadIdx.x >> 4);
    if (row < a.r)
      put_bytes8(a.Q + row * a.ldq, c, a.c, u32x2{pack4<F>(v[p], s), pack4<F>(v[p] + 4, s)});
  }
}

// X with its columns contiguous: a workgroup reads 128 x 128 along the columns
// (16 lanes a column, 8 rows each), and writes rows from bytes turned in LDS.
template <typename T, int F, bool TOGETHER>
__global__ __launch_bounds__(256) void quantize_outer_kernel(const QuantizeArgs a) {
  constexpr int LD = 128 + 16;                       // bytes of a row
  __shared__ float tops[TOGETHER ? 4 : 16 * 128];
  __shared__ __attribute__((aligned(16))) uint8_t tile[128 * LD];
  const long long id = a.first + blockIdx.x;
  const int i = (int)(id / a.blocks), b = (int)(id - (long long)i * a.blocks);
  const int r0 = i * kScaleBlock, c0 = b * kScaleBlock;
  const int part = threadIdx.x & 15, lane = threadIdx.x >> 4;   // rows 8 part.., columns 8 lane..
  float v[8][8];                                     // [column][row]
  float top[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const long long col = c0 + 8 * lane + p;
    get_row8<T>(a.X, col * a.ldx, col < a.c ? r0 + 8 * part : a.r, a.r, v[p]);
#pragma unroll
    for (int j = 0; j < 8; ++j) top[j] = worse(top[j], fabsf(v[p][j]));
  }
  float s[8];
  if constexpr (TOGETHER) {
    float t = top[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) t = worse(t, top[j]);
    t = scale_of<F>(workgroup_top(t, tops));
    if (threadIdx.x == 0) a.scales[i * a.srow + b * a.sblock] = t;
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = t;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) tops[lane * 128 + 8 * part + j] = top[j];
    __syncthreads();
    if (threadIdx.x < 128) {
      float t = tops[threadIdx.x];
#pragma unroll
      for (int l = 1; l < 16; ++l) t = worse(t, tops[l * 128 + threadIdx.x]);
      t = scale_of<F>(t);
      tops[threadIdx.x] = t;
      const long long row = r0 + (int)threadIdx.x;
      if (row < a.r) a.scales[row * a.srow + b * a.sblock] = t;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = tops[8 * part + j];
  }
  // this thread's 8 columns of each of its rows
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float w[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) w[p] = v[p][j];
    *reinterpret_cast<u32x2*>(tile + (8 * part + j) * LD + 8 * lane) =
        u32x2{pack4<F>(w, s[j]), pack4<F>(w + 4, s[j])};
  }
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int row = p * 16 + (threadIdx.x >> 4);
    if (r0 + (long long)row < a.r)
      put_bytes8(a.Q + (r0 + (long long)row) * a.ldq, c0 + (threadIdx.x & 15) * 8, a.c,
                 *reinterpret_cast<const u32x2*>(tile + row * LD + (threadIdx.x & 15) * 8));
  }
}

}  // namespace blocks
}  // namespace pgemm
