// Blocks of 128 columns, of one row or of 128 rows together, to 8 bits:
//
//   s = max(largest |x| of the block / F, 2^-126),  q = x / s rounded to nearest even,
//
// F the largest number of the 8-bit type.  Quotients are correctly rounded before their
// rounding to 8 bits.  The lower limit keeps blocks of zeros, and of numbers that an fp32 scale
// could not tell from 0, without a special case.  A block that holds an infinity or
// a NaN gets NaN for its scale and its values.
//
// Bound by memory: each element is read and written once.  Scales of rows, 8192 x 4096 bf16:
// 21.2 us (101 MB: 4.8 TB/s; a copy reaches 5.0); blocks of 128 x 128 of 4096^2 fp32, in
// columns: 16.5 us (84 MB: 5.1).  That needs few instructions: with the compiler's divisions,
// NaNs compared as numbers and a 64-bit division for each thread's place they took 26.5 and
// 18.7.  Two rows in flight per thread: 21.2 us, one 21.7, four 21.2.
#pragma once

#include "../layers/prod.hpp"
#include "rows8.hpp"

namespace pgemm {
namespace blocks {

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
  int beside;             // log2 of a workgroup's blocks of one row (a scale for each row)
  long long first;        // the launch's first workgroup (a scale for each row: in y)
};

template <int F>
__device__ __forceinline__ float largest() {
  return F == kE4M3 ? 448.0f : 57344.0f;
}

// Magnitudes are compared as whole numbers, without their sign bit: infinity is larger than
// every number, a NaN larger still.
template <typename T>
__device__ __forceinline__ uint32_t top8(const Stored8<T>& s) {
  if constexpr (sizeof(T) == 4) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) m = max(m, s.v[k][j] & 0x7fffffffu);
    return m;
  } else {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 m = {0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t x = s.v[0][j] & 0x7fff7fffu;
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, x));
    }
    return max((uint32_t)m[0], (uint32_t)m[1]);
  }
}
// The bits of a T's magnitude as a number.
template <typename T>
__device__ __forceinline__ float number(uint32_t bits) {
  if constexpr (sizeof(T) == 4) return __builtin_bit_cast(float, bits);
  else return (float)__builtin_bit_cast(T, (uint16_t)bits);
}

template <int F>
__device__ __forceinline__ float scale_of(float top) {
  if (!(top <= 3.402823466e38f)) return __builtin_nanf("");
  const float s = top / largest<F>();
  return s > 1.17549435e-38f ? s : 1.17549435e-38f;
}

// x / s, rounded once, from r = 1 / s rounded once.  x r is within 1.5 steps of x / s, the
// first correction brings it within one, and from there the second gives the quotient's
// rounding (Markstein's theorem; the remainders are exact).  Six instructions, where the
// division itself takes some thirteen.  For s of at least 2^-80: below that remainders of
// quotients that 8 bits can tell from 0 may underflow.
__device__ __forceinline__ float quotient(float x, float s, float r) {
  float q = x * r;
  q = fmaf(fmaf(-q, s, x), r, q);
  q = fmaf(fmaf(-q, s, x), r, q);
  return copysignf(q, x);
}

// Four values rounded to 8 bits, and eight over their scale.
template <int F>
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  int p = 0;
  if constexpr (F == kE4M3) {
    p = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, p, false);
    p = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, p, true);
  } else {
    p = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, p, false);
    p = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, p, true);
  }
  return (uint32_t)p;
}
template <int F>
__device__ __forceinline__ u32x2 pack8(const float* v, float s, float r) {
  float q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j] = quotient(v[j], s, r);
  if (s < 8.27180613e-25f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = v[j] / s;
  }
  return u32x2{pack4<F>(q[0], q[1], q[2], q[3]), pack4<F>(q[4], q[5], q[6], q[7])};
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

// X with its rows contiguous, a scale for each row's block: 16 lanes a block.  A workgroup
// has 2^a.beside blocks of a row beside each other and 16 >> a.beside rows, kRowsAhead times.
constexpr int kRowsAhead = 2;
template <typename T, int F>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const QuantizeArgs a) {
  constexpr int ROWS = kRowsAhead;
  const int high = 16 >> a.beside, g = threadIdx.x >> 4;
  const int b = ((int)blockIdx.x << a.beside) + (g & ((1 << a.beside) - 1));
  const long long row0 = (a.first + blockIdx.y) * (high * ROWS) + (g >> a.beside);
  const int c = b * kScaleBlock + (threadIdx.x & 15) * 8;
  Stored8<T> raw[ROWS];
  rows8<T>(a.c, [&](auto get) {
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const long long row = row0 + k * high;
      raw[k] = get(a.X, (row < a.r ? row : a.r - 1) * a.ldx, c);
    }
  });
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    const long long row = row0 + k * high;
    settle8<T>(raw[k], c, a.c);
    uint32_t top = top8<T>(raw[k]);
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) top = max(top, __shfl_xor(top, d));
    const float s = scale_of<F>(number<T>(top));
    float v[8];
    widen8<T>(raw[k], v);
    const u32x2 q = pack8<F>(v, s, 1.0f / s);
    if (row >= a.r || b >= a.blocks) continue;
    if ((threadIdx.x & 15) == 0) a.scales[row * a.srow + b * a.sblock] = s;
    put_bytes8(a.Q + row * a.ldq, c, a.c, q);
  }
}

// The largest of `top` over the workgroup's 256 threads.
__device__ __forceinline__ uint32_t workgroup_top(uint32_t top, uint32_t* lds) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) top = max(top, __shfl_xor(top, d));
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = top;
  __syncthreads();
  return max(max(lds[0], lds[1]), max(lds[2], lds[3]));
}

// The same with a scale for 128 rows together: a block per workgroup, in registers.
template <typename T, int F>
__global__ __launch_bounds__(256) void quantize_blocks_kernel(const QuantizeArgs a) {
  __shared__ uint32_t lds[4];
  const long long id = a.first + blockIdx.x;
  const int i = (int)(id / a.blocks), b = (int)(id - (long long)i * a.blocks);
  const int c = b * kScaleBlock + (threadIdx.x & 15) * 8;
  Stored8<T> raw[8];
  rows8<T>(a.c, [&](auto get) {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const long long row = (long long)i * kScaleBlock + p * 16 + (threadIdx.x >> 4);
      raw[p] = get(a.X, (row < a.r ? row : a.r - 1) * a.ldx, c);
    }
  });
  uint32_t top = 0;
#pragma unroll
  for (int p = 0; p < 8; ++p) {   // (rows behind the last repeat it: the same largest)
    settle8<T>(raw[p], c, a.c);
    top = max(top, top8<T>(raw[p]));
  }
  const float s = scale_of<F>(number<T>(workgroup_top(top, lds))), inverse = 1.0f / s;
  if (threadIdx.x == 0) a.scales[i * a.srow + b * a.sblock] = s;
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const long long row = (long long)i * kScaleBlock + p * 16 + (threadIdx.x >> 4);
    float v[8];
    widen8<T>(raw[p], v);
    if (row < a.r) put_bytes8(a.Q + row * a.ldq, c, a.c, pack8<F>(v, s, inverse));
  }
}

// X with its columns contiguous: a workgroup reads 128 x 128 along the columns
// (16 lanes a column, 8 rows each), and writes rows from bytes turned in LDS.
template <typename T, int F, bool TOGETHER>
__global__ __launch_bounds__(256) void quantize_outer_kernel(const QuantizeArgs a) {
  constexpr int LD = 128 + 8;                        // bytes of a row
  __shared__ __attribute__((aligned(16))) uint32_t tops[TOGETHER ? 4 : 16 * 128];
  __shared__ float scales[TOGETHER ? 1 : 128];
  __shared__ __attribute__((aligned(16))) uint8_t tile[128 * LD];
  const long long id = a.first + blockIdx.x;
  const int i = (int)(id / a.blocks), b = (int)(id - (long long)i * a.blocks);
  const int r0 = i * kScaleBlock, c0 = b * kScaleBlock;
  const int part = threadIdx.x & 15, lane = threadIdx.x >> 4;   // rows 8 part.., columns 8 lane..
  Stored8<T> raw[8];
  rows8<T>(a.r, [&](auto get) {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const long long col = c0 + 8 * lane + p;
      raw[p] = get(a.X, (col < a.c ? col : a.c - 1) * a.ldx, r0 + 8 * part);
    }
  });
#pragma unroll
  for (int p = 0; p < 8; ++p) settle8<T>(raw[p], r0 + 8 * part, a.r);
  // (columns behind the last repeat it: the same largest)
  float s[8];
  if constexpr (TOGETHER) {
    uint32_t top = 0;
#pragma unroll
    for (int p = 0; p < 8; ++p) top = max(top, top8<T>(raw[p]));
    const float t = scale_of<F>(number<T>(workgroup_top(top, tops)));
    if (threadIdx.x == 0) a.scales[i * a.srow + b * a.sblock] = t;
    s[0] = t;
  } else {
    float v[8][8];
#pragma unroll
    for (int p = 0; p < 8; ++p) widen8<T>(raw[p], v[p]);
    u32x4 top[2];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t m = 0;
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        const float x = v[p][j];
        m = max(m, __builtin_bit_cast(uint32_t, x) & 0x7fffffffu);
      }
      top[j >> 2][j & 3] = m;
    }
    u32x4* const to = reinterpret_cast<u32x4*>(tops + lane * 128 + 8 * part);
    to[0] = top[0];
    to[1] = top[1];
    __syncthreads();
    if (threadIdx.x < 128) {
      uint32_t top = tops[threadIdx.x];
#pragma unroll
      for (int l = 1; l < 16; ++l) top = max(top, tops[l * 128 + threadIdx.x]);
      const float t = scale_of<F>(__builtin_bit_cast(float, top));
      scales[threadIdx.x] = t;
      const long long row = r0 + (int)threadIdx.x;
      if (row < a.r) a.scales[row * a.srow + b * a.sblock] = t;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = scales[8 * part + j];
  }
  float v[8][8];                                     // [column][row]
#pragma unroll
  for (int p = 0; p < 8; ++p) widen8<T>(raw[p], v[p]);
  const float inverse = TOGETHER ? 1.0f / s[0] : 0.0f;
  // this thread's 8 columns of each of its rows
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float w[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) w[p] = v[p][j];
    const float t = TOGETHER ? s[0] : s[j];
    *reinterpret_cast<u32x2*>(tile + (8 * part + j) * LD + 8 * lane) =
        pack8<F>(w, t, TOGETHER ? inverse : 1.0f / t);
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
