// Layer norm and its gradients.  Both are bound by memory: 4097 x 3001 fp32 24.9 us back to
// back, 20.3 alone with warm caches (98 MB: 3.9 to 4.8 TB/s); gradients of 8192 x 4096 bf16
// with a residual 54.6 us (268 MB: 4.9 TB/s, the sums' second launch of 4.8 us included); one
// row of 4096 6.0 us, a launch.
//
//   forward:  mu = mean(x), v = mean((x - mu)^2), r = 1 / sqrt(v + eps),
//             y = (x - mu) r w + b
//   backward: h = (x - mu) r, g = dy w,
//             dx = r (g - mean(g) - h mean(g h)) + residual,
//             dw = sum over rows of dy h,  db = sum over rows of dy
//
// A row lives in the registers of TPR threads, C chunks of 8 elements each, so
// that it is read once; longer rows are read again, from the caches.
// Everything is fp32 in between (64 bits where a thread adds more than a few
// dozen numbers of one row, and for a row whose squares leave fp32's range), each result
// rounded once.
#pragma once

#include "../layers/prod.hpp"
#include "rows8.hpp"

namespace pgemm {
namespace blocks {

using layers::get_row8;
using layers::put_row8;
using layers::u32x4;

struct NormArgs {
  const void* X;
  const void* W;          // n of T (nullptr: ones)
  const void* B;          // n of T (nullptr: zeros)
  void* Y;
  float* mean;            // m (nullptr: not kept)
  float* rstd;
  long long ldx, ldy;
  int m, n;
  float eps;
};

struct NormBackArgs {
  const void* dY;
  const void* X;
  const float* mean;
  const float* rstd;
  const void* W;          // n of T (nullptr: ones)
  const void* R;          // residual, T (nullptr: none)
  void* dX;               // (norm_sums_kernel writes none)
  float* partial;         // [groups][2][n] column sums: of dy h, of dy (nullptr: not wanted)
  long long ldy, ldx, ldr, ldd;
  int m, n;
  int groups;             // workgroups along the rows
};

struct NormColumnArgs {
  const float* partial;   // [groups][2][n]
  void* dw;               // n of T or fp32 (nullptr: not wanted)
  void* db;
  int n, groups, out32;
};

// Rows of up to kRowMost elements stay in registers, in the gradients up to kBackMost,
// with column sums up to kSumMost (their sums take as many registers again, twice).
constexpr int kRowMost = 1024 * 8 * 4, kBackMost = 1024 * 8 * 2, kSumMost = 1024 * 8;

// N sums over the TPR threads of a row, the same bits for all of them, with one
// barrier.  Calls that follow each other take other parts of `lds`.
template <int TPR, int N, typename S>
__device__ __forceinline__ void row_sums(S (&v)[N], S (*lds)[16]) {
#pragma unroll
  for (int d = 1; d < (TPR < 64 ? TPR : 64); d <<= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor(v[k], d);
  if constexpr (TPR > 64) {
    constexpr int WAVES = TPR / 64;
    const int first = threadIdx.x / TPR * WAVES;
#pragma unroll
    for (int k = 0; k < N; ++k)
      if ((threadIdx.x & 63) == 0) lds[k][threadIdx.x >> 6] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      v[k] = lds[k][first];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) v[k] += lds[k][first + w];
    }
  }
}

// One row in 64 bits, by TPR threads of which this is t, read three times.
template <typename T, int TPR>
__device__ __forceinline__ void norm_row(const NormArgs& a, long long row, int t, double (*lds)[16]) {
  double s[1] = {0.0};
  for (uint32_t c = t * 8; c < (uint32_t)a.n; c += TPR * 8) {
    float x[8];
    get_row8<T>(a.X, row * a.ldx, (int)c, a.n, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) s[0] += x[j];
  }
  row_sums<TPR>(s, lds);
  const double mean = s[0] / a.n;
  s[0] = 0.0;
  for (uint32_t c = t * 8; c < (uint32_t)a.n; c += TPR * 8) {
    float x[8];
    get_row8<T>(a.X, row * a.ldx, (int)c, a.n, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double d = (int)c + j < a.n ? x[j] - mean : 0.0;
      s[0] += d * d;
    }
  }
  row_sums<TPR>(s, lds + 1);
  const double rstd = 1.0 / sqrt(s[0] / a.n + (double)a.eps);
  if (t == 0) {
    if (a.mean != nullptr) a.mean[row] = (float)mean;
    if (a.rstd != nullptr) a.rstd[row] = (float)rstd;
  }
  for (uint32_t c = t * 8; c < (uint32_t)a.n; c += TPR * 8) {
    float x[8], w[8], b[8];
    get_row8<T>(a.X, row * a.ldx, (int)c, a.n, x);
    if (a.W != nullptr) get_row8<T>(a.W, 0, (int)c, a.n, w);
    if (a.B != nullptr) get_row8<T>(a.B, 0, (int)c, a.n, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float y = (float)((x[j] - mean) * rstd);
      if (a.W != nullptr) y *= w[j];
      if (a.B != nullptr) y += b[j];
      x[j] = y;
    }
    put_row8<T>(a.Y, row * a.ldy, (int)c, a.n, x);
  }
}

template <typename T, int TPR, int C, int NT>
__global__ __launch_bounds__(NT) void norm_kernel(const NormArgs a) {
  __shared__ float lds[3][16];
  __shared__ double wide[2][16];
  constexpr int ROWS = NT / TPR;
  const int t = threadIdx.x % TPR;
  const long long row = ROWS == 1 ? blockIdx.x : (long long)blockIdx.x * ROWS + threadIdx.x / TPR;
  const bool live = ROWS == 1 || row < a.m;
  const long long at = (live ? row : a.m - 1) * a.ldx;
  Stored8<T> raw[C];
  rows8<T>(a.n, [&](auto get) {
#pragma unroll
    for (int c = 0; c < C; ++c) raw[c] = get(a.X, at, (c * TPR + t) * 8);
  });
  float x[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    settle8<T>(raw[c], (c * TPR + t) * 8, a.n);
    widen8<T>(raw[c], x[c]);
  }
  float s[1] = {0.0f};
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) s[0] += x[c][j];
  row_sums<TPR>(s, lds);
  const float inv = 1.0f / (float)a.n, mean = s[0] * inv;
  // around the rounded mean; what is left of the mean corrects both
  float q[2] = {0.0f, 0.0f};
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = (c * TPR + t) * 8 + j < a.n ? x[c][j] - mean : 0.0f;
      x[c][j] = d;
      q[0] += d;
      q[1] += d * d;
    }
  row_sums<TPR>(q, lds + 1);
  const float d1 = q[0] * inv, var = q[1] * inv - d1 * d1;
  if (!live) return;
  // squares beyond fp32 (or a NaN), or where what they lose below it matters (where waves have
  // one row the branch is a scalar one, so that the row's registers are free behind it)
  int far = !(var < 3e38f && (var > 0.0f ? var : 0.0f) + a.eps > 1e-30f);
  if constexpr (TPR >= 64) far = __builtin_amdgcn_readfirstlane(far);
  if (far) {
    norm_row<T, TPR>(a, row, t, wide);
    return;
  }
  const float rstd = 1.0f / sqrtf((var > 0.0f ? var : 0.0f) + a.eps);
  if (t == 0) {
    if (a.mean != nullptr) a.mean[row] = mean + d1;
    if (a.rstd != nullptr) a.rstd[row] = rstd;
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * TPR + t) * 8;
    if (col >= a.n) break;
    float w[8], b[8];
    if (a.W != nullptr) get_row8<T>(a.W, 0, col, a.n, w);
    if (a.B != nullptr) get_row8<T>(a.B, 0, col, a.n, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float y = (x[c][j] - d1) * rstd;
      if (a.W != nullptr) y *= w[j];
      if (a.B != nullptr) y += b[j];
      x[c][j] = y;
    }
    put_row8<T>(a.Y, row * a.ldy, col, a.n, x[c]);
  }
}

// Rows longer than registers hold, one per workgroup.
template <typename T>
__global__ __launch_bounds__(1024) void norm_long_kernel(const NormArgs a) {
  __shared__ double lds[2][16];
  norm_row<T, 1024>(a, blockIdx.x, threadIdx.x, lds);
}

// dX and, with SUMS, the column sums of this workgroup's rows: row group by row
// group, each thread adds its columns in order; the groups of one workgroup
// are then added in order through LDS.  The next row is asked for before the sums
// of this one, where the registers hold both; rows are kept as they are stored (16-bit
// ones in half the registers).  Rows over 8192 take the column sums apart, in a second pass over
// X and dY (4096 rows of 16384, bf16: 139 us for a floor of 80): with the sums in registers 75
// to 135 of them were spilled (190 us).  Sums in LDS, 128 KB of them for 16384 features, have
// not been tried.
template <typename T, int TPR, int C, int NT, bool SUMS>
__global__ __launch_bounds__(NT) void norm_back_kernel(const NormBackArgs a) {
  constexpr int ROWS = NT / TPR;
  constexpr bool AHEAD = C == 1;
  __shared__ float lds[4][16];
  __shared__ float cols[SUMS && ROWS > 1 ? NT * 8 : 1];
  const int t = threadIdx.x % TPR, mine = threadIdx.x / TPR;
  const float inv = 1.0f / (float)a.n;
  Stored8<T> w[C];
  float sw[SUMS ? C : 1][8], sb[SUMS ? C : 1][8];
  if (a.W != nullptr) {
    rows8<T>(a.n, [&](auto get) {
#pragma unroll
      for (int c = 0; c < C; ++c) w[c] = get(a.W, 0, (c * TPR + t) * 8);
    });
#pragma unroll
    for (int c = 0; c < C; ++c) settle8<T>(w[c], (c * TPR + t) * 8, a.n);
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if constexpr (SUMS) {
#pragma unroll
      for (int j = 0; j < 8; ++j) sw[c][j] = sb[c][j] = 0.0f;
    }
  }
  struct Row {
    Stored8<T> x[C], d[C], r[AHEAD ? C : 1];
    float mean, rstd;
  };
  auto load = [&](long long r0) {
    const long long row = r0 + mine < a.m ? r0 + mine : a.m - 1;
    Row v;
    v.mean = a.mean[row];
    v.rstd = a.rstd[row];
    rows8<T>(a.n, [&](auto get) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        v.x[c] = get(a.X, row * a.ldx, (c * TPR + t) * 8);
        v.d[c] = get(a.dY, row * a.ldy, (c * TPR + t) * 8);
        if (AHEAD && a.R != nullptr) v.r[c] = get(a.R, row * a.ldr, (c * TPR + t) * 8);
      }
    });
    return v;
  };
  auto settle = [&](Row& v) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      settle8<T>(v.x[c], (c * TPR + t) * 8, a.n);
      settle8<T>(v.d[c], (c * TPR + t) * 8, a.n);
      if (AHEAD && a.R != nullptr) settle8<T>(v.r[c], (c * TPR + t) * 8, a.n);
    }
  };
  // h and g of chunk c
  auto values = [&](const Row& v, int c, float* h, float* g) {
    float x[8];
    widen8<T>(v.x[c], x);
    widen8<T>(v.d[c], g);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      h[j] = (c * TPR + t) * 8 + j < a.n ? (x[j] - v.mean) * v.rstd : 0.0f;
  };
  auto weigh = [&](int c, float* g) {
    if (a.W == nullptr) return;
    float k[8];
    widen8<T>(w[c], k);
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] *= k[j];
  };
  const long long step = (long long)a.groups * ROWS;
  long long r0 = (long long)blockIdx.x * ROWS;
  int slot = 0;
  Row next;
  if (AHEAD && r0 < a.m) next = load(r0);
#pragma unroll 1
  for (; r0 < a.m; r0 += step) {
    if (!AHEAD) next = load(r0);
    Row v = next;
    const bool live = r0 + mine < a.m;
    if (AHEAD && r0 + step < a.m) next = load(r0 + step);
    settle(v);
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float h[8], g[8];
      values(v, c, h, g);
      if constexpr (SUMS) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          sw[c][j] += live ? g[j] * h[j] : 0.0f;
          sb[c][j] += live ? g[j] : 0.0f;
        }
      }
      weigh(c, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s[0] += g[j];
        s[1] += g[j] * h[j];
      }
    }
    row_sums<TPR>(s, lds + slot);
    slot ^= 2;
    const float s1 = s[0] * inv, s2 = s[1] * inv;
    if (live) {
      const long long row = r0 + mine;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int col = (c * TPR + t) * 8;
        if (col >= a.n) break;
        float h[8], g[8], res[8];
        values(v, c, h, g);
        weigh(c, g);
        if (a.R != nullptr) {
          if constexpr (AHEAD) widen8<T>(v.r[c], res);
          else get_row8<T>(a.R, row * a.ldr, col, a.n, res);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          g[j] = v.rstd * (g[j] - s1 - h[j] * s2);
          if (a.R != nullptr) g[j] += res[j];
        }
        put_row8<T>(a.dX, row * a.ldd, col, a.n, g);
      }
    }
  }
  if constexpr (SUMS) {
    float* out = a.partial + (long long)blockIdx.x * 2 * a.n;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = k == 0 ? sw[c][j] : sb[c][j];
        if constexpr (ROWS > 1) {
          __syncthreads();
#pragma unroll
          for (int j = 0; j < 8; ++j) cols[threadIdx.x * 8 + j] = v[j];
          __syncthreads();
          if (mine == 0) {
#pragma unroll 1
            for (int r = 1; r < ROWS; ++r)
#pragma unroll
              for (int j = 0; j < 8; ++j) v[j] += cols[(r * TPR + t) * 8 + j];
          }
        }
        if (mine == 0) put_row8<float>(out, (long long)k * a.n, (c * TPR + t) * 8, a.n, v);
      }
  }
}

// dX of rows longer than registers hold: read twice.
template <typename T>
__global__ __launch_bounds__(1024) void norm_back_long_kernel(const NormBackArgs a) {
  __shared__ double lds[2][16];
  const long long row = blockIdx.x;
  const float mean = a.mean[row], rstd = a.rstd[row];
  auto load = [&](int c, float* h, float* g) {
    float w[8];
    get_row8<T>(a.X, row * a.ldx, c, a.n, h);
    get_row8<T>(a.dY, row * a.ldy, c, a.n, g);
    if (a.W != nullptr) get_row8<T>(a.W, 0, c, a.n, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h[j] = c + j < a.n ? (h[j] - mean) * rstd : 0.0f;
      if (a.W != nullptr) g[j] *= w[j];
    }
  };
  double s[2] = {0.0, 0.0};
  for (long long c = threadIdx.x * 8; c < a.n; c += 8192) {
    float h[8], g[8];
    load((int)c, h, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      s[0] += g[j];
      s[1] += (double)g[j] * h[j];
    }
  }
  row_sums<1024>(s, lds);
  const float m1 = (float)(s[0] / a.n), m2 = (float)(s[1] / a.n);
  for (long long c = threadIdx.x * 8; c < a.n; c += 8192) {
    float h[8], g[8], res[8];
    load((int)c, h, g);
    if (a.R != nullptr) get_row8<T>(a.R, row * a.ldr, (int)c, a.n, res);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g[j] = rstd * (g[j] - m1 - h[j] * m2);
      if (a.R != nullptr) g[j] += res[j];
    }
    put_row8<T>(a.dX, row * a.ldd, (int)c, a.n, g);
  }
}

// The column sums alone (rows longer than registers hold, or no dX): 512
// columns per workgroup, 4 rows at once.
template <typename T>
__global__ __launch_bounds__(256) void norm_sums_kernel(const NormBackArgs a) {
  __shared__ float cols[256 * 8];
  const int t = threadIdx.x & 63, mine = threadIdx.x >> 6;
  const int group = blockIdx.x % a.groups;
  const long long c = ((long long)(blockIdx.x / a.groups) * 64 + t) * 8;
  float sw[8] = {0, 0, 0, 0, 0, 0, 0, 0}, sb[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (c < a.n) {
    for (long long r = (long long)group * 4 + mine; r < a.m; r += (long long)a.groups * 4) {
      const float mean = a.mean[r], rstd = a.rstd[r];
      Stored8<T> raw[2];
      rows8<T>(a.n, [&](auto get) {
        raw[0] = get(a.X, r * a.ldx, (int)c);
        raw[1] = get(a.dY, r * a.ldy, (int)c);
      });
      float x[8], d[8];
      settle8<T>(raw[0], (int)c, a.n);
      settle8<T>(raw[1], (int)c, a.n);
      widen8<T>(raw[0], x);
      widen8<T>(raw[1], d);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sw[j] += d[j] * ((x[j] - mean) * rstd);
        sb[j] += d[j];
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) cols[threadIdx.x * 8 + j] = k == 0 ? sw[j] : sb[j];
    __syncthreads();
    if (mine == 0 && c < a.n) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = ((cols[t * 8 + j] + cols[(64 + t) * 8 + j]) + cols[(128 + t) * 8 + j]) +
               cols[(192 + t) * 8 + j];
      put_row8<float>(a.partial + ((long long)group * 2 + k) * a.n, 0, (int)c, a.n, v);
    }
  }
}

// dweight and dbias (blockIdx.y) from the groups' column sums: 64 columns per
// workgroup, 16 threads per column that each add every sixteenth group in order,
// then their sums in order.
template <typename T>
__global__ __launch_bounds__(1024) void norm_columns_kernel(const NormColumnArgs a) {
  __shared__ float sums[16][64];
  void* out = blockIdx.y == 0 ? a.dw : a.db;
  if (out == nullptr) return;
  const int t = threadIdx.x & 63, part = threadIdx.x >> 6;
  for (long long c0 = (long long)blockIdx.x * 64; c0 < a.n; c0 += (long long)gridDim.x * 64) {
    const long long c = c0 + t;
    float v = 0.0f;
    if (c < a.n) {
      const float* from = a.partial + (long long)blockIdx.y * a.n + c;
#pragma unroll 8
      for (int g = part; g < a.groups; g += 16) v += from[(long long)g * 2 * a.n];
    }
    __syncthreads();
    sums[part][t] = v;
    __syncthreads();
    if (part != 0 || c >= a.n) continue;
#pragma unroll
    for (int p = 1; p < 16; ++p) v += sums[p][t];
    if (a.out32) static_cast<float*>(out)[c] = v;
    else static_cast<T*>(out)[c] = (T)v;
  }
}

}  // namespace blocks
}  // namespace pgemm
