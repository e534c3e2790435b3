// Few rows: up to 32 rows of D against the whole of B, bound by reading B
// once.  A workgroup takes NB blocks of 16 columns and all of the summed index
// (or one split of it); its 8 waves take units of 128 bytes of the summed
// index in turn, each adding into its own 16 x 16 accumulators, which are
// summed over the waves through LDS in a fixed order.
//
// Inner-order B goes from memory straight into the matrix instruction's
// operand registers (16 rows of 128 consecutive bytes per unit).  Outer-order
// B arrives as rows of 64 columns and passes through a wave-private LDS tile,
// whose transposing reads give the operand.  The loads of the next units are
// issued before the current ones are used.
#pragma once

#include "prod_tile.hpp"

namespace pgemm {
namespace layers {

template <typename T, int LB, int MB, int MODE>
struct RowsShape {
  static constexpr int WAVES = 8;
  static constexpr int NB = LB == kInner ? 1 : 4;     // column blocks
  static constexpr int BN = 16 * NB;
  static constexpr int U = LB == kInner ? 2 : 1;      // units in flight per step
};

template <typename T, int LB, int MB, int MODE>
__global__ __launch_bounds__(512) void prod_rows_kernel(const ProdArgs a) {
  using S = RowsShape<T, LB, MB, MODE>;
  constexpr int WAVES = S::WAVES, NB = S::NB, BN = S::BN, U = S::U;
  constexpr int V = 16 / (int)sizeof(T), BK = 128 / (int)sizeof(T);
  constexpr int RED_LD = BN + 4;
  constexpr int RED = WAVES * MB * 16 * RED_LD * 4;
  constexpr int STG = LB == kOuter ? WAVES * BN * 128 : 0;
  constexpr int LDS = RED > STG ? RED : STG;
  __shared__ __attribute__((aligned(128))) char lds[LDS];
  using TB = OperandTile<T, kOuter, 64, 64, 16>;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, i = lane & 15;
  int nb = blockIdx.x, e = 0, lo = 0, hi = a.M;
  const T* Bb = static_cast<const T*>(a.B);
  const void* bias = a.bias;
  if constexpr (MODE == kRows) {
    e = blockIdx.x / a.tiles_n;
    nb = blockIdx.x % a.tiles_n;
    group_bounds(a.offsets, e, a.rows, &lo, &hi);
    if (lo == hi) return;
    Bb += e * a.strideB;
    if (bias != nullptr) bias = static_cast<const T*>(bias) + e * a.strideBias;
  }
  const int col0 = nb * BN;
  int k_lo = 0, k_hi = a.K;
  if (MODE == kDense && a.splits > 1) {
    k_lo = blockIdx.y * a.k_split;
    k_hi = k_lo + a.k_split < a.K ? k_lo + a.k_split : a.K;
  }
  const int units = (k_hi - k_lo + BK - 1) / BK;
  Source<T> sa = {static_cast<const T*>(a.A), a.lda, hi, k_hi,
                  MODE == kRows ? a.gather : nullptr, a.gather_rows};
  const T* brow = nullptr;                      // inner order: the lane's row of B
  if (LB == kInner && col0 + i < a.N) brow = Bb + (long long)(col0 + i) * a.ldb;

  for (int m0 = lo; m0 < hi; m0 += 16 * MB) {
    const T* arow[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) arow[b] = sa.row(m0 + 16 * b + i);

    f32x4 acc[MB][NB];
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int c = 0; c < NB; ++c) acc[b][c] = f32x4{0, 0, 0, 0};

    constexpr int BL = LB == kInner ? 2 : 8;    // loads of B per unit and lane
    u32x4 xb[U][BL], xa[U][MB][2], yb[U][BL], ya[U][MB][2];
    auto load_unit = [&](auto whole, int u, int k0, u32x4(&rb)[U][BL], u32x4(&ra)[U][MB][2]) {
        constexpr bool W = decltype(whole)::value;
        if constexpr (LB == kInner) {
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
            rb[u][kk] = W ? load_whole(brow, k0 + (4 * kk + g) * V)
                          : load_guarded(brow, k0 + (4 * kk + g) * V, k_hi);
        } else {
#pragma unroll
          for (int j = 0; j < BL; ++j) {
            int r, c;
            TB::slot(j * 64 + lane, &r, &c);
            const T* row = k0 + r < k_hi ? Bb + (long long)(k0 + r) * a.ldb : nullptr;
            rb[u][j] = W ? load_whole(row, col0 + c * V) : load_guarded(row, col0 + c * V, a.N);
          }
        }
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
            ra[u][b][kk] = W ? load_whole(arow[b], k0 + (4 * kk + g) * V)
                             : load_guarded(arow[b], k0 + (4 * kk + g) * V, k_hi);
    };
    auto load = [&](int u0, u32x4(&rb)[U][BL], u32x4(&ra)[U][MB][2]) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k0 = k_lo + (u0 + u * WAVES) * BK;
        if (k0 + BK <= k_hi && (LB == kInner || col0 + BN <= a.N))
          load_unit(std::integral_constant<bool, true>{}, u, k0, rb, ra);
        else
          load_unit(std::integral_constant<bool, false>{}, u, k0, rb, ra);
      }
    };
    auto use = [&](u32x4(&rb)[U][BL], u32x4(&ra)[U][MB][2]) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if constexpr (LB == kInner) {
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int b = 0; b < MB; ++b)
              acc[b][0] = Elem<T>::mfma(rb[u][kk], ra[u][b][kk], acc[b][0]);
        } else {
          char* mine = lds + wave * BN * 128;
#pragma unroll
          for (int j = 0; j < BL; ++j)
            *reinterpret_cast<u32x4*>(mine + (j * 64 + lane) * 16) = rb[u][j];
          __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
          __builtin_amdgcn_wave_barrier();
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int c = 0; c < NB; ++c) {
              const u32x4 f = TB::frag(mine, 0, c, kk);
#pragma unroll
              for (int b = 0; b < MB; ++b) acc[b][c] = Elem<T>::mfma(f, ra[u][b][kk], acc[b][c]);
            }
          __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
          __builtin_amdgcn_wave_barrier();
        }
      }
    };
    // units of this wave: wave, wave + WAVES, ...; loads past the end give zeros
    constexpr int STEP = U * WAVES;
    if (wave < units) load(wave, xb, xa);
    for (int u0 = wave; u0 < units; u0 += 2 * STEP) {
      if (u0 + STEP < units) load(u0 + STEP, yb, ya);
      use(xb, xa);
      if (u0 + STEP < units) {
        if (u0 + 2 * STEP < units) load(u0 + 2 * STEP, xb, xa);
        use(yb, ya);
      }
    }

    // sum over the waves, then 8 columns per thread
    __syncthreads();
    float* red = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int c = 0; c < NB; ++c)
        *reinterpret_cast<f32x4*>(red + ((wave * MB + b) * 16 + i) * RED_LD + 16 * c + 4 * g) =
            acc[b][c];
    __syncthreads();
    for (int t = threadIdx.x; t < MB * 16 * (BN / 8); t += 512) {
      const int row = t / (BN / 8), col = (t % (BN / 8)) * 8;
      const int m = m0 + row, n = col0 + col;
      if (m < hi && n < a.N) {
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
          const float* from = red + (w * MB * 16 + row) * RED_LD + col;
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] += from[j];
        }
        if (MODE == kDense && a.splits > 1) {
          float* to = a.partial + ((long long)blockIdx.y * a.M + m) * a.N + n;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (n + j < a.N) to[j] = v[j];
        } else {
          finish8<T>(a, bias, a.D, m, n, v);
        }
      }
    }
    __syncthreads();   // before the next row block reuses the LDS
  }
}

// Sums the splits of a product in order and runs its epilogue: 8 columns per
// thread.
template <typename T>
__global__ __launch_bounds__(256) void prod_reduce_kernel(const ProdArgs a) {
  const int per_row = (a.N + 7) / 8;
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
  if (id >= (long long)a.M * per_row) return;
  const long long m = id / per_row;
  const int n = (int)(id % per_row) * 8;
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int s = 0; s < a.splits; ++s) {
    const float* from = a.partial + ((long long)s * a.M + m) * a.N + n;
    if (n + 8 <= a.N) {
      float x[8];
      get8<float>(from, 0, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += x[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (n + j < a.N) v[j] += from[j];
    }
  }
  finish8<T>(a, a.bias, a.D, m, n, v);
}

}  // namespace layers
}  // namespace pgemm
