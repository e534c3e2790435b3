// Few rows: up to 32 rows of D against the whole of B, bound by reading B
// once.  A workgroup takes NB blocks of 16 columns and all of the summed index
// (or one split of it); its waves take units of 128 bytes of the summed index
// in turn, each adding into its own 16 x 16 accumulators, which are summed over
// the waves through LDS in a fixed order.
//
// Inner-order B goes from memory straight into the matrix instruction's
// operand registers (16 rows of 128 consecutive bytes per unit and block).
// Outer-order B arrives as rows of 16 NB columns and passes through a
// wave-private LDS tile, whose transposing reads give the operand.  The loads
// of the next units are issued before the current ones are used.
//
// NB = 4 where that gives every compute unit its workgroups; otherwise NB = 1,
// with more units in flight per wave, so that a small B is still spread over the
// whole chip and most of it is in flight at
// once.  Workgroups of neighbouring columns run on one XCD: with NB = 1 they
// share outer-order B's cache lines.
//
// Rows of an expert beyond 32 read its weight again for every 16 or 32: the class
// is chosen by the average, so that 1024 rows, half of them on one of 64 experts
// (1024 x 2048), take 218 us, evenly spread 57.
//
// Measured, bf16: one row through 4096 x 4096 8.2 us a call (33.6 MB: 4.1 TB/s
// with the launch); 64 rows over the experts of 64 that 16 tokens chose, 1024 x
// 2048 each, 47 us (213 MB: 4.5 TB/s; a large copy reaches 5.1).
#pragma once

#include "prod_tile.hpp"

namespace pgemm {
namespace layers {

template <typename T, int LB, int MB, int NB, int WAVES, int MODE>
__global__ __launch_bounds__(WAVES * 64) void prod_rows_kernel(const ProdArgs a) {
  constexpr int BN = 16 * NB, U = NB == 1 ? (MB == 1 ? 4 : 2) : 1;   // U: units per load
  constexpr int V = 16 / (int)sizeof(T), BK = 128 / (int)sizeof(T);
  constexpr int RED_LD = BN + 4;
  constexpr int RED = WAVES * MB * 16 * RED_LD * 4;
  constexpr int STG = LB == kOuter ? WAVES * BN * 128 : 0;
  constexpr int LDS = RED > STG ? RED : STG;
  __shared__ __attribute__((aligned(128))) char lds[LDS];
  using TB = OperandTile<T, kOuter, BN, 64>;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, i = lane & 15;
  const int id = map_range(blockIdx.x, gridDim.x);
  int nb = id, e = 0, lo = 0, hi = a.M;
  const T* Bb = static_cast<const T*>(a.B);
  const void* bias = a.bias;
  if constexpr (MODE == kRows) {
    nb = id % a.tiles_n;
    e = id / a.tiles_n;
    if (a.rows < a.groups) {
      // fewer rows than groups: the e-th group that has some (the search takes
      // longer than to end a workgroup: 64 rows over 64 groups 46 us, so 58)
      int left;
      e = find_group(a.offsets, a.groups, a.rows, 0, e, &lo, &left);
      if (e < 0) return;
      hi = lo + left;
    } else {
      group_bounds(a.offsets, e, a.rows, &lo, &hi);
      if (lo == hi) return;
    }
    Bb += e * a.strideB;
    if (bias != nullptr) bias = static_cast<const T*>(bias) + e * a.strideBias;
  }
  const int col0 = nb * BN;
  int k_lo = 0, k_hi = a.K;
  if (MODE == kDense && a.splits > 1) {
    k_lo = blockIdx.y * a.k_split;
    k_hi = k_lo + a.k_split < a.K ? k_lo + a.k_split : a.K;
  }
  // Units loaded without guards, and those at the end of the summed index
  // that need them.  Rows and columns outside the operands read the last row
  // or the first chunk instead (their results are never stored); a chunk of
  // outer-order B that straddles its row's end goes on into the next rows,
  // which is inside B except near its end.
  const int units = (k_hi - k_lo + BK - 1) / BK;
  int whole = (k_hi - k_lo) / BK;
  if (LB == kOuter && col0 + BN > a.N) {
    const int inside = a.K - V - k_lo;
    whole = inside < 0 ? 0 : (inside / BK < whole ? inside / BK : whole);
  }
  Source<T> sa = {static_cast<const T*>(a.A), a.lda, hi, k_hi,
                  MODE == kRows ? a.gather : nullptr, a.gather_rows};
  constexpr int BL = 2 * NB;                    // loads of B per unit and lane
  const T* bptr[LB == kInner ? NB : BL];        // without the summed index
#pragma unroll
  for (int c = 0; c < (LB == kInner ? NB : BL); ++c) {
    if constexpr (LB == kInner) {
      const int n = col0 + 16 * c + i;
      bptr[c] = Bb + (long long)(n < a.N ? n : a.N - 1) * a.ldb;
    } else {
      int r, q;
      TB::slot(c * 64 + lane, &r, &q);
      const int n = col0 + q * V;
      bptr[c] = Bb + (long long)r * a.ldb + (n < a.N ? n : 0);
    }
  }

  for (int m0 = lo; m0 < hi; m0 += 16 * MB) {
    const T* arow[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) {
      const int m = m0 + 16 * b + i;
      arow[b] = sa.row(m < hi ? m : hi - 1);
    }

    f32x4 acc[MB][NB];
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int c = 0; c < NB; ++c) acc[b][c] = f32x4{0, 0, 0, 0};

    // multiply one unit's operands (outer order: through the wave's own LDS)
    auto use = [&](u32x4(&rb)[BL], u32x4(&ra)[MB][2]) {
      if constexpr (LB == kInner) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
          for (int c = 0; c < NB; ++c)
#pragma unroll
            for (int b = 0; b < MB; ++b)
              acc[b][c] = Elem<T>::mfma(rb[2 * c + kk], ra[b][kk], acc[b][c]);
      } else {
        char* mine = lds + wave * BN * 128;
#pragma unroll
        for (int j = 0; j < BL; ++j)
          *reinterpret_cast<u32x4*>(mine + (j * 64 + lane) * 16) = rb[j];
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
          for (int c = 0; c < NB; ++c) {
            const u32x4 f = TB::frag(mine, 0, c, kk);
#pragma unroll
            for (int b = 0; b < MB; ++b) acc[b][c] = Elem<T>::mfma(f, ra[b][kk], acc[b][c]);
          }
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        __builtin_amdgcn_wave_barrier();
      }
    };
    // this wave's units: wave, wave + WAVES, ..., U of them per load
    constexpr int STEP = U * WAVES;
    u32x4 xb[U][BL], xa[U][MB][2], yb[U][BL], ya[U][MB][2];
    auto load = [&](int u0, u32x4(&rb)[U][BL], u32x4(&ra)[U][MB][2]) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int unit = u0 + u * WAVES;
        if (unit >= whole) break;
        const int k0 = k_lo + unit * BK;
#pragma unroll
        for (int j = 0; j < BL; ++j) {
          if constexpr (LB == kInner) rb[u][j] = load16(bptr[j >> 1] + k0 + (4 * (j & 1) + g) * V);
          else rb[u][j] = load16(bptr[j] + (long long)k0 * a.ldb);
        }
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) ra[u][b][kk] = load16(arow[b] + k0 + (4 * kk + g) * V);
      }
    };
    auto use_all = [&](int u0, u32x4(&rb)[U][BL], u32x4(&ra)[U][MB][2]) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u0 + u * WAVES >= whole) break;
        use(rb[u], ra[u]);
      }
    };
    load(wave, xb, xa);
#pragma unroll 1
    for (int u0 = wave; u0 < whole; u0 += 2 * STEP) {
      load(u0 + STEP, yb, ya);
      use_all(u0, xb, xa);
      load(u0 + 2 * STEP, xb, xa);
      use_all(u0 + STEP, yb, ya);
    }
#pragma unroll 1
    for (int unit = whole + wave; unit < units; unit += WAVES) {
      const int k0 = k_lo + unit * BK;
      {
        u32x4 rb[BL], ra[MB][2];
#pragma unroll
        for (int q = 0; q < BL; ++q) {
          if constexpr (LB == kInner) {
            rb[q] = load_guarded(bptr[q >> 1], k0 + (4 * (q & 1) + g) * V, k_hi);
          } else {
            int r, c;
            TB::slot(q * 64 + lane, &r, &c);
            const T* row = k0 + r < k_hi ? Bb + (long long)(k0 + r) * a.ldb : nullptr;
            rb[q] = load_guarded(row, col0 + c * V, a.N);
          }
        }
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
            ra[b][kk] = load_guarded(arow[b], k0 + (4 * kk + g) * V, k_hi);
        use(rb, ra);
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
    for (int t = threadIdx.x; t < MB * 16 * (BN / 8); t += WAVES * 64) {
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

// Sums the splits of a product (of every group's, for grouped sums) in order and
// runs its epilogue: 8 columns per thread.
template <typename T>
__global__ __launch_bounds__(256) void prod_reduce_kernel(const ProdArgs a) {
  const int per_row = (a.N + 7) / 8, groups = a.groups > 0 ? a.groups : 1;
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
  if (id >= (long long)groups * a.M * per_row) return;
  const long long row = id / per_row;
  const int n = (int)(id % per_row) * 8;
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s) {
    const float* from = a.partial + ((long long)s * groups * a.M + row) * a.N + n;
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
  const long long e = row / a.M, m = row - e * a.M;
  char* D = static_cast<char*>(a.D) + e * a.strideD * (a.out32 ? 4 : (int)sizeof(T));
  finish8<T>(a, a.bias, D, m, n, v);
}

}  // namespace layers
}  // namespace pgemm
