// Gated products: Y = act(X Wg + bg) * (X Wu + bu), and the gradient of X,
// dX = dZg Wg^T + dZu Wu^T.  Either is one product whose right operand comes from two
// weights: the first takes both weights' columns side by side, the second sums
// over both weights' columns one after the other.  Tiles, LDS layout and pipeline are
// those of prod_tile.hpp.
//
// Large products are bound by the matrix cores at the power-limited clock, as there.  The
// tile kernel here takes what pair_whole_kernel does not: rows that are not whole chunks and
// that are not copied into such, through registers (512 x 2047 x 2047 n x k 23.4 us, 0.37
// PFLOP/s), and strides beyond its offsets.
#pragma once

#include "../layers/prod_rows.hpp"
#include "rows8.hpp"

namespace pgemm {
namespace blocks {

using namespace layers;

enum Pair { kColumns = 0, kHalves = 1, kApart = 2 };

struct PairArgs {
  ProdArgs p;             // B: the first weight; N: outputs; K: summed (kHalves: of both)
  const void* B2;         // the second weight, in the first one's order and ld
  // kApart (pair_whole_kernel alone): `count` (1, 2) products of one shape, the second of A2
  // and B2 into D2
  const void* A2;
  void* D2;
  int count;
  // kColumns: the second weight's bias and pre-activations
  const void* bias2;
  void* Z2;
  long long ldz2;
  // kHalves: the first `half` summed indices are the first weight's, of which `inner`
  // exist; half is a multiple of the kernels' steps
  int half, inner;
};

// The right operand's loads, tile after tile of the summed index (see Loader).
//
// kColumns: of a wave's CB blocks of 16 output indices the first half are the first
// weight's, the others the same columns of the second; the tile holds EXT / 2
// columns from `first` on.
// kHalves: output indices from `first` on; the addresses go on from the first
// weight to the second by a constant, since both have one ld.
template <typename T, int ORDER, int EXT, int NT, int LOADING, int PAIR, int CB>
struct PairLoader {
  static constexpr bool DIRECT = LOADING != kThrough;
  using Tile = OperandTile<T, ORDER, EXT, NT>;
  static constexpr int L = Tile::LOADS, BK = Tile::BK, V = Tile::V;
  const T* base[2];
  long long ld;
  int first, n;                    // first output index; how many there are
  int half, inner;                 // summed indices of a weight (kColumns: half unused)
  int k;                           // first summed index of the next load
  long long step, jump;            // elements per tile; to the second weight
  const T* ptr[L];
  u32x4 reg[DIRECT ? 1 : L];

  // Weight and column of the tile's output index j.
  __device__ __forceinline__ void place(int j, int* w, int* col) const {
    if constexpr (PAIR == kColumns) {
      const int p = j / 16, in = p % CB;
      *w = in >= CB / 2;
      *col = first + (p / CB * (CB / 2) + in % (CB / 2)) * 16 + j % 16;
    } else {
      *w = k >= half;
      *col = first + j;
    }
  }
  // The next load's first summed index within its weight.
  __device__ __forceinline__ int within() const {
    return PAIR == kHalves && k >= half ? k - half : k;
  }

  __device__ __forceinline__ void init(const PairArgs& a, int first_out, int k_lo, int k_hi) {
    base[0] = static_cast<const T*>(a.p.B);
    base[1] = static_cast<const T*>(a.B2);
    ld = a.p.ldb;
    first = first_out;
    n = a.p.N;
    half = a.half;
    inner = PAIR == kHalves ? a.inner : k_hi;
    k = k_lo;
    const int at = within();
#pragma unroll
    for (int j = 0; j < L; ++j) {
      int r, c, w, col;
      Tile::slot(j * NT + (int)threadIdx.x, &r, &c);
      place(ORDER == kInner ? r : c * V, &w, &col);
      const T* b = w ? base[1] : base[0];
      if constexpr (ORDER == kInner) {
        ptr[j] = b + (long long)(col < n ? col : n - 1) * ld + at + c * V;
      } else {
        ptr[j] = b + (col < n ? col : 0) + (long long)(at + r) * ld;
      }
    }
    step = ORDER == kInner ? BK : BK * ld;
    jump = PAIR == kHalves ? (base[1] - base[0]) - (ORDER == kInner ? half : half * ld) : 0;
  }

  // Chunks J0 .. J1-1 of the load of summed indices k .. k+BK-1.
  template <int J0, int J1>
  __device__ __forceinline__ void load(char* lds) {
    const int at = within();
    const long long move = step + (PAIR == kHalves && k + BK == half ? jump : 0);
    if constexpr (LOADING == kDirect) {
      load_as<false, J0, J1>(lds, at, move);
    } else if constexpr (LOADING == kRagged) {
      if (at + BK + V >= inner) load_guards<J0, J1>(lds, at, move);
      else load_as<true, J0, J1>(lds, at, move);
    } else {
      const bool edge = ORDER == kOuter && first + (PAIR == kColumns ? EXT / 2 : EXT) > n;
      if (edge || at + BK > inner) load_as<false, J0, J1>(lds, at, move);
      else load_as<true, J0, J1>(lds, at, move);
    }
    if constexpr (J1 == L) k += BK;
  }

  template <bool WHOLE, int J0, int J1>
  __device__ __forceinline__ void load_as(char* lds, int at, long long move) {
#pragma unroll
    for (int j = J0; j < J1; ++j) {
      int r, c;
      Tile::slot(j * NT + (int)threadIdx.x, &r, &c);
      if constexpr (DIRECT) {
        const void* from = ptr[j];
        if constexpr (!WHOLE) {
          const bool in = at + (ORDER == kInner ? c * V : r) < inner;
          from = in ? from : (const void*)&kZeroChunk;
        }
        load_to_lds(from, lds + (j * NT + ((int)threadIdx.x & ~63)) * 16);
      } else if constexpr (WHOLE) {
        reg[j] = load16(ptr[j]);
      } else {
        reg[j] = guarded(ptr[j], r, c, at);
      }
      ptr[j] += move;
    }
  }

  __device__ __forceinline__ u32x4 guarded(const T* p, int r, int c, int at) const {
    if constexpr (ORDER == kInner) {
      const int i = at + c * V;
      return load_guarded(p - i, i, inner);
    } else {
      int w, col;
      place(c * V, &w, &col);
      const T* b = w ? base[1] : base[0];
      return load_edge(p, at + r < inner ? n - col : 0, b + (long long)(inner - 1) * ld + n);
    }
  }

  template <int J0, int J1>
  __device__ __forceinline__ void load_guards(char* lds, int at, long long move) {
    if constexpr (J0 < J1) wait_loads<0>();
#pragma unroll
    for (int j = J0; j < J1; ++j) {
      int r, c;
      Tile::slot(j * NT + (int)threadIdx.x, &r, &c);
      *reinterpret_cast<u32x4*>(lds + (j * NT + (int)threadIdx.x) * 16) = guarded(ptr[j], r, c, at);
      ptr[j] += move;
    }
  }

  __device__ __forceinline__ void store(char* lds) {
    if constexpr (!DIRECT) {
#pragma unroll
      for (int j = 0; j < L; ++j)
        *reinterpret_cast<u32x4*>(lds + (j * NT + (int)threadIdx.x) * 16) = reg[j];
    }
  }
};

// Eight gated results of row m from column n on, from the sums of both weights: adds
// the biases, keeps the pre-activations, and rounds the product of the
// activation and the other once.
template <typename T>
__device__ __forceinline__ void finish_gate(const PairArgs& args, long long m, int n, float* g,
                                            float* u, const float* bg, const float* bu) {
  const ProdArgs& a = args.p;
  constexpr int Whole = sizeof(T) == 4 ? kExact : kFine;   // fp32 results
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    g[j] += bg[j];
    u[j] += bu[j];
  }
  if (a.Z != nullptr) put_row8<T>(a.Z, m * a.ldz, n, a.N, g);
  if (args.Z2 != nullptr) put_row8<T>(args.Z2, m * args.ldz2, n, a.N, u);
  if (a.act != kNone) {
    if (sizeof(T) == 2 && !a.out32) act8<kFast>(g, a.act);
    else act8<Whole>(g, a.act);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) g[j] *= u[j];
  if (a.out32) put_row8<float>(a.D, m * a.ldd, n, a.N, g);
  else put_row8<T>(a.D, m * a.ldd, n, a.N, g);
}

// A split's sums of weight w to its partial sums.
__device__ __forceinline__ void put_partial(const ProdArgs& a, int split, int w, long long m, int n,
                                            const float* v) {
  put_row8<float>(a.partial, ((2LL * split + w) * a.M + m) * a.N, n, a.N, v);
}

template <typename T>
__device__ __forceinline__ void gate_bias(const PairArgs& a, int n, float* bg, float* bu) {
  load_bias<T>(a.p, a.p.bias, n, bg);
  load_bias<T>(a.p, a.bias2, n, bu);
}

// The K loop's reasons are with prod_tile_kernel, which it follows.
template <typename T, int LB, int BM, int BN, int WGM, int WGN, int LOADING, int PAIR>
__global__ __launch_bounds__(WGM* WGN * 64) void pair_tile_kernel(const PairArgs args) {
  const ProdArgs& a = args.p;
  constexpr bool DIRECT = LOADING != kThrough;
  constexpr int NT = WGM * WGN * 64;
  constexpr int WM = BM / WGM, WN = BN / WGN, RB = WM / 16, CB = WN / 16;
  constexpr int BK = 128 / (int)sizeof(T);
  constexpr int SLOT = (BM > BN ? BM : BN) * 128;   // one operand's tile
  constexpr int SLOTS = DIRECT ? 5 : 4;
  constexpr int EPI_LD = WN + 4;
  constexpr int EPI = WGM * WGN * 32 * EPI_LD * 4;   // 32 rows per wave
  constexpr int LDS = SLOTS * SLOT > EPI ? SLOTS * SLOT : EPI;
  __shared__ __attribute__((aligned(128))) char lds[LDS];

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = (wave / WGN) * WM, wn = (wave % WGN) * WN;
  constexpr int COLS = PAIR == kColumns ? BN / 2 : BN;   // results of a tile
  int tm, tn, k_lo = 0, k_hi = a.K;
  map_tile(blockIdx.x, a.tiles_m, a.tiles_n, &tm, &tn);
  const int row0 = tm * BM, col0 = tn * COLS;
  if (a.splits > 1) {
    k_lo = blockIdx.y * a.k_split;
    k_hi = k_lo + a.k_split < a.K ? k_lo + a.k_split : a.K;
  }

  using TA = OperandTile<T, kInner, BM, NT>;
  using TB = OperandTile<T, LB, BN, NT>;
  using LoadA = Loader<T, kInner, BM, NT, LOADING, false>;
  using LoadB = PairLoader<T, LB, BN, NT, LOADING, PAIR, CB>;
  LoadA la;
  LoadB lb;
  la.init({static_cast<const T*>(a.A), a.lda, a.M, k_hi, nullptr, 0}, row0, k_lo);
  lb.init(args, col0, k_lo, k_hi);

  f32x4 acc[RB][CB];
#pragma unroll
  for (int r = 0; r < RB; ++r)
#pragma unroll
    for (int c = 0; c < CB; ++c) acc[r][c] = f32x4{0, 0, 0, 0};

  constexpr int GP = RB / 2, G = 2 * GP;
  static_assert(RB % 2 == 0 && (G == 2 || G % 4 == 0), "the loads' places below");
  u32x4 fa[2][2], fb[2][CB];
  auto read_a = [&](const char* a_slot, int g) {
    fa[g & 1][0] = TA::frag(a_slot, wm, 2 * (g % GP), g / GP);
    fa[g & 1][1] = TA::frag(a_slot, wm, 2 * (g % GP) + 1, g / GP);
  };
  auto read_b = [&](const char* b_slot, int step) {
#pragma unroll
    for (int c = 0; c < CB; ++c) fb[step][c] = TB::frag(b_slot, wn, c, step);
  };
  auto slot = [&](int i) { return lds + (i >= SLOTS ? i - SLOTS : i) * SLOT; };
  constexpr int HA = LoadA::L / 2, HB = LoadB::L / 2;

  const int nk = (k_hi - k_lo + BK - 1) / BK;
  if (nk > 0) {
    la.template load<0, LoadA::L>(slot(0));
    lb.template load<0, LoadB::L>(slot(1));
    if constexpr (DIRECT) {
      la.template load<0, LoadA::L>(slot(2));
      lb.template load<0, HB>(slot(3));
      wait_loads<LoadA::L + HB>();
    } else {
      la.store(slot(0));
      lb.store(slot(1));
      if (nk > 1) {
        la.template load<0, LoadA::L>(nullptr);
        lb.template load<0, LoadB::L>(nullptr);
      }
    }
    workgroup_barrier();
    read_a(slot(0), 0);
    read_b(slot(1), 0);
    int at = 0;                                // slot of A(kt)
    for (int kt = 0; kt < nk; ++kt) {
      char *const a0 = slot(at), *const b0 = slot(at + 1);
      char *const a1 = slot(at + 2), *const b1 = slot(at + 3);
      char *const a2 = slot(at + 4), *const b2 = a0;
      at = at + 2 >= SLOTS ? at + 2 - SLOTS : at + 2;
      if constexpr (!DIRECT) {
        if (kt + 1 < nk) {
          la.store(a1);
          lb.store(b1);
        }
        if (kt + 2 < nk) {
          la.template load<0, LoadA::L>(nullptr);
          lb.template load<0, LoadB::L>(nullptr);
        }
      }
      static_for<G>([&](auto gc) {
        constexpr int g = decltype(gc)::value, step = g / GP, p = g % GP;
        if constexpr (g == G - 1) {
          if constexpr (DIRECT) wait_loads<LoadA::L>();
          workgroup_barrier();
          read_a(a1, 0);          // past the last tile: some LDS, never used
          read_b(b1, 0);
        } else {
          read_a(a0, g + 1);
          if constexpr (p == GP - 1) read_b(b0, 1);
        }
        constexpr int Q = G < 4 ? 1 : G / 4, q = g / Q, h = g % Q;
        constexpr int IB = LoadB::L - HB, IA = LoadA::L - HA;
        if constexpr (DIRECT && G == 2) {
          if constexpr (g == 0) {
            lb.template load<HB, LoadB::L>(b1);
            la.template load<0, LoadA::L>(a2);
          } else {
            lb.template load<0, HB>(b2);
          }
        } else if constexpr (DIRECT) {
          if constexpr (q == 0) lb.template load<HB + IB * h / Q, HB + IB*(h + 1) / Q>(b1);
          if constexpr (q == 1) la.template load<HA * h / Q, HA*(h + 1) / Q>(a2);
          if constexpr (q == 2) la.template load<HA + IA * h / Q, HA + IA*(h + 1) / Q>(a2);
          if constexpr (g == G - 1) lb.template load<0, HB>(b2);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int c = 0; c < CB; ++c)
            acc[2 * p + r][c] = Elem<T>::mfma(fb[step][c], fa[g & 1][r], acc[2 * p + r][c]);
        constexpr int loads = !DIRECT        ? 0
                              : G == 2       ? (g == 0 ? LoadA::L + IB : HB)
                              : g == G - 1   ? HB
                              : q == 3       ? 0
                              : q == 0       ? IB / Q
                                             : HA / Q;
        spread<2 * TA::READS + (p == GP - 1 ? CB * TB::READS : 0), 2 * CB * Elem<T>::kMfmas,
               loads>();
        __builtin_amdgcn_sched_barrier(0);
      });
    }
    if constexpr (DIRECT) wait_loads<0>();     // the loads past the end
  }
  __syncthreads();   // the operands' LDS becomes the epilogue's

  // Epilogue: 32 rows of the wave tile at a time through the wave's own LDS, so that
  // each lane finishes 8 consecutive columns with 16-byte accesses.
  float* stg = reinterpret_cast<float*>(lds) + wave * 32 * EPI_LD;
  constexpr int WC = PAIR == kColumns ? WN / 2 : WN;               // results of a wave's row
  constexpr int LPR = WC / 8, RPP = 64 / LPR, PASSES = 32 / RPP;   // lanes per row, rows per pass
  const int col = (lane % LPR) * 8, n = col0 + (wn / WN) * WC + col;
  float bg[8], bu[8];
  if constexpr (PAIR == kColumns) {
    if (a.splits <= 1) gate_bias<T>(args, n, bg, bu);
  }
#pragma unroll 1
  for (int r = 0; r < RB / 2; ++r) {
    const int m0 = row0 + wm + 32 * r + lane / LPR;
    static_for<RB / 2>([&](auto rc) {
      constexpr int q = decltype(rc)::value;
      if (r == q) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int c = 0; c < CB; ++c)
            *reinterpret_cast<f32x4*>(stg + (16 * h + (lane & 15)) * EPI_LD + 16 * c +
                                      4 * (lane >> 4)) = acc[2 * q + h][c];
      }
    });
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const float* from = stg + (p * RPP + lane / LPR) * EPI_LD + col;
      const int m = m0 + p * RPP;
      if (m < a.M && n < a.N) {
        float v[8], u[8];
        *reinterpret_cast<f32x4*>(v) = *reinterpret_cast<const f32x4*>(from);
        *reinterpret_cast<f32x4*>(v + 4) = *reinterpret_cast<const f32x4*>(from + 4);
        if constexpr (PAIR == kColumns) {
          *reinterpret_cast<f32x4*>(u) = *reinterpret_cast<const f32x4*>(from + WC);
          *reinterpret_cast<f32x4*>(u + 4) = *reinterpret_cast<const f32x4*>(from + WC + 4);
          if (a.splits > 1) {
            put_partial(a, blockIdx.y, 0, m, n, v);
            put_partial(a, blockIdx.y, 1, m, n, u);
          } else {
            finish_gate<T>(args, m, n, v, u, bg, bu);
          }
        } else if (a.splits > 1) {
          put_row8<float>(a.partial, ((long long)blockIdx.y * a.M + m) * a.N, n, a.N, v);
        } else {
          put_row8<T>(a.D, m * a.ldd, n, a.N, v);
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// Few rows: M of at most 16 MB (few_plan) against both weights, bound by reading those once.  A
// workgroup takes 8 NB columns of each (NB / 2 blocks of 16 of either); see
// prod_rows_kernel, which it follows.  One row, 4096 to 8192, bf16: 24.9 us (134 MB of
// weights: 5.4 TB/s, part of it from the last-level cache; three pairs of weights in turn,
// which that cache does not hold, 28.9 us and 4.6, where a copy reaches 5.0).
template <typename T, int LB, int MB, int NB, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void gate_rows_kernel(const PairArgs args) {
  const ProdArgs& a = args.p;
  constexpr int BN = 16 * NB, COLS = BN / 2;
  constexpr int U = NB == 2 && MB == 1 ? 2 : 1;          // units per load
  constexpr int V = 16 / (int)sizeof(T), BK = 128 / (int)sizeof(T);
  constexpr int RED_LD = BN + 4, RED = WAVES * MB * 16 * RED_LD * 4;
  constexpr int STG = LB == kOuter ? WAVES * BN * 128 : 0;
  constexpr int LDS = RED > STG ? RED : STG;
  __shared__ __attribute__((aligned(128))) char lds[LDS];
  using TB = OperandTile<T, kOuter, BN, 64>;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, i = lane & 15;
  const int col0 = map_range(blockIdx.x, gridDim.x) * COLS;
  int k_lo = 0, k_hi = a.K;
  if (a.splits > 1) {
    k_lo = blockIdx.y * a.k_split;
    k_hi = k_lo + a.k_split < a.K ? k_lo + a.k_split : a.K;
  }
  // units loaded without guards, and those at the end that need them
  const int units = (k_hi - k_lo + BK - 1) / BK;
  int whole = (k_hi - k_lo) / BK;
  if (LB == kOuter && col0 + COLS > a.N) {
    const int inside = a.K - V - k_lo;
    whole = inside < 0 ? 0 : (inside / BK < whole ? inside / BK : whole);
  }
  constexpr int BL = 2 * NB;                    // loads of B per unit and lane
  const T* bptr[LB == kInner ? NB : BL];        // without the summed index
  auto weight = [&](int block) { return static_cast<const T*>(block >= NB / 2 ? args.B2 : a.B); };
  auto column = [&](int c) { return col0 + 16 * (c / 16 % (NB / 2)) + c % 16; };
#pragma unroll
  for (int c = 0; c < (LB == kInner ? NB : BL); ++c) {
    if constexpr (LB == kInner) {
      const int n = column(16 * c + i);
      bptr[c] = weight(c) + (long long)(n < a.N ? n : a.N - 1) * a.ldb;
    } else {
      int r, q;
      TB::slot(c * 64 + lane, &r, &q);
      const int n = column(q * V);
      bptr[c] = weight(q * V / 16) + (long long)r * a.ldb + (n < a.N ? n : 0);
    }
  }

  const T* arow[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    const int m = 16 * b + i;
    arow[b] = static_cast<const T*>(a.A) + (long long)(m < a.M ? m : a.M - 1) * a.lda;
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
    u32x4 rb[BL], ra[MB][2];
#pragma unroll
    for (int q = 0; q < BL; ++q) {
      if constexpr (LB == kInner) {
        rb[q] = load_guarded(bptr[q >> 1], k0 + (4 * (q & 1) + g) * V, k_hi);
      } else {
        int r, c;
        TB::slot(q * 64 + lane, &r, &c);
        const T* row = k0 + r < k_hi ? weight(c * V / 16) + (long long)(k0 + r) * a.ldb : nullptr;
        rb[q] = load_guarded(row, column(c * V), a.N);
      }
    }
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) ra[b][kk] = load_guarded(arow[b], k0 + (4 * kk + g) * V, k_hi);
    use(rb, ra);
  }

  // sum over the waves, then 8 columns of both weights per thread
  __syncthreads();
  float* red = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int c = 0; c < NB; ++c)
      *reinterpret_cast<f32x4*>(red + ((wave * MB + b) * 16 + i) * RED_LD + 16 * c + 4 * g) =
          acc[b][c];
  __syncthreads();
  for (int t = threadIdx.x; t < MB * 16 * (COLS / 8); t += WAVES * 64) {
    const int m = t / (COLS / 8), col = (t % (COLS / 8)) * 8, n = col0 + col;
    if (m < a.M && n < a.N) {
      float v[8] = {0, 0, 0, 0, 0, 0, 0, 0}, u[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        const float* from = red + (w * MB * 16 + m) * RED_LD + col;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[j] += from[j];
          u[j] += from[COLS + j];
        }
      }
      if (a.splits > 1) {
        put_partial(a, blockIdx.y, 0, m, n, v);
        put_partial(a, blockIdx.y, 1, m, n, u);
      } else {
        float bg[8], bu[8];
        gate_bias<T>(args, n, bg, bu);
        finish_gate<T>(args, m, n, v, u, bg, bu);
      }
    }
  }
}

// Sums the splits in order and finishes: 8 columns per thread.
template <typename T>
__global__ __launch_bounds__(256) void gate_reduce_kernel(const PairArgs args) {
  const ProdArgs& a = args.p;
  const int per_row = (a.N + 7) / 8;
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
  if (id >= (long long)a.M * per_row) return;
  const long long m = id / per_row;
  const int n = (int)(id % per_row) * 8;
  float v[2][8] = {{0, 0, 0, 0, 0, 0, 0, 0}, {0, 0, 0, 0, 0, 0, 0, 0}};
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s)
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      float x[8];
      get_row8<float>(a.partial, ((2LL * s + w) * a.M + m) * a.N, n, a.N, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[w][j] += x[j];
    }
  float bg[8], bu[8];
  gate_bias<T>(args, n, bg, bu);
  finish_gate<T>(args, m, n, v[0], v[1], bg, bu);
}

// Sums the splits of the other products (blockIdx.y: of the first or the second).
template <typename T>
__global__ __launch_bounds__(256) void pair_reduce_kernel(const PairArgs args) {
  const ProdArgs& a = args.p;
  const int per_row = (a.N + 7) / 8, count = gridDim.y, w = blockIdx.y;
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
  if (id >= (long long)a.M * per_row) return;
  const long long m = id / per_row;
  const int n = (int)(id % per_row) * 8;
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s) {
    float x[8];
    get_row8<float>(a.partial, (((long long)s * count + w) * a.M + m) * a.N, n, a.N, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += x[j];
  }
  void* D = w == 0 ? a.D : args.D2;
  if (a.out32) put_row8<float>(D, m * a.ldd, n, a.N, v);
  else put_row8<T>(D, m * a.ldd, n, a.N, v);
}

struct GateSlopeArgs {
  const void* dY;
  const void* Zg;
  const void* Zu;
  void* dZ;               // m rows of ldd: dZg in the first `half` columns, dZu behind them
  long long ldy, ldg, ldu, ldd;
  int n, half, act, rows;
  int chunks;             // row chunks (grid y)
  int tpr;                // threads per row (a power of two, at most 64)
  float* partial;         // [chunk][weight][n] column sums (nullptr: not wanted)
};

// dZg = dY Zu act'(Zg) and dZu = dY act(Zg), each rounded once, zeros behind column n,
// and the column sums of a chunk of rows (before the rounding): see slope_kernel.  Bound by
// memory: 8192 x 8192 bf16 143 us (671 MB: 4.7 TB/s); two rows asked for at once 144.
//
// A kept pre-activation may be infinite although the result was finite (an fp16 sum
// beyond 65504).  Its products then take their limits: an activation far below 0 is 0, and
// what is multiplied by an exact 0 (of the slope or of dY) is 0, not NaN.  (3 us of the 832
// of 8192 x 4096 x 4096's gradients.  A branch around it where a chunk has no infinity, and
// a second pass over its rows for a thread whose sums became NaN, cost 2 to 4.)
template <typename T, int F>
__global__ __launch_bounds__(256) void gate_slope_kernel(const GateSlopeArgs a) {
  __shared__ float sums[256 * 8];
  const int r0 = (int)((long long)a.rows * blockIdx.y / a.chunks);
  const int r1 = (int)((long long)a.rows * (blockIdx.y + 1) / a.chunks);
  const int c = (blockIdx.x * a.tpr + threadIdx.x % a.tpr) * 8;
  const int rpb = 256 / a.tpr;
  const float inf = __builtin_inff();
  const float lowest = a.act == kNone ? -inf : -3.402823466e38f;   // where act_value has its limit
  float sg[8] = {0, 0, 0, 0, 0, 0, 0, 0}, su[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (c < a.half) {
#pragma unroll 2
    for (int r = r0 + threadIdx.x / a.tpr; r < r1; r += rpb) {
      Stored8<T> raw[3];
      rows8<T>(a.n, [&](auto get) {
        raw[0] = get(a.dY, (long long)r * a.ldy, c);
        raw[1] = get(a.Zg, (long long)r * a.ldg, c);
        raw[2] = get(a.Zu, (long long)r * a.ldu, c);
      });
      float d[8], g[8], u[8];
      settle8<T>(raw[0], c, a.n);
      settle8<T>(raw[1], c, a.n);
      settle8<T>(raw[2], c, a.n);
      widen8<T>(raw[0], d);
      widen8<T>(raw[1], g);
      widen8<T>(raw[2], u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float z = g[j], dj = d[j];
        const float s = act_slope<F>(z, a.act), v = act_value<F>(z < lowest ? lowest : z, a.act);
        g[j] = fabsf(u[j]) == inf && dj * s == 0.0f ? 0.0f : dj * u[j] * s;
        u[j] = fabsf(v) == inf && dj == 0.0f ? 0.0f : dj * v;
        if (c + j >= a.n) g[j] = u[j] = 0.0f;
        sg[j] += g[j];
        su[j] += u[j];
      }
      put8<T>(a.dZ, (long long)r * a.ldd + c, g);
      put8<T>(a.dZ, (long long)r * a.ldd + a.half + c, u);
    }
  }
  if (a.partial == nullptr) return;
  const int width = a.tpr * 8;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) sums[threadIdx.x * 8 + j] = w == 0 ? sg[j] : su[j];
    __syncthreads();
    for (int x = threadIdx.x; x < width; x += 256) {
      const int n = blockIdx.x * width + x;
      if (n >= a.n) break;
      float v = 0.0f;
      for (int r = 0; r < rpb; ++r) v += sums[r * width + x];
      a.partial[((long long)blockIdx.y * 2 + w) * a.n + n] = v;
    }
  }
}

// Matrices (blockIdx.y) with rows of ld elements into rows of ldt, a multiple of eight, zeros
// behind the columns: a workgroup takes 256 / tpr rows at once.
struct PadRowsArgs {
  struct {
    const void* from;
    void* to;
    long long ld, ldt;
    int rows, cols;
    int tpr;                // threads per row (a power of two, at most 256)
  } of[3];
};
template <typename T>
__global__ __launch_bounds__(256) void pad_rows_kernel(const PadRowsArgs args) {
  const auto& a = args.of[blockIdx.y];
  const int per = 256 / a.tpr, t = threadIdx.x & (a.tpr - 1);
  for (long long r = (long long)blockIdx.x * per + threadIdx.x / a.tpr; r < a.rows;
       r += (long long)gridDim.x * per)
    for (long long c = t * 8; c < a.ldt; c += a.tpr * 8) {
      Stored8<T> x;
      rows8<T>(a.cols, [&](auto get) { x = get(a.from, r * a.ld, (int)c); });
      settle8<T>(x, (int)c, a.cols);
      T* const to = static_cast<T*>(a.to) + r * a.ldt + c;
#pragma unroll
      for (int k = 0; k < (int)sizeof(T) / 2; ++k) layers::store16(to + k * 16 / sizeof(T), x.v[k]);
    }
}

}  // namespace blocks
}  // namespace pgemm
