// Products of 8-bit floating-point operands with a scale for each block of 128
// along the summed index:
//
//   D[i, j] = act( sum over blocks B of sx[i, B] sw[j, B] * (sum over k in B of
//             A[i, k] W[j, k]) + bias[j] ) + residual
//
// A (M x K) has a scale for each row's block; W (N x K) for each row's or for 128
// rows together.  Both are contiguous along the summed index.  The inner sums
// run on the matrix cores, a block of 128 at a time; each is then scaled and added in
// fp32 by the vector units, one fused multiply-add per result and block (two where
// every column has its own scale).
//
// For results of 16 bits the inner sums take the 8-bit instructions.  These form exact
// products, but add eight neighbouring ones after cutting each off at 2^-13 of the
// largest's power of two (measured, for the 128- and the 32-deep ones alike; the
// groups' sums and the addend are fp32): off by 1.4e-5 of the result (relative norm,
// random data), a hundredth of a bf16 rounding, and by 7 2^-12 of a group's largest
// product at most.  For fp32 results (WIDE) the operands become bf16 in registers,
// which holds every 8-bit number, and the 16-bit instructions add them in fp32, at
// half the rate.
#pragma once

#include "../layers/prod_tile.hpp"
#include "quantize.hpp"

namespace pgemm {
namespace blocks {

using namespace layers;

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct Prod8Args {
  ProdArgs p;             // A: X, B: W; bias, Z, R and D of `type` (p.out32: fp32)
  int type;               // of the result: 0 fp32 (WIDE), 1 fp16, 2 bf16
  const float* sx;        // scale of block b of row i at i * sx_row + b * sx_block
  const float* sw;        // of row j's (or of 128 rows') at j * sw_row + b * sw_block
  long long sx_row, sx_block, sw_row, sw_block;
  int w_shift;            // 7: 128 rows of W share a scale, 0: each has its own
};

// One lane's 32 numbers of a block of 128 of the summed index: as they are, or widened
// to bf16.  (Which 32 does not matter: both operands take the same ones.)
template <bool WIDE>
struct Part {
  u32x4 v[WIDE ? 4 : 2];
};

template <int F>
__device__ __forceinline__ uint32_t widen2(uint32_t four, bool high) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  bf16x2 r;
  if constexpr (F == kE4M3) {
    r = high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(four, 1.0f, true)
             : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(four, 1.0f, false);
  } else {
    r = high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(four, 1.0f, true)
             : __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(four, 1.0f, false);
  }
  return __builtin_bit_cast(uint32_t, r);
}

template <bool WIDE, int F>
__device__ __forceinline__ Part<WIDE> part(u32x4 a, u32x4 b) {
  Part<WIDE> p;
  if constexpr (WIDE) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t four = j < 4 ? a[j] : b[j - 4];
      p.v[j >> 1][2 * (j & 1)] = widen2<F>(four, false);
      p.v[j >> 1][2 * (j & 1) + 1] = widen2<F>(four, true);
    }
  } else {
    p.v[0] = a;
    p.v[1] = b;
  }
  return p;
}

// D(16 x 16) = A B over 128 of the summed index.
template <bool WIDE, int FA, int FB>
__device__ __forceinline__ f32x4 block_sum(const Part<WIDE>& a, const Part<WIDE>& b) {
  f32x4 d = {0, 0, 0, 0};
  if constexpr (WIDE) {
#pragma unroll
    for (int j = 0; j < 4; ++j) d = Elem<__bf16>::mfma(a.v[j], b.v[j], d);
    return d;
  } else {
    const i32x8 x = {(int)a.v[0][0], (int)a.v[0][1], (int)a.v[0][2], (int)a.v[0][3],
                     (int)a.v[1][0], (int)a.v[1][1], (int)a.v[1][2], (int)a.v[1][3]};
    const i32x8 y = {(int)b.v[0][0], (int)b.v[0][1], (int)b.v[0][2], (int)b.v[0][3],
                     (int)b.v[1][0], (int)b.v[1][1], (int)b.v[1][2], (int)b.v[1][3]};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, d, FA, FB, 0, 0, 0, 0);
  }
}

// 4 bytes per lane from its own address straight to LDS (see load_to_lds).
__device__ __forceinline__ void load4_to_lds(const void* from, char* to) {
  const int at = __builtin_amdgcn_readfirstlane(
      (int)(uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)to);
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dword %1, off"
      :
      : "s"(at), "v"(from));
}

// Eight sums of row m from column n on: a split's to its partial sums, the others
// through the epilogue.
template <bool WIDE>
__device__ __forceinline__ void finish8_any(const Prod8Args& args, long long m, int n, const float* v,
                                            int split) {
  const ProdArgs& a = args.p;
  if (a.splits > 1) {
    float* to = a.partial + (split * (long long)a.M + m) * a.N + n;
    if (n + 8 <= a.N) {
      put8<float>(to, 0, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (n + j < a.N) to[j] = v[j];
    }
  } else if constexpr (WIDE) {
    finish8<float>(a, a.bias, a.D, m, n, v);
  } else if (args.type == 2) {
    finish8<__bf16>(a, a.bias, a.D, m, n, v);
  } else {
    finish8<_Float16>(a, a.bias, a.D, m, n, v);
  }
}

// The tile kernel: BM x BN of D per workgroup.
//
// One tile of the summed index is a block of 128: 128 bytes of each row.  Of the
// LDS, four slots hold A and W of this tile and the next, two small stages the
// scales of their rows.  A wave's W operands of a tile stay in registers (CB x 8),
// read at the end of the tile before, so that W's slot is free for the tile after
// next almost a whole tile early; A's blocks are read one ahead of their use.  Two
// barriers a tile: M, behind the first block, frees W's slot; E, before the last,
// frees A's and waits for the next tile (for A's loads, the younger ones; W's of
// the tile after next may be in flight).
//
// A block's sums are scaled and added while the matrix cores run the next
// block's, so that neither waits for the other.  fp32 results of 4096^3 take 143 to 155 us
// (0.9 to 0.96 PFLOP/s of the 16-bit instructions' 2.5, with widening in the vector units),
// 16-bit ones prod8_whole_kernel's 66.  Rows that are not whole chunks (DIRECT false) are loaded
// through guards and stored at once, a memory latency a tile: 8191 x 8192 x 4095 948 us, fp32
// results 1255; 1000 x 1000 x 1001 14.7 and 16.5, where k = 1008 takes 9.0 and 9.3.
template <int FA, int FB, int BM, int BN, int WGM, int WGN, bool DIRECT, bool COLS, bool WIDE>
__global__ __launch_bounds__(WGM* WGN * 64) void prod8_tile_kernel(const Prod8Args args) {
  const ProdArgs& a = args.p;
  constexpr int NT = WGM * WGN * 64;
  constexpr int WM = BM / WGM, WN = BN / WGN, RB = WM / 16, CB = WN / 16;
  constexpr int BK = 128;
  constexpr int SLOT_A = BM * BK, SLOT_B = BN * BK, SCALES = (BM + BN) * 4;
  constexpr int OPERANDS = 2 * (SLOT_A + SLOT_B + SCALES);
  constexpr int EPI_LD = WN + 4, EPI = WGM * WGN * 32 * EPI_LD * 4;   // 32 rows per wave
  constexpr int LDS = OPERANDS > EPI ? OPERANDS : EPI;
  static_assert(LDS <= 160 * 1024 && BM + BN <= NT, "of a compute unit; one scale a thread");
  static_assert(RB % 2 == 0, "the epilogue's pairs of blocks");
  __shared__ __attribute__((aligned(128))) char lds[LDS];

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i16 = lane & 15, g4 = lane >> 4;
  const int wm = (wave / WGN) * WM, wn = (wave % WGN) * WN;
  int tm, tn, k_lo = 0, k_hi = a.K;
  map_tile(blockIdx.x, a.tiles_m, a.tiles_n, &tm, &tn);
  if (a.splits > 1) {
    k_lo = blockIdx.y * a.k_split;
    k_hi = k_lo + a.k_split < a.K ? k_lo + a.k_split : a.K;
  }
  const int row0 = tm * BM, col0 = tn * BN;

  using TA = OperandTile<uint8_t, kInner, BM, NT>;
  using TB = OperandTile<uint8_t, kInner, BN, NT>;
  using LoadA = Loader<uint8_t, kInner, BM, NT, DIRECT ? kDirect : kThrough, false>;
  using LoadB = Loader<uint8_t, kInner, BN, NT, DIRECT ? kDirect : kThrough, false>;
  LoadA la;
  LoadB lb;
  la.init({static_cast<const uint8_t*>(a.A), a.lda, a.M, k_hi, nullptr, 0}, row0, k_lo);
  lb.init({static_cast<const uint8_t*>(a.B), a.ldb, a.N, k_hi, nullptr, 0}, col0, k_lo);

  const int b_lo = k_lo / BK, nk = (k_hi - k_lo + BK - 1) / BK;
  // this thread's scale: of a row of A or of W
  const float* scale;
  long long scale_step;
  {
    const int t = threadIdx.x;
    if (t < BM) {
      const int r = row0 + t < a.M ? row0 + t : a.M - 1;
      scale = args.sx + r * args.sx_row;
      scale_step = args.sx_block;
    } else {
      const int c = col0 + (t - BM) < a.N ? col0 + (t - BM) : a.N - 1;
      scale = args.sw + (c >> args.w_shift) * args.sw_row;
      scale_step = args.sw_block;
    }
    scale += b_lo * scale_step;
  }

  char* const slot_a = lds;
  char* const slot_b = lds + 2 * SLOT_A;
  char* const slot_s = lds + 2 * (SLOT_A + SLOT_B);
  int kb = 0;                       // the tile whose scales are loaded next
  auto load_a = [&](int at) {       // A and the scales, into slot `at`
    if constexpr (DIRECT) {
      la.template load<0, LoadA::L>(slot_a + at * SLOT_A);
    } else {
      la.template load_guards<0, LoadA::L>(slot_a + at * SLOT_A);
      la.k += BK;
    }
    if (BM + BN == NT || (wave << 6) < BM + BN) {
      if constexpr (DIRECT) {
        load4_to_lds(scale, slot_s + at * SCALES + (wave << 8));
      } else {
        *reinterpret_cast<float*>(slot_s + at * SCALES + threadIdx.x * 4) = *scale;
      }
    }
    if (++kb < nk) scale += scale_step;       // past the end: the last again
  };
  auto load_b = [&](int at) {
    if constexpr (DIRECT) {
      lb.template load<0, LoadB::L>(slot_b + at * SLOT_B);
    } else {
      lb.template load_guards<0, LoadB::L>(slot_b + at * SLOT_B);
      lb.k += BK;
    }
  };

  f32x4 acc[RB][CB];
#pragma unroll
  for (int r = 0; r < RB; ++r)
#pragma unroll
    for (int c = 0; c < CB; ++c) acc[r][c] = f32x4{0, 0, 0, 0};

  if (nk > 0) {
    load_a(0);
    load_b(0);
    load_b(1);
    load_a(1);
    // all but the second tile (waves without scales have one load less)
    if constexpr (DIRECT) wait_loads<LoadA::L + LoadB::L>();
    workgroup_barrier();

    u32x4 fa[2][2], fb[CB][2];
    Part<WIDE> wb[CB];
    f32x4 sum[CB];
    float px[RB], last = 0.0f;                  // scales of this tile's rows; of the last block's
    f32x4 pw[COLS ? CB : 1];
    auto read_a = [&](const char* from, int g) {
      fa[g & 1][0] = TA::frag(from, wm, g, 0);
      fa[g & 1][1] = TA::frag(from, wm, g, 1);
    };
    auto read_b = [&](const char* from, int c) {
      fb[c][0] = TB::frag(from, wn, c, 0);
      fb[c][1] = TB::frag(from, wn, c, 1);
    };
    // block (r, c)'s sums times their scale
    auto add = [&](int r, int c, float p) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (COLS) acc[r][c][j] += sum[c][j] * (p * pw[c][j]);
        else acc[r][c][j] += sum[c][j] * p;
      }
    };
    read_a(slot_a, 0);
#pragma unroll
    for (int c = 0; c < CB; ++c) {
      read_b(slot_b, c);
      sum[c] = f32x4{0, 0, 0, 0};
    }
    for (int t = 0; t < nk; ++t) {
      const int at = t & 1;
      const char *const a0 = slot_a + at * SLOT_A, *const a1 = slot_a + (at ^ 1) * SLOT_A;
      const char* const b1 = slot_b + (at ^ 1) * SLOT_B;
      const float* const sc = reinterpret_cast<const float*>(slot_s + at * SCALES);
      // the scales of this tile
      if constexpr (COLS) {
#pragma unroll
        for (int c = 0; c < CB; ++c)
          pw[c] = *reinterpret_cast<const f32x4*>(sc + BM + wn + 16 * c + 4 * g4);
#pragma unroll
        for (int r = 0; r < RB; ++r) px[r] = sc[wm + 16 * r + i16];
      } else {
        const float w = sc[BM + wn];
#pragma unroll
        for (int r = 0; r < RB; ++r) px[r] = sc[wm + 16 * r + i16] * w;
      }
      if constexpr (WIDE) {                     // once a tile (not widened: fb itself)
#pragma unroll
        for (int c = 0; c < CB; ++c) wb[c] = part<WIDE, FB>(fb[c][0], fb[c][1]);
      }
      static_for<RB>([&](auto gc) {
        constexpr int g = decltype(gc)::value;
        if constexpr (g == 1) {
          workgroup_barrier();                  // M: W's slot is free
          load_b(at);
        }
        if constexpr (g == RB - 1) {
          // E: A's slot is free, the next tile is there
          if constexpr (DIRECT) wait_loads<LoadB::L>();
          workgroup_barrier();
          load_a(at);
          read_a(a1, 0);                        // past the last tile: some LDS, never used
        } else {
          read_a(a0, g + 1);
        }
        const Part<WIDE> xa = part<WIDE, FA>(fa[g & 1][0], fa[g & 1][1]);
#pragma unroll
        for (int c = 0; c < CB; ++c) {
          // the block before (in the first: the last of the tile before; with a scale
          // for each column, the registers that would hold both tiles' are not there)
          if constexpr (g > 0) add(g - 1, c, px[g - 1]);
          else if constexpr (!COLS) add(RB - 1, c, last);
          if constexpr (!WIDE) wb[c] = part<WIDE, FB>(fb[c][0], fb[c][1]);
          sum[c] = block_sum<WIDE, FB, FA>(wb[c], xa);
          if constexpr (g == RB - 1) read_b(b1, c);
        }
        __builtin_amdgcn_sched_barrier(0);
      });
      last = px[RB - 1];
      if constexpr (COLS) {
#pragma unroll
        for (int c = 0; c < CB; ++c) add(RB - 1, c, last);
      }
    }
    if constexpr (!COLS) {
#pragma unroll
      for (int c = 0; c < CB; ++c) add(RB - 1, c, last);
    }
    if constexpr (DIRECT) wait_loads<0>();      // the loads past the end
  }
  __syncthreads();   // the operands' LDS becomes the epilogue's

  // Epilogue: 32 rows of the wave tile at a time through the wave's own LDS, so that
  // each lane finishes 8 consecutive columns with 16-byte accesses.
  float* stg = reinterpret_cast<float*>(lds) + wave * 32 * EPI_LD;
  constexpr int LPR = WN / 8, RPP = 64 / LPR, PASSES = 32 / RPP;   // lanes per row, rows per pass
  const int col = (lane % LPR) * 8, n = col0 + wn + col;
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
            *reinterpret_cast<f32x4*>(stg + (16 * h + i16) * EPI_LD + 16 * c + 4 * g4) =
                acc[2 * q + h][c];
      }
    });
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll 1
    for (int p = 0; p < PASSES; ++p) {
      const float* from = stg + (p * RPP + lane / LPR) * EPI_LD + col;
      const f32x4 x = *reinterpret_cast<const f32x4*>(from);
      const f32x4 y = *reinterpret_cast<const f32x4*>(from + 4);
      const int m = m0 + p * RPP;
      if (m < a.M && n < a.N) {
        float v[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
        finish8_any<WIDE>(args, m, n, v, blockIdx.y);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// Few rows: M of at most 16 MB (few_plan) against all of W, bound by reading W once.  A
// workgroup takes 16 NB columns; its waves take blocks of 128 of the summed index
// in turn (U of them in flight), from memory straight into the matrix
// instruction's registers, each adding into its own sums, which are added over
// the waves through LDS in a fixed order.  The scales of all its blocks are read
// once into LDS, under the first blocks' loads (one by one, each row's would be a
// cache line for itself), where they fit.  16 x 4096 x 4096 8.7 us back to back, 8.0 in a trace
// (17 MB of W: 2 TB/s; there a launch of one workgroup over a row takes 2.7, the bf16 product
// of these sizes 11.2): latency, since a wave's second blocks are asked for behind the
// barrier of the scales, and each workgroup reads X as well, as many bytes as its part of W.
template <int FA, int FB, int MB, int NB, int WAVES, bool COLS, bool WIDE>
__global__ __launch_bounds__(WAVES * 64) void prod8_rows_kernel(const Prod8Args args) {
  const ProdArgs& a = args.p;
  constexpr int BN = 16 * NB, U = NB == 1 && MB == 1 ? 2 : 1;
  constexpr int V = 16, BK = 128, RED_LD = BN + 4;
  constexpr int XS = 16 * MB, WS = COLS ? BN : 1, ROOM = 4096;   // rows of scales; their room
  __shared__ __attribute__((aligned(128))) float red[WAVES * MB * 16 * RED_LD];
  __shared__ float scales[ROOM];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
  const int col0 = map_range(blockIdx.x, gridDim.x) * BN;
  int k_lo = 0, k_hi = a.K;
  if (a.splits > 1) {
    k_lo = blockIdx.y * a.k_split;
    k_hi = k_lo + a.k_split < a.K ? k_lo + a.k_split : a.K;
  }
  const int units = (k_hi - k_lo + BK - 1) / BK, whole = (k_hi - k_lo) / BK, b_lo = k_lo / BK;
  const int pitch = units | 1;                   // (odd: a column's 16 rows lie in 16 banks)
  const bool staged = (long long)pitch * (XS + WS) <= ROOM;
  // rows and columns outside read the last one (their results are never stored)
  const uint8_t* wrow[NB];
#pragma unroll
  for (int c = 0; c < NB; ++c) {
    const int n = col0 + 16 * c + i;
    wrow[c] = static_cast<const uint8_t*>(a.B) + (long long)(n < a.N ? n : a.N - 1) * a.ldb;
  }
  auto w_scale = [&](int n, int unit) {
    return args.sw[((n < a.N ? n : a.N - 1) >> args.w_shift) * args.sw_row +
                   (b_lo + unit) * args.sw_block];
  };

  auto x_scale = [&](int r, int unit) {
    return args.sx[(r < a.M ? r : a.M - 1) * args.sx_row + (b_lo + unit) * args.sx_block];
  };
  const uint8_t* arow[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    const int m = 16 * b + i < a.M ? 16 * b + i : a.M - 1;
    arow[b] = static_cast<const uint8_t*>(a.A) + m * a.lda;
  }
  f32x4 acc[MB][NB];
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int c = 0; c < NB; ++c) acc[b][c] = f32x4{0, 0, 0, 0};

  struct Unit {
    u32x4 w[NB][2], x[MB][2];
  };
  auto use = [&](const Unit& u, int unit) {
    float sx[MB], sw[WS == 1 ? 1 : NB][COLS ? 4 : 1];
#pragma unroll
    for (int b = 0; b < MB; ++b)
      sx[b] = staged ? scales[(16 * b + i) * pitch + unit] : x_scale(16 * b + i, unit);
#pragma unroll
    for (int c = 0; c < (COLS ? NB : 1); ++c)
#pragma unroll
      for (int j = 0; j < (COLS ? 4 : 1); ++j) {
        const int n = COLS ? 16 * c + 4 * g + j : 0;
        sw[c][j] = staged ? scales[(XS + n) * pitch + unit] : w_scale(col0 + n, unit);
      }
    Part<WIDE> x[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) x[b] = part<WIDE, FA>(u.x[b][0], u.x[b][1]);
#pragma unroll
    for (int c = 0; c < NB; ++c) {
      const Part<WIDE> w = part<WIDE, FB>(u.w[c][0], u.w[c][1]);
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        const f32x4 t = block_sum<WIDE, FB, FA>(w, x[b]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[b][c][j] += t[j] * (sx[b] * sw[COLS ? c : 0][COLS ? j : 0]);
      }
    }
  };
  constexpr int STEP = U * WAVES;
  Unit xs[U], ys[U];
  auto load = [&](int u0, Unit(&us)[U]) {
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int unit = u0 + q * WAVES;
      if (unit >= whole) break;
      const int k0 = k_lo + unit * BK;
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
        for (int c = 0; c < NB; ++c) us[q].w[c][kk] = load16(wrow[c] + k0 + (4 * kk + g) * V);
#pragma unroll
        for (int b = 0; b < MB; ++b) us[q].x[b][kk] = load16(arow[b] + k0 + (4 * kk + g) * V);
      }
    }
  };
  auto use_all = [&](int u0, Unit(&us)[U]) {
#pragma unroll
    for (int q = 0; q < U; ++q) {
      if (u0 + q * WAVES >= whole) break;
      use(us[q], u0 + q * WAVES);
    }
  };
  load(wave, xs);
  if (staged) {
    for (int t = threadIdx.x; t < (XS + WS) * units; t += WAVES * 64) {
      const int r = t / units, unit = t - r * units;
      scales[r * pitch + unit] = r < XS ? x_scale(r, unit) : w_scale(col0 + r - XS, unit);
    }
    __syncthreads();
  }
#pragma unroll 1
  for (int u0 = wave; u0 < whole; u0 += 2 * STEP) {
    load(u0 + STEP, ys);
    use_all(u0, xs);
    load(u0 + 2 * STEP, xs);
    use_all(u0 + STEP, ys);
  }
  if (whole < units && whole % WAVES == wave) {     // the last, partly filled block
    Unit u;
    const int k0 = k_lo + whole * BK;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
      for (int c = 0; c < NB; ++c) u.w[c][kk] = load_guarded(wrow[c], k0 + (4 * kk + g) * V, k_hi);
#pragma unroll
      for (int b = 0; b < MB; ++b) u.x[b][kk] = load_guarded(arow[b], k0 + (4 * kk + g) * V, k_hi);
    }
    use(u, whole);
  }

  // sum over the waves, then 8 columns per thread
  __syncthreads();
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int c = 0; c < NB; ++c)
      *reinterpret_cast<f32x4*>(red + ((wave * MB + b) * 16 + i) * RED_LD + 16 * c + 4 * g) =
          acc[b][c];
  __syncthreads();
  for (int t = threadIdx.x; t < MB * 16 * (BN / 8); t += WAVES * 64) {
    const int m = t / (BN / 8), n = col0 + (t % (BN / 8)) * 8;
    if (m < a.M && n < a.N) {
      float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        const float* from = red + (w * MB * 16 + m) * RED_LD + (t % (BN / 8)) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += from[j];
      }
      finish8_any<WIDE>(args, m, n, v, blockIdx.y);
    }
  }
}

// Sums the splits in order and runs the epilogue: 8 columns per thread.  (FA
// and WIDE: a kernel of its own for each source file.)
template <int FA, bool WIDE>
__global__ __launch_bounds__(256) void prod8_reduce_kernel(const Prod8Args args) {
  const ProdArgs& a = args.p;
  const int per_row = (a.N + 7) / 8;
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
  if (id >= (long long)a.M * per_row) return;
  const long long m = id / per_row;
  const int n = (int)(id % per_row) * 8;
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s) {
    float x[8];
    get_row8<float>(a.partial, (s * (long long)a.M + m) * a.N, n, a.N, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += x[j];
  }
  Prod8Args whole = args;
  whole.p.splits = 1;
  finish8_any<WIDE>(whole, m, n, v, 0);
}

}  // namespace blocks
}  // namespace pgemm
