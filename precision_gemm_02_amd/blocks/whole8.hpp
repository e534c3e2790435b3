// The 8-bit products' tile kernel for operands in whole 16-byte chunks (aligned rows) and
// 16-bit results: prod8_tile_kernel with its loads through buffer descriptors, as
// pair_whole_kernel has them.
//
// 8192 x 8192 x 4096 over the same operands again and again 252 to 262 us (2.1 PFLOP/s; others in
// turn, with an epilogue 272 to 287 by the card), 313 with a scale for each column of W; of
// zeros, which need little power, 227.  LDS, the vector units and the matrix cores share a tile's
// time: with a quarter of A's LDS reads 218 us, with a quarter of the multiply-adds 244.  A
// wave's tile of 128 x 64 reads 24 KB for its 32 matrix instructions, and a larger one does
// not fit the registers, since the sums that the vector units add to cannot lie in the
// accumulation registers.  Tried and level or slower: A's blocks read two ahead, half of W's
// next tile read early, one barrier a tile, an order for each instruction.
#pragma once

#include "fp8.hpp"
#include "whole.hpp"

namespace pgemm {
namespace blocks {

// 4 bytes per lane straight to LDS (see tile_load).
__device__ __forceinline__ void tile_load4(u32x4 from, uint32_t offset, uint32_t to) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dword %1, %2, 0 offen lds"
      :
      : "s"(to), "v"(offset), "s"(from));
}

template <int FA, int FB, int BM, int BN, int WGM, int WGN, bool COLS, bool TAIL>
__global__ __launch_bounds__(WGM* WGN * 64) void prod8_whole_kernel(const Prod8Args args) {
  const ProdArgs& a = args.p;
  constexpr int NT = WGM * WGN * 64;
  constexpr int WM = BM / WGM, WN = BN / WGN, RB = WM / 16, CB = WN / 16;
  constexpr int BK = 128;
  constexpr int SLOT_A = BM * BK, SLOT_B = BN * BK, SCALES = (BM + BN) * 4;
  constexpr int AT_B = 2 * SLOT_A, AT_S = AT_B + 2 * SLOT_B;
  static_assert(BM % 64 == 0 && BM + BN <= NT, "a wave's scales are of one operand");
  __shared__ __attribute__((aligned(128))) char lds[AT_S + 2 * SCALES];

  const int lane = threadIdx.x & 63, i16 = lane & 15, g4 = lane >> 4;
  (void)g4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = (wave / WGN) * WM, wn = (wave % WGN) * WN;
  int tm, tn, k_lo = 0, k_hi = a.K;
  map_tile(blockIdx.x, a.tiles_m, a.tiles_n, &tm, &tn);
  if (a.splits > 1) {
    k_lo = blockIdx.y * a.k_split;
    k_hi = k_lo + a.k_split < a.K ? k_lo + a.k_split : a.K;
  }
  const int row0 = tm * BM, col0 = tn * BN, nk = (k_hi - k_lo + BK - 1) / BK;

  using TA = OperandTile<uint8_t, kInner, BM, NT>;
  using TB = OperandTile<uint8_t, kInner, BN, NT>;
  constexpr int NA = TA::LOADS, NB = TB::LOADS;
  // a lane's offsets from its operand's tile; rows outside read the last one
  uint32_t va[NA], vb[NB], vs;
  // TAIL: summed indices of a partly filled last tile (0: it is whole); this lane's chunk (the same
  // of every row) is outside them
  const int tail = TAIL ? a.K % BK : 0;
  uint32_t out = 0;
#pragma unroll
  for (int j = 0; j < NA; ++j) {
    int r, c;
    TA::slot(j * NT + (int)threadIdx.x, &r, &c);
    out = c * 16 >= tail ? kOutside : 0;
    va[j] = (uint32_t)(row0 + r < a.M ? r : a.M - 1 - row0) * (uint32_t)a.lda + c * 16;
  }
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    int r, c;
    TB::slot(j * NT + (int)threadIdx.x, &r, &c);
    vb[j] = (uint32_t)(col0 + r < a.N ? r : a.N - 1 - col0) * (uint32_t)a.ldb + c * 16;
  }
  Walk wa, wb, ws;
  wa.at = static_cast<const char*>(a.A) + (long long)row0 * a.lda + k_lo;
  wb.at = static_cast<const char*>(a.B) + (long long)col0 * a.ldb + k_lo;
  wa.step = wb.step = BK;
  wa.left = wb.left = ws.left = nk;
  if (wave * 64 < BM) {
    const int r = threadIdx.x;
    vs = (uint32_t)(row0 + r < a.M ? r : a.M - 1 - row0) * (uint32_t)(args.sx_row * 4);
    ws.at = reinterpret_cast<const char*>(args.sx + row0 * args.sx_row + k_lo / BK * args.sx_block);
    ws.step = args.sx_block * 4;
  } else {
    const int c = col0 + (int)threadIdx.x - BM, first = col0 >> args.w_shift;
    vs = (uint32_t)(((c < a.N ? c : a.N - 1) >> args.w_shift) - first) * (uint32_t)(args.sw_row * 4);
    ws.at = reinterpret_cast<const char*>(args.sw + first * args.sw_row + k_lo / BK * args.sw_block);
    ws.step = args.sw_block * 4;
  }
  const uint32_t lds_wave = lds_address(lds) + wave * 1024;

  // A and the scales of the next tile, into place `to`
  auto load_a = [&](int to) {
    const u32x4 d = descriptor(wa.at);
    const uint32_t cut = TAIL && tail > 0 && k_hi == a.K && wa.left <= 1 ? kOutside : 0;
#pragma unroll
    for (int j = 0; j < NA; ++j)
      tile_load(d, va[j] | (cut & out), lds_wave + to * SLOT_A + j * NT * 16);
    if (BM + BN == NT || wave * 64 < BM + BN)
      tile_load4(descriptor(ws.at), vs, lds_address(lds) + AT_S + to * SCALES + wave * 256);
    wa.next(0);
    ws.next(0);
  };
  auto load_b = [&](auto j0, auto j1, int to) {
    const u32x4 d = descriptor(wb.at);
    const uint32_t cut = TAIL && tail > 0 && k_hi == a.K && wb.left <= 1 ? kOutside : 0;
#pragma unroll
    for (int j = decltype(j0)::value; j < decltype(j1)::value; ++j)
      tile_load(d, vb[j] | (cut & out), lds_wave + AT_B + to * SLOT_B + j * NT * 16);
    if constexpr (decltype(j1)::value == NB) wb.next(0);
  };

  // Of the two waves of a SIMD one goes first, so that one's matrix instructions run under the
  // other's multiply-adds: 8192 x 8192 x 4096 262 us, 277 with both alike.
  if (wave & 4) __builtin_amdgcn_s_setprio(1);
  f32x4 acc[RB][CB];
#pragma unroll
  for (int r = 0; r < RB; ++r)
#pragma unroll
    for (int c = 0; c < CB; ++c) acc[r][c] = f32x4{0, 0, 0, 0};

  if (nk > 0) {
    constexpr std::integral_constant<int, 0> zero{};
    constexpr std::integral_constant<int, NB> all_b{};
    load_a(0);
    load_b(zero, all_b, 0);
    load_b(zero, all_b, 1);
    load_a(1);
    wait_loads<NA + NB>();          // all but the second tile (a wave may have no scales)
    workgroup_barrier();

    u32x4 fa[2][2], fb[CB][2];
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
    auto add = [&](int r, int c, float p) {     // block (r, c)'s sums times their scale
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (COLS) acc[r][c][j] += sum[c][j] * (p * pw[c][j]);
        else acc[r][c][j] += sum[c][j] * p;
      }
    };
    read_a(lds, 0);
#pragma unroll
    for (int c = 0; c < CB; ++c) {
      read_b(lds + AT_B, c);
      sum[c] = f32x4{0, 0, 0, 0};
    }
    auto tile = [&](auto place) {
      constexpr int at = decltype(place)::value;
      const char *const a0 = lds + at * SLOT_A, *const a1 = lds + (at ^ 1) * SLOT_A;
      const char* const b1 = lds + AT_B + (at ^ 1) * SLOT_B;
      const float* const sc = reinterpret_cast<const float*>(lds + AT_S + at * SCALES);
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
      static_for<RB>([&](auto gc) {
        constexpr int g = decltype(gc)::value;
        constexpr int AT = RB > 4 ? 3 : 1;      // (the waves may drift apart by half a tile)
        constexpr bool M = g == AT, E = g == RB - 1;
        if constexpr (E) {
          wait_loads<M ? 0 : NB>();             // the next tile (in two blocks: no other)
          workgroup_barrier();
          read_a(a1, 0);                        // past the last tile: some LDS, never used
        } else {
          if constexpr (M) workgroup_barrier();
          read_a(a0, g + 1);
        }
        constexpr int PARTS = RB > 2 ? RB - 1 - AT : 1;
        constexpr bool ask = g >= AT && (g < RB - 1 || RB == 2);
        constexpr int from = ask ? NB * (g - AT) / PARTS : 0, to = ask ? NB * (g - AT + 1) / PARTS : 0;
        if constexpr (from < to)
          load_b(std::integral_constant<int, from>{}, std::integral_constant<int, to>{}, at);
        if constexpr (E) load_a(at);
#pragma unroll
        for (int c = 0; c < CB; ++c) {
          // the block before (in the first: the last of the tile before; with a scale for
          // each column, the registers that would hold both tiles' are not there)
          if constexpr (g > 0) add(g - 1, c, px[g - 1]);
          else if constexpr (!COLS) add(RB - 1, c, last);
          sum[c] = block_sum<false, FB, FA>({{fb[c][0], fb[c][1]}}, {{fa[g & 1][0], fa[g & 1][1]}});
          if constexpr (E) read_b(b1, c);
        }
        __builtin_amdgcn_sched_barrier(0);
      });
      last = px[RB - 1];
      if constexpr (COLS) {
#pragma unroll
        for (int c = 0; c < CB; ++c) add(RB - 1, c, last);
      }
    };
#pragma unroll 1
    for (int t = 0; t < nk; t += 2) {
      tile(zero);
      if (t + 1 < nk) tile(std::integral_constant<int, 1>{});
    }
    if constexpr (!COLS) {
#pragma unroll
      for (int c = 0; c < CB; ++c) add(RB - 1, c, last);
    }
    wait_loads<0>();                            // the loads past the end
  }

  // Epilogue: 8 consecutive columns per lane, of two blocks beside each other
  const int n0 = col0 + wn + 16 * (lane >> 4 & 1) + 8 * (lane >> 5);
#pragma unroll 1
  for (int r = 0; r < RB; ++r) {
    const int m = row0 + wm + 16 * r + i16;
    f32x4 row[CB];
    take<RB, CB>(acc, r, row);
#pragma unroll
    for (int c = 0; c < CB; c += 2) {
      float v[8];
      join(row[c], row[c + 1], v);
      if (m < a.M && n0 + 16 * c < a.N) finish8_any<false>(args, m, n0 + 16 * c, v, blockIdx.y);
    }
  }
}

}  // namespace blocks
}  // namespace pgemm
