// The pair products' tile kernel for operands in whole 16-byte chunks (aligned rows).
// Beside pair_tile_kernel it spends no vector instruction on the loads' addresses: an
// operand's tile is a buffer descriptor whose scalar base moves along the summed index,
// and each lane's 32-bit offsets within a tile stay as they are.  In a last, partly
// filled tile of the summed index, lanes outside take an offset behind the descriptor's
// end, for which the load writes zeros to LDS.
//
// A tile of the summed index is 128 bytes of each row.  Of the LDS, three slots hold A's
// tiles, two B's.  A wave's B operands of a whole tile stay in registers (CB x 8), read
// at the end of the tile before, so that B's slot is free for the tile after next as
// soon as every wave has passed barrier M behind its first block; A's blocks of 16
// rows are read one ahead of their use, and its slot is free behind barrier E, before
// the last block, which also waits for the next tile: both operands are loaded about
// two tiles ahead.  A tile's code is repeated for the six places that the slots take
// in turn, so that every LDS address is a constant.
//
// Bound by the matrix cores at the power-limited clock: 8192 x 8192 x 4096 bf16 with both Z
// 800 to 824 us by the card (1.33 to 1.37 PFLOP/s), where a library product of 8192 x 16384 x
// 4096 without an epilogue takes 719; of 8192 x 4096 x 4096 dX 381 and both dW 381 (1.44).  With 16384 summed indices the loops are
// level; what is left is each tile's prologue and epilogue.  Tried and slower: four waves of
// 128 x 128 (843 us against 797 then), one barrier a tile, B's reads earlier.
#pragma once

#include "gated.hpp"

namespace pgemm {
namespace blocks {

// A descriptor of 2^31 bytes from `base` on.  Offsets below are in bounds of the operand by
// construction; kOutside is behind it.
constexpr uint32_t kOutside = 0x80000000u;
__device__ __forceinline__ u32x4 descriptor(const char* base) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return u32x4{(uint32_t)a, (uint32_t)(a >> 32) & 0xffffu, kOutside, 0x00020000u};
}

// 16 bytes per lane straight to LDS: lane l of the wave writes at to + 16 l (an LDS
// address, the same for all lanes).  As the instruction for load_to_lds's reasons.
__device__ __forceinline__ void tile_load(u32x4 from, uint32_t offset, uint32_t to) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, 0 offen lds"
      :
      : "s"(to), "v"(offset), "s"(from));
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)p;
}

// An operand's descriptor base and what moves it from tile to tile.  Past the last
// tile it stays (the loads repeat it; nothing uses them).
struct Walk {
  const char* at;
  long long step;
  int left;                // tiles from `at` on
  __device__ __forceinline__ void next(long long extra) {
    if (--left > 0) at += step + extra;
  }
};

// Two blocks of results (lane 16 g + i: row i, columns 4 g .. 4 g + 3) as 8 consecutive
// columns per lane: lane group g has columns 8 (g / 2) .. of block g % 2.
__device__ __forceinline__ void join(f32x4 x, f32x4 y, float* v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float xj = x[j], yj = y[j];           // (a bit_cast of x[j] itself takes element 0)
    const auto p = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, xj),
                                                    __builtin_bit_cast(uint32_t, yj), false, false);
    const uint32_t lo = p[0], hi = p[1];
    v[j] = __builtin_bit_cast(float, lo);
    v[4 + j] = __builtin_bit_cast(float, hi);
  }
}

// Row r of the blocks of results, by branches (r is the same for the wave).  The empty asm
// keeps the compiler from making one indexed copy of them, through memory.
template <int RB, int CB>
__device__ __forceinline__ void take(const f32x4 (&acc)[RB][CB], int r, f32x4 (&row)[CB]) {
  static_for<RB>([&](auto q) {
    if (r == decltype(q)::value) {
#pragma unroll
      for (int c = 0; c < CB; ++c) {
        f32x4 t = acc[decltype(q)::value][c];
        asm volatile("" : "+v"(t));
        row[c] = t;
      }
    }
  });
}

template <typename T, int LA, int LB, int BM, int BN, int WGM, int WGN, int PAIR, bool TAIL>
__global__ __launch_bounds__(WGM* WGN * 64) void pair_whole_kernel(const PairArgs args) {
  const ProdArgs& a = args.p;
  constexpr int S = sizeof(T), NT = WGM * WGN * 64;
  constexpr int WM = BM / WGM, WN = BN / WGN, RB = WM / 16, CB = WN / 16;
  constexpr int BK = 128 / S;
  constexpr int SLOT_A = BM * 128, SLOT_B = BN * 128;
  __shared__ __attribute__((aligned(128))) char lds[3 * SLOT_A + 2 * SLOT_B];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = (wave / WGN) * WM, wn = (wave % WGN) * WN;
  constexpr int COLS = PAIR == kColumns ? BN / 2 : BN;   // results of a tile
  int tm, tn, k_lo = 0, k_hi = a.K;
  map_tile(blockIdx.x, a.tiles_m, PAIR == kApart ? a.tiles_n * args.count : a.tiles_n, &tm, &tn);
  const bool other = PAIR == kApart && tn >= a.tiles_n;
  if (other) tn -= a.tiles_n;
  const int row0 = tm * BM, col0 = tn * COLS;
  if (a.splits > 1) {
    k_lo = blockIdx.y * a.k_split;
    k_hi = k_lo + a.k_split < a.K ? k_lo + a.k_split : a.K;
  }
  const int nk = (k_hi - k_lo + BK - 1) / BK;

  // kColumns: B's slot holds a tile of either weight, half as wide
  constexpr int SUBS = PAIR == kColumns ? 2 : 1, SUB = BN / SUBS, SUB_BYTES = SUB * 128;
  using TA = OperandTile<T, LA, BM, NT>;
  using TB = OperandTile<T, LB, SUB, NT>;
  constexpr int NA = TA::LOADS, NB = SUBS * TB::LOADS;
  // a lane's offsets from its operand's tile; rows and columns outside read the last row
  // or the first chunk (they reach results that are never stored)
  uint32_t va[NA], vb[TB::LOADS];
  // TAIL: summed indices of a partly filled last tile (0: it is whole), and the loads outside
  // them; kHalves: of B alone, in both halves (dZ's rows hold zeros there)
  const int tail = !TAIL ? 0 : (PAIR == kHalves ? args.inner : a.K) % BK;
  const bool ends = k_hi == a.K || (PAIR == kHalves && k_hi == args.half);
  uint32_t out_a = 0, out_b = 0;   // bit 31 - j: a lane's load j is outside (inner: all alike)
#pragma unroll
  for (int j = 0; j < NA; ++j) {
    int r, c;
    TA::slot(j * NT + (int)threadIdx.x, &r, &c);
    if (PAIR != kHalves && (LA == kInner ? c * TA::V : r) >= tail) out_a |= kOutside >> j;
    if constexpr (LA == kInner) {
      const int row = row0 + r < a.M ? r : a.M - 1 - row0;
      va[j] = (uint32_t)row * (uint32_t)(a.lda * S) + c * 16;
    } else {
      va[j] = (uint32_t)r * (uint32_t)(a.lda * S) + (row0 + c * TA::V < a.M ? c * 16 : 0);
    }
  }
#pragma unroll
  for (int j = 0; j < TB::LOADS; ++j) {
    int r, c;
    TB::slot(j * NT + (int)threadIdx.x, &r, &c);
    if ((LB == kInner ? c * TB::V : r) >= tail) out_b |= kOutside >> j;
    if constexpr (LB == kInner) {
      const int col = col0 + r < a.N ? r : a.N - 1 - col0;
      vb[j] = (uint32_t)col * (uint32_t)(a.ldb * S) + c * 16;
    } else {
      vb[j] = (uint32_t)r * (uint32_t)(a.ldb * S) + (col0 + c * TB::V < a.N ? c * 16 : 0);
    }
  }
  // element (output index, summed index) of an operand
  auto place = [](const void* base, int order, long long ld, long long out, long long in) {
    return static_cast<const char*>(base) + (order == kInner ? out * ld + in : in * ld + out) * S;
  };
  Walk wa, wb;
  wa.at = place(other ? args.A2 : a.A, LA, a.lda, row0, k_lo);
  wa.step = LA == kInner ? 128 : BK * a.lda * S;
  wb.step = LB == kInner ? 128 : BK * a.ldb * S;
  wa.left = wb.left = nk;
  const long long second = static_cast<const char*>(args.B2) - static_cast<const char*>(a.B);
  long long jump = 0;
  int before = -1;                 // kHalves: B's tiles left when the second weight begins
  if constexpr (PAIR == kHalves) {
    const bool on = k_lo >= args.half;
    wb.at = place(on ? args.B2 : a.B, LB, a.ldb, col0, on ? k_lo - args.half : k_lo);
    jump = second - (LB == kInner ? args.half : args.half * a.ldb) * S;
    before = (k_hi - args.half) / BK;
  } else {
    wb.at = place(other ? args.B2 : a.B, LB, a.ldb, col0, k_lo);
  }
  const uint32_t lds_wave = lds_address(lds) + wave * 1024;

  // loads J0 .. J1-1 of the next tile, into slot `to`
  auto load_a = [&](auto j0, auto j1, int to) {
    const u32x4 d = descriptor(wa.at);
    const uint32_t cut = TAIL && tail > 0 && ends && wa.left <= 1 ? kOutside : 0;
#pragma unroll
    for (int j = decltype(j0)::value; j < decltype(j1)::value; ++j)
      tile_load(d, PAIR == kHalves ? va[j] : va[j] | ((LA == kInner ? out_a : out_a << j) & cut),
                lds_wave + to * SLOT_A + j * NT * 16);
    if constexpr (decltype(j1)::value == NA) wa.next(0);
  };
  auto load_b = [&](auto j0, auto j1, int to) {
    const u32x4 d = descriptor(wb.at);
    const u32x4 e = PAIR == kColumns ? descriptor(wb.at + second) : d;
    const uint32_t cut =
        TAIL && tail > 0 && (wb.left <= 1 ? ends : wb.left - 1 == before) ? kOutside : 0;
#pragma unroll
    for (int j = decltype(j0)::value; j < decltype(j1)::value; ++j)
      tile_load(j < TB::LOADS ? d : e,
                vb[j % TB::LOADS] | ((LB == kInner ? out_b : out_b << j % TB::LOADS) & cut),
                lds_wave + 3 * SLOT_A + to * SLOT_B + j * NT * 16);
    if constexpr (decltype(j1)::value == NB)
      wb.next(PAIR == kHalves && wb.left - 1 == before ? jump : 0);
  };

  f32x4 acc[RB][CB];
#pragma unroll
  for (int r = 0; r < RB; ++r)
#pragma unroll
    for (int c = 0; c < CB; ++c) acc[r][c] = f32x4{0, 0, 0, 0};

  if (nk > 0) {
    constexpr std::integral_constant<int, 0> zero{};
    constexpr std::integral_constant<int, NA> all_a{};
    constexpr std::integral_constant<int, NB> all_b{};
    load_a(zero, all_a, 0);
    load_b(zero, all_b, 0);
    load_a(zero, all_a, 1);
    load_b(zero, all_b, 1);
    load_a(zero, all_a, 2);
    wait_loads<2 * NA + NB>();
    workgroup_barrier();

    // B's first halves of two tiles in turn: those of the next are read under the last
    // block; its second halves follow as this tile's come free
    u32x4 fa[2][2], fb0[2][CB], fb1[CB];
    auto read_a = [&](const char* from, int g) {
      fa[g & 1][0] = TA::frag(from, wm, g, 0);
      fa[g & 1][1] = TA::frag(from, wm, g, 1);
    };
    auto read_b = [&](const char* from, int c, int half) {
      if constexpr (PAIR == kColumns)
        return TB::frag(from + (c >= CB / 2 ? SUB_BYTES : 0), wn / 2, c % (CB / 2), half);
      else
        return TB::frag(from, wn, c, half);
    };
    read_a(lds, 0);
#pragma unroll
    for (int c = 0; c < CB; ++c) {
      fb0[0][c] = read_b(lds + 3 * SLOT_A, c, 0);
      fb1[c] = read_b(lds + 3 * SLOT_A, c, 1);
    }
    auto tile = [&](auto place_) {
      constexpr int sa = decltype(place_)::value % 3, sb = decltype(place_)::value % 2;
      const char* const a0 = lds + sa * SLOT_A;
      const char* const a1 = lds + (sa + 1) % 3 * SLOT_A;
      const char* const b1 = lds + 3 * SLOT_A + (sb ^ 1) * SLOT_B;
      static_for<RB>([&](auto gc) {
        constexpr int g = decltype(gc)::value;
        constexpr bool M = g == 1, E = g == RB - 1;
        if constexpr (E) {
          // all but the tile after next (of which, in two blocks, B's is not yet asked for)
          wait_loads<M ? NA : NA + NB>();
          workgroup_barrier();
          read_a(a1, 0);                        // past the last tile: some LDS, never used
#pragma unroll
          for (int c = 0; c < CB; ++c) fb0[sb ^ 1][c] = read_b(b1, c, 0);
        } else {
          if constexpr (M) workgroup_barrier();
          read_a(a0, g + 1);
        }
        // B's loads over the blocks behind M, A's in the last one
        constexpr int PARTS = RB > 2 ? RB - 2 : 1;
        constexpr bool ask = g >= 1 && (g < RB - 1 || RB == 2);
        constexpr int from = ask ? NB * (g - 1) / PARTS : 0, to = ask ? NB * g / PARTS : 0;
        if constexpr (from < to)
          load_b(std::integral_constant<int, from>{}, std::integral_constant<int, to>{}, sb);
        if constexpr (E) load_a(zero, all_a, sa);
#pragma unroll
        for (int c = 0; c < CB; ++c) acc[g][c] = Elem<T>::mfma(fb0[sb][c], fa[g & 1][0], acc[g][c]);
#pragma unroll
        for (int c = 0; c < CB; ++c) {
          acc[g][c] = Elem<T>::mfma(fb1[c], fa[g & 1][1], acc[g][c]);
          if constexpr (E) fb1[c] = read_b(b1, c, 1);
        }
        spread<2 * TA::READS + (E ? 2 * CB * TB::READS : 0), 2 * CB * Elem<T>::kMfmas, 0>();
        __builtin_amdgcn_sched_barrier(0);
      });
    };
#pragma unroll 1
    for (int t = 0; t < nk; t += 6)
      static_for<6>([&](auto i) {
        if (t + decltype(i)::value < nk) tile(i);
      });
    wait_loads<0>();                            // the loads past the end
  }
  // Epilogue: 8 consecutive columns per lane, of two blocks beside each other, or (where a
  // wave has one block of a weight) below each other.
  constexpr int WC = PAIR == kColumns ? WN / 2 : WN, WCB = WC / 16;   // results of a wave's row
  constexpr bool BELOW = WCB == 1;
  const int which = lane >> 4 & 1;
  const int n0 = col0 + wn / WN * WC + (BELOW ? 0 : 16 * which) + 8 * (lane >> 5);
  float bg[WCB / 2 + 1][8], bu[WCB / 2 + 1][8];
  if constexpr (PAIR == kColumns) {
#pragma unroll
    for (int c = 0; c < WCB; c += 2)
      if (a.splits <= 1) gate_bias<T>(args, n0 + 16 * c, bg[c / 2], bu[c / 2]);
  }
#pragma unroll 1
  for (int r = 0; r < RB; r += BELOW ? 2 : 1) {
    const int m = row0 + wm + 16 * (BELOW ? r + which : r) + (lane & 15);
    f32x4 row[CB], below[CB];
    take<RB, CB>(acc, r, row);
    if constexpr (BELOW) take<RB, CB>(acc, r + 1, below);
#pragma unroll
    for (int c = 0; c < WCB; c += 2) {
      const int n = n0 + 16 * c;
      float v[8], u[8];
      join(row[c], BELOW ? below[c] : row[c + 1 - BELOW], v);
      if constexpr (PAIR == kColumns)
        join(row[WCB + c], BELOW ? below[WCB + c] : row[WCB + c + 1 - BELOW], u);
      if (m >= a.M || n >= a.N) continue;
      if constexpr (PAIR == kColumns) {
        if (a.splits > 1) {
          put_partial(a, blockIdx.y, 0, m, n, v);
          put_partial(a, blockIdx.y, 1, m, n, u);
        } else {
          finish_gate<T>(args, m, n, v, u, bg[c / 2], bu[c / 2]);
        }
      } else if (a.splits > 1) {
        const long long matrix = PAIR == kApart ? (long long)blockIdx.y * args.count + other
                                                : blockIdx.y;
        put_row8<float>(a.partial, (matrix * a.M + m) * a.N, n, a.N, v);
      } else {
        void* D = other ? args.D2 : a.D;
        if (a.out32) put_row8<float>(D, m * a.ldd, n, a.N, v);
        else put_row8<T>(D, m * a.ldd, n, a.N, v);
      }
    }
  }
}

}  // namespace blocks
}  // namespace pgemm
