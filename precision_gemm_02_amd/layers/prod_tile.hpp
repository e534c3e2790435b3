// The tile kernel: one BM x BN tile of D per workgroup, WGM x WGN waves,
// matrix cores fed from LDS.  See prod.hpp for the operands' orders and the
// groups.
//
// Large products are bound by the matrix cores at the power-limited clock:
// 8192 x 8192 x 4096 bf16 with activation and Z 455 us (1.21 PFLOP/s; a plain
// library product of that shape 420 to 440), 4096^3 114 to 118 us, fp32 4096^3
// 966 us (142 TFLOP/s).  256 x 256 tiles (8 waves of 128 x 64, all of a compute
// unit's LDS) halve the LDS and cache traffic per flop of 128 x 128 ones (two
// workgroups per unit), which win where 256 x 256 would leave units idle; 64 x
// 64 (four per unit) for small products.  4 waves of 128 x 128 measured 6 to 9
// % slower than 8.
#pragma once

#include <type_traits>

#include "prod.hpp"

namespace pgemm {
namespace layers {

// 16 zero bytes: what a lane loads for a chunk outside its operand.
static __device__ const u32x4 kZeroChunk = {0, 0, 0, 0};

// One operand's tile: `EXT` output indices by 128 bytes' worth of the summed
// index (BK = 64 16-bit or 32 fp32 elements), in 16-byte chunks, read in
// fragments of 16 output indices by 64 bytes (two steps per tile).
//
// Inner order: LDS row r holds output index r, 8 chunks along the summed
// index; chunk c sits at c ^ (r & 7).  A b128 read serves the 8-lane blocks b
// and b ^ 3 together; of these one reads chunk c and the other c ^ 1, so their
// flipped positions never meet.
//
// Outer order: LDS row p holds summed index p, EXT contiguous output indices.
// 16-bit operands are read through the transposing ds_read_b64_tr_b16 (16
// lanes read a 4 x 16 block by rows and receive it by columns), fp32 with one
// b32 per inner index.  The 32-byte (16-bit) or 64-byte (fp32) pieces that
// 16 columns take from a row are flipped by the row so that the pieces read
// together fall into different banks.
template <typename T, int ORDER, int EXT, int NT>
struct OperandTile {
  static constexpr int S = sizeof(T);
  static constexpr int V = 16 / S;              // elements per chunk
  static constexpr int BK = 128 / S;
  static constexpr int BYTES = EXT * 128;
  static constexpr int ROW_CHUNKS = ORDER == kInner ? 8 : EXT / V;
  static constexpr int ROW_BYTES = ROW_CHUNKS * 16;
  static constexpr int LOADS = BYTES / (16 * NT);
  static constexpr int READS = ORDER == kInner ? 1 : S;   // LDS reads per fragment
  static_assert(BYTES % (16 * NT) == 0, "whole chunks per thread");
  // outer order: pieces of 16 output indices per row
  static constexpr int PIECE = 16 * S;          // bytes
  static constexpr int PIECES = EXT / 16;

  // The flip of row p's pieces (outer order).
  static __device__ __forceinline__ int flip(int p) {
    constexpr int b = PIECES >= 8 ? 3 : PIECES == 4 ? 2 : PIECES == 2 ? 1 : 0;
    if constexpr (S == 2) {
      // a half wave reads one piece of 8 rows (p & 3, bit 3 of p)
      return ((p & 3) | (((p >> 3) & 1) << 2)) >> (3 - b);
    } else {
      // one piece of four rows 4 apart
      return (p >> 2) & (b >= 2 ? 3 : b);
    }
  }

  // Global chunk (row, chunk in row) that LDS slot s of the tile holds.
  static __device__ __forceinline__ void slot(int s, int* row, int* chunk) {
    const int r = s / ROW_CHUNKS, pos = s % ROW_CHUNKS;
    *row = r;
    if constexpr (ORDER == kInner) {
      *chunk = pos ^ (r & 7);
    } else {
      constexpr int CPP = PIECE / 16;           // chunks per piece: 2 or 4
      *chunk = ((pos / CPP) ^ flip(r)) * CPP + pos % CPP;
    }
  }

  // Fragment of 16-index block b (from index `first`), step s, from the tile at
  // lds.
  static __device__ __forceinline__ u32x4 frag(const char* lds, int first, int b, int s) {
    const int l = threadIdx.x & 63, g = l >> 4, i = l & 15;
    if constexpr (ORDER == kInner) {
      const int row = first + 16 * b + i, c = (4 * s + g) ^ (i & 7);
      return *reinterpret_cast<const u32x4*>(lds + row * 128 + c * 16);
    } else {
      u32x4 out;
      const int piece = first / 16 + b;
      if constexpr (S == 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int p = 32 * s + 8 * g + 4 * h + (i >> 2);
          const int f = flip(8 * g + (i >> 2));   // 32 s and 4 h do not enter
          const char* at = lds + p * ROW_BYTES + (piece ^ f) * PIECE + (i & 3) * 8;
          const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (__attribute__((address_space(3))) s16x4*)(const_cast<char*>(at)));
          const u32x2 w = __builtin_bit_cast(u32x2, v);
          out[2 * h] = w[0];
          out[2 * h + 1] = w[1];
        }
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int p = 16 * s + 4 * g + q;
          const char* at = lds + p * ROW_BYTES + (piece ^ flip(4 * g)) * PIECE + i * 4;
          out[q] = *reinterpret_cast<const uint32_t*>(at);
        }
      }
      return out;
    }
  }
};

// Where a workgroup's tile reads an operand from.  Inner order: `outer` rows
// (output indices) of `inner` summed elements.  Outer order: `outer` summed
// indices of `inner` output elements.  Row r starts at base + r * ld, or
// base + gather[r] * ld.
template <typename T>
struct Source {
  const T* base;
  long long ld;
  int outer, inner;
  const int* gather;
  int gather_rows;

  // The gathered row of r: one outside the source reads the nearest inside.
  __device__ __forceinline__ int token(int r) const {
    const int t = gather[r];
    return t < 0 ? 0 : (t < gather_rows ? t : gather_rows - 1);
  }
  // Behind the last element of the last row.
  __device__ __forceinline__ const T* end() const {
    return base + (long long)((gather != nullptr ? gather_rows : outer) - 1) * ld + inner;
  }
  __device__ __forceinline__ const T* row(int r) const {
    if (r >= outer) return nullptr;
    return base + (long long)(gather != nullptr ? token(r) : r) * ld;
  }
};

// A chunk of V elements at row + c0, zeros past `inner`.
template <typename T>
__device__ __forceinline__ u32x4 load_guarded(const T* row, int c0, int inner) {
  constexpr int V = 16 / (int)sizeof(T);
  if (row == nullptr || c0 >= inner) return u32x4{0, 0, 0, 0};
  if (c0 + V <= inner) return load16(row + c0);
  typedef T tv __attribute__((ext_vector_type(V)));
  tv v;
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = c0 + j < inner ? row[c0 + j] : (T)0.0f;
  return __builtin_bit_cast(u32x4, v);
}

// A chunk at p, outer order, of which `live` elements exist in its row: what
// follows them only reaches results that are never stored, so the whole chunk
// is read wherever it ends before the operand's end.
template <typename T>
__device__ __forceinline__ u32x4 load_edge(const T* p, int live, const T* end) {
  constexpr int V = 16 / (int)sizeof(T);
  if (live <= 0) return u32x4{0, 0, 0, 0};
  if (p + V <= end) return load16(p);
  return load_guarded(p, 0, live);
}

// 16 bytes per lane from its own address straight to LDS: lane l of the wave
// writes at to + 16 l (`to` is the same for all lanes).  Written as the
// instruction, without a memory clobber: behind the builtin the compiler waits
// for all loads before every transposing LDS read (it cannot tell their slots
// apart), which cost outer-order operands the whole overlap.  The order that
// matters is kept by hand: wait_loads and workgroup_barrier are volatile, like
// this, and clobber memory; between two barriers no slot is both loaded and
// read (see the K loop).  There is no register output, and the address
// registers are read at issue.  m0 is reserved, so the compiler does not name it
// as a clobber; these kernels use it for nothing else.
__device__ __forceinline__ void load_to_lds(const void* from, char* to) {
  const int at = __builtin_amdgcn_readfirstlane(
      (int)(uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)to);
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, off"
      :
      : "s"(at), "v"(from));
}

// At most N of this wave's global loads are outstanding.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64, "the counter's range");
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// One operand's loads, tile after tile of the summed index.
//
// DIRECT: straight into LDS (global_load_lds_dwordx4: a wave writes 64
// consecutive chunks, so the layout's flips are applied to the global
// addresses).  It needs rows at 16-byte boundaries and no chunk that straddles
// the operand's end.  Each thread keeps one address per chunk and moves it by
// a constant step.  Output indices outside the operand read its last row or
// first chunk instead: they reach only results that are never stored.  The
// last, partly filled tile of the summed index takes zeros there.
// RAGGED: the same for rows at 4-byte boundaries and any sizes.  A chunk that
// straddles the end of an outer-order row goes on into the next rows; the tiles
// near the end of the summed index go through registers with guards instead.
// (Not for gathered outer-order rows, whose next row may be outside.)
// THROUGH: through registers, with guards, for any alignment.
template <typename T, int ORDER, int EXT, int NT, int LOADING, bool GATHER>
struct Loader {
  static constexpr bool DIRECT = LOADING != kThrough;
  using Tile = OperandTile<T, ORDER, EXT, NT>;
  static constexpr int L = Tile::LOADS;
  static_assert(LOADING != kRagged || !GATHER, "see above");
  Source<T> src;
  int first;                       // first output index of the tile
  int k;                           // first summed index of the next load
  const T* ptr[L];                 // the next load's addresses
  int token[L];                    // its gathered rows (outer order, GATHER)
  long long step;                  // outer order: elements per tile
  u32x4 reg[DIRECT ? 1 : L];

  __device__ __forceinline__ void init(const Source<T>& s, int first_out, int k0) {
    src = s;
    first = first_out;
    k = k0;
#pragma unroll
    for (int j = 0; j < L; ++j) {
      int r, c;
      Tile::slot(j * NT + (int)threadIdx.x, &r, &c);
      if constexpr (ORDER == kInner) {
        const int row = first + r < src.outer ? first + r : src.outer - 1;
        ptr[j] = src.row(row) + k + c * Tile::V;
      } else {
        const int at = first + c * Tile::V;
        ptr[j] = src.base + (at < src.inner ? at : 0);
        if constexpr (!GATHER) ptr[j] += (long long)(k + r) * src.ld;
      }
    }
    step = (long long)Tile::BK * src.ld;
    if constexpr (ORDER == kOuter && GATHER) next_tokens();
  }

  __device__ __forceinline__ void next_tokens() {
#pragma unroll
    for (int j = 0; j < L; ++j) {
      int r, c;
      Tile::slot(j * NT + (int)threadIdx.x, &r, &c);
      token[j] = k + r >= src.outer ? 0 : src.gather != nullptr ? src.token(k + r) : k + r;
    }
  }

  // Whether a chunk of the next load (through registers) is outside the operand
  // or straddles its end.  The same for the whole workgroup.
  __device__ __forceinline__ bool ragged() const {
    if constexpr (ORDER == kInner) return k + Tile::BK > src.inner;
    return k + Tile::BK > src.outer || first + EXT > src.inner;
  }

  // Chunks J0 .. J1-1 of the load of summed indices k .. k+BK-1.  Direct loads
  // take no branch: a chunk past the end of the summed index (all of them
  // past the last tile) comes from the zero chunk.
  template <int J0, int J1>
  __device__ __forceinline__ void load(char* lds) {
    if constexpr (LOADING == kDirect) {
      load_as<false, J0, J1>(lds);
    } else if constexpr (LOADING == kRagged) {
      // near the end: V rows of margin for the chunks that go on into the next
      if (k + Tile::BK + Tile::V >= (ORDER == kInner ? src.inner : src.outer)) {
        load_guards<J0, J1>(lds);
      } else {
        load_as<true, J0, J1>(lds);
      }
    } else {
      if (ragged()) load_as<false, J0, J1>(lds);
      else load_as<true, J0, J1>(lds);
    }
    if constexpr (J1 == L) {
      k += Tile::BK;
      if constexpr (ORDER == kOuter && GATHER) next_tokens();
    }
  }

  template <bool WHOLE, int J0, int J1>
  __device__ __forceinline__ void load_as(char* lds) {
#pragma unroll
    for (int j = J0; j < J1; ++j) {
      int r, c;
      Tile::slot(j * NT + (int)threadIdx.x, &r, &c);
      const T* p = ptr[j];
      if constexpr (ORDER == kOuter && GATHER) p += (long long)token[j] * src.ld;
      if constexpr (DIRECT) {
        const void* from = p;
        if constexpr (!WHOLE) {
          const bool in = ORDER == kInner ? k + c * Tile::V < src.inner : k + r < src.outer;
          from = in ? from : (const void*)&kZeroChunk;
        }
        // a wave's 64 chunks; the same LDS base for all its lanes
        load_to_lds(from, lds + (j * NT + ((int)threadIdx.x & ~63)) * 16);
      } else if constexpr (WHOLE) {
        reg[j] = load16(p);
      } else {
        reg[j] = guarded(p, r, c);
      }
      if constexpr (ORDER == kInner) ptr[j] += Tile::BK;
      else if constexpr (!GATHER) ptr[j] += step;
    }
  }

  // Chunk c of row r, at p, with guards.
  __device__ __forceinline__ u32x4 guarded(const T* p, int r, int c) const {
    if constexpr (ORDER == kInner) {
      const int at = k + c * Tile::V;
      return load_guarded(first + r < src.outer ? p - at : nullptr, at, src.inner);
    } else {
      const int at = first + c * Tile::V;
      return load_edge(p, k + r < src.outer ? src.inner - at : 0, src.end());
    }
  }

  // RAGGED: the same chunks with guards, through registers, at once.  The K loop
  // counts on these chunks as loads in flight behind the tile it waits for; here
  // there may be none (a wave whose rows are all outside), so that everything
  // issued before them has to land first.
  template <int J0, int J1>
  __device__ __forceinline__ void load_guards(char* lds) {
    if constexpr (J0 < J1) wait_loads<0>();
#pragma unroll
    for (int j = J0; j < J1; ++j) {
      int r, c;
      Tile::slot(j * NT + (int)threadIdx.x, &r, &c);
      *reinterpret_cast<u32x4*>(lds + (j * NT + (int)threadIdx.x) * 16) = guarded(ptr[j], r, c);
      if constexpr (ORDER == kInner) ptr[j] += Tile::BK;
      else if constexpr (!GATHER) ptr[j] += step;
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

// Workgroup ids regrouped so that each of the 8 XCDs takes a contiguous range
// (workgroups go round-robin over XCDs, each with its own L2).
__device__ __forceinline__ int map_range(int id, int total) {
  const int per = total / 8, extra = total % 8, x = id % 8;
  return x * per + (x < extra ? x : extra) + id / 8;
}

// Tile (tm, tn) of workgroup id: down `GM` tile rows before the next tile
// column.
__device__ __forceinline__ void map_tile(int id, int tiles_m, int tiles_n, int* tm, int* tn) {
  const int t = map_range(id, tiles_m * tiles_n);
  constexpr int GM = 8;
  const int span = GM * tiles_n, band = t / span, m0 = band * GM;
  const int rows = tiles_m - m0 < GM ? tiles_m - m0 : GM;
  const int in = t - band * span;
  *tm = m0 + in % rows;
  *tn = in / rows;
}

template <int N, typename F>
__device__ __forceinline__ void static_for(F f) {
  if constexpr (N > 0) {
    static_for<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
  }
}

// All waves of the workgroup are here, and their LDS accesses are done.
__device__ __forceinline__ void workgroup_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Spread READS LDS reads and LOADS global loads evenly over the M matrix
// instructions of a step.
template <int READS, int M, int LOADS>
__device__ __forceinline__ void spread() {
#pragma unroll
  for (int i = 0; i < M; ++i) {
    const int n = (i + 1) * READS / M - i * READS / M;
    if (n == 1) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    if (n == 2) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
    if (n == 3) __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);
    if (n == 4) __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    const int v = (i + 1) * LOADS / M - i * LOADS / M;
    if (v == 1) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    if (v == 2) __builtin_amdgcn_sched_group_barrier(0x020, 2, 0);
    if (v == 3) __builtin_amdgcn_sched_group_barrier(0x020, 3, 0);
    if (v == 4) __builtin_amdgcn_sched_group_barrier(0x020, 4, 0);
  }
}

template <typename T, int LA, int LB, int BM, int BN, int WGM, int WGN, int LOADING, int MODE>
__global__ __launch_bounds__(WGM* WGN * 64) void prod_tile_kernel(const ProdArgs a) {
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

  // this workgroup's tile, operands and range of the summed index
  int tm, tn, e = 0, rows = a.M, row0 = 0, k_lo = 0, k_hi = a.K;
  if constexpr (MODE == kSums) {
    const int tiles = a.tiles_m * a.tiles_n;
    e = blockIdx.x / tiles;
    map_tile(blockIdx.x % tiles, a.tiles_m, a.tiles_n, &tm, &tn);
    group_bounds(a.offsets, e, a.rows, &k_lo, &k_hi);
    row0 = tm * BM;
    if (a.splits > 1) {
      const int part = ((k_hi - k_lo + a.splits - 1) / a.splits + BK - 1) / BK * BK;
      const long long from = k_lo + (long long)part * blockIdx.y;
      k_lo = from < k_hi ? (int)from : k_hi;
      k_hi = k_hi - k_lo < part ? k_hi : k_lo + part;
    }
  } else {
    map_tile(blockIdx.x, a.tiles_m, a.tiles_n, &tm, &tn);
    if constexpr (MODE == kRows) {
      int left;
      e = find_group(a.offsets, a.groups, a.rows, BM, tm, &row0, &left);
      if (e < 0) return;
      rows = row0 + left;
    } else {
      row0 = tm * BM;
      if (a.splits > 1) {
        k_lo = blockIdx.y * a.k_split;
        k_hi = k_lo + a.k_split < a.K ? k_lo + a.k_split : a.K;
      }
    }
  }
  const int col0 = tn * BN;

  const T* Ab = static_cast<const T*>(a.A);
  const T* Bb = static_cast<const T*>(a.B);
  if constexpr (MODE == kRows) Bb += e * a.strideB;
  Source<T> sa, sb;
  if constexpr (LA == kInner) {
    sa = {Ab, a.lda, rows, k_hi, a.gather, a.gather_rows};
  } else {
    sa = {Ab, a.lda, k_hi, a.M, a.gather, a.gather_rows};
  }
  if constexpr (LB == kInner) {
    sb = {Bb, a.ldb, a.N, k_hi, nullptr, 0};
  } else {
    sb = {Bb, a.ldb, k_hi, a.N, MODE == kSums ? a.gather_b : nullptr, a.gather_rows};
  }
  if constexpr (MODE == kDense) sa.gather = nullptr;

  using TA = OperandTile<T, LA, BM, NT>;
  using TB = OperandTile<T, LB, BN, NT>;
  // (a grouped sum's rows may be gathered on either side)
  using LoadA = Loader<T, LA, BM, NT, LOADING, MODE == kSums>;
  using LoadB = Loader<T, LB, BN, NT, LOADING, MODE == kSums>;
  LoadA la;
  LoadB lb;
  la.init(sa, row0, k_lo);
  lb.init(sb, col0, k_lo);

  f32x4 acc[RB][CB];
#pragma unroll
  for (int r = 0; r < RB; ++r)
#pragma unroll
    for (int c = 0; c < CB; ++c) acc[r][c] = f32x4{0, 0, 0, 0};

  // The K loop.  A tile's two steps (64 bytes of the summed index each) are cut
  // into G groups of one pair of A blocks against all B blocks.  While the
  // matrix cores run a group, the operands of the next are read from LDS into
  // the other registers; the last group of a tile reads the next tile's first
  // operands.  The one barrier per tile stands before that last group, whose
  // operands are already in registers: behind it every wave has read all of
  // this tile and the next tile has landed.
  //
  // Operand tiles A(0), B(0), A(1), B(1), ... follow each other through a ring of
  // LDS slots.  Direct loads use five of them (all of a compute unit's 160 KiB
  // for the 256 x 256 tiles): A(t + 2) and B(t + 1) are fetched during tile t,
  // two loads a step, so that the memory pipe never runs empty at a barrier.
  // (With two whole stages, all of tile t + 1 was fetched within tile t and
  // awaited at its end: 25.3 ns per inner index at 4096 x 4096 bf16, with the
  // ring 24.4, with the loads written as the instruction 22.8; the matrix
  // cores alone, no loads in the loop, take 20.4 at the clock this load leaves.)
  // Register loads use four: tile t + 1 is stored during tile t, tile t + 2
  // fetched.
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
        // reads first: the compiler keeps LDS reads behind loads into LDS
        if constexpr (g == G - 1) {
          // all but A(t + 2) has landed
          if constexpr (DIRECT) wait_loads<LoadA::L>();
          workgroup_barrier();
          read_a(a1, 0);          // past the last tile: some LDS, never used
          read_b(b1, 0);
        } else {
          read_a(a0, g + 1);
          if constexpr (p == GP - 1) read_b(b0, 1);
        }
        // the rest of B(t + 1), A(t + 2), and behind the barrier the first half
        // of B(t + 2), by quarters of the tile's groups
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
        // B's block as the instruction's rows: a lane then holds four
        // consecutive columns of one row of D
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

  // Epilogue: 32 rows of the wave tile at a time through the wave's own LDS,
  // so that each lane finishes 8 consecutive columns with 16-byte accesses.
  const void* bias = a.bias;
  char* D = static_cast<char*>(a.D);
  const int dsize = a.out32 ? 4 : (int)sizeof(T);
  if constexpr (MODE == kRows) {
    if (bias != nullptr) bias = static_cast<const T*>(bias) + e * a.strideBias;
  }
  if constexpr (MODE == kSums) {
    D += e * a.strideD * dsize;
    rows = a.M;
  }
  float* stg = reinterpret_cast<float*>(lds) + wave * 32 * EPI_LD;
  constexpr int LPR = WN / 8, RPP = 64 / LPR, PASSES = 32 / RPP;   // lanes per row, rows per pass
  const int col = (lane % LPR) * 8, n = col0 + wn + col;
  const bool split = MODE != kRows && a.splits > 1;
  float b8[8];
  load_bias<T>(a, split ? nullptr : bias, n, b8);
#pragma unroll 1
  for (int r = 0; r < RB / 2; ++r) {
    const int m0 = row0 + wm + 32 * r + lane / LPR;
    Raw8 res[PASSES] = {};
    if (a.R != nullptr && !split && n + 8 <= a.N) {
#pragma unroll
      for (int p = 0; p < PASSES; ++p)
        if (m0 + p * RPP < rows) res[p] = load_residual<T>(a, m0 + p * RPP, n);
    }
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
      const f32x4 x = *reinterpret_cast<const f32x4*>(from);
      const f32x4 y = *reinterpret_cast<const f32x4*>(from + 4);
      const int m = m0 + p * RPP;
      if (m < rows && n < a.N) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] = x[j] + b8[j];
          v[4 + j] = y[j] + b8[4 + j];
        }
        if (split) {
          const long long matrix = MODE == kSums ? (long long)blockIdx.y * a.groups + e : blockIdx.y;
          float* to = a.partial + (matrix * a.M + m) * a.N + n;
          if (n + 8 <= a.N) {
            put8<float>(to, 0, v);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (n + j < a.N) to[j] = v[j];
          }
        } else {
          finish_row<T>(a, D, m, n, v, res[p]);
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

}  // namespace layers
}  // namespace pgemm
