// The tile kernel: one BM x BN tile of D per workgroup, WGM x WGN waves,
// matrix cores fed from LDS.  See prod.hpp for the operands' orders and the
// groups.
#pragma once

#include "prod.hpp"

namespace pgemm {
namespace layers {

// 16 zero bytes: what a lane loads for a chunk outside its operand.
static __device__ const u32x4 kZeroChunk = {0, 0, 0, 0};

// One operand's tile: `EXT` output indices by 128 bytes' worth of the summed
// index (BK = 64 16-bit or 32 fp32 elements), in 16-byte chunks.
//
// Inner order: LDS row r holds output index r, 8 chunks along the summed
// index; chunk c sits at c ^ (r & 7).  The b128 operand reads (16 rows, one
// chunk per lane group) then touch every 16-byte bank group once per
// cycle: of the two 8-row blocks served together, one reads chunk c and the
// other c ^ 1, so their flipped positions never meet.
//
// Outer order: LDS row p holds summed index p, EXT contiguous output indices.
// 16-bit operands are read through the transposing ds_read_b64_tr_b16 (16
// lanes read a 4 x 16 block by rows and receive it by columns), fp32 with one
// b32 per inner index.  The 32-byte (16-bit) or 64-byte (fp32) pieces that
// one 16-column block takes from a row are flipped by the row so that the
// rows read together fall into different banks.
template <typename T, int ORDER, int EXT, int NT>
struct OperandTile {
  static constexpr int S = sizeof(T);
  static constexpr int V = 16 / S;              // elements per chunk
  static constexpr int BK = 128 / S;
  static constexpr int BYTES = EXT * 128;
  static constexpr int ROW_CHUNKS = ORDER == kInner ? 8 : EXT / V;
  static constexpr int ROW_BYTES = ROW_CHUNKS * 16;
  static constexpr int LOADS = BYTES / (16 * NT);
  static_assert(BYTES % (16 * NT) == 0, "whole chunks per thread");
  // outer order: pieces per row (of one 16-column block), as a power of two
  static constexpr int PIECE = 16 * S;          // bytes
  static constexpr int PIECES = EXT / 16;

  // The flip of row p's pieces (outer order).
  static __device__ __forceinline__ int flip(int p) {
    if constexpr (S == 2) {
      const int q = (p & 3) | (((p >> 3) & 1) << 2);
      constexpr int b = PIECES >= 8 ? 3 : PIECES == 4 ? 2 : 1;
      return q >> (3 - b);
    } else {
      return (p >> 2) & (PIECES >= 4 ? 3 : 1);
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

  // Fragment of 16-index block b (from index `first`), step kk (64 bytes of
  // the summed index), from the tile at lds.
  static __device__ __forceinline__ u32x4 frag(const char* lds, int first, int b, int kk) {
    const int l = threadIdx.x & 63, g = l >> 4, i = l & 15;
    if constexpr (ORDER == kInner) {
      const int row = first + 16 * b + i;
      const int c = (4 * kk + g) ^ (i & 7);
      return *reinterpret_cast<const u32x4*>(lds + row * 128 + c * 16);
    } else if constexpr (S == 2) {
      u32x4 out;
      const int piece = first / 16 + b;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int p = 32 * kk + 8 * g + 4 * h + (i >> 2);
        const int f = flip(8 * g + (i >> 2));   // 32 kk and 4 h do not enter
        const char* at = lds + p * ROW_BYTES + (piece ^ f) * PIECE + (i & 3) * 8;
        const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s16x4*)(const_cast<char*>(at)));
        const u32x2 w = __builtin_bit_cast(u32x2, v);
        out[2 * h] = w[0];
        out[2 * h + 1] = w[1];
      }
      return out;
    } else {
      u32x4 out;
      const int piece = first / 16 + b;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int p = 16 * kk + 4 * g + s;
        const char* at = lds + p * ROW_BYTES + (piece ^ flip(4 * g)) * PIECE + i * 4;
        out[s] = *reinterpret_cast<const uint32_t*>(at);
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

  __device__ __forceinline__ const T* row(int r) const {
    if (r >= outer) return nullptr;
    if (gather != nullptr) {
      const int t = gather[r];
      if ((unsigned)t >= (unsigned)gather_rows) return nullptr;
      return base + (long long)t * ld;
    }
    return base + (long long)r * ld;
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

// The same where the whole chunk is known to be inside: no branch, a row that
// is not there reads the zero chunk.
template <typename T>
__device__ __forceinline__ u32x4 load_whole(const T* row, int c0) {
  return load16(row != nullptr ? (const void*)(row + c0) : (const void*)&kZeroChunk);
}

// One operand's loads.  DIRECT: straight into LDS (global_load_lds_dwordx4:
// a wave writes 64 consecutive chunks, so the layout's flips are applied to
// the global addresses).  It needs 16-byte aligned rows and no chunk that
// straddles the operand's end.  Otherwise through registers, with guards.
template <typename T, int ORDER, int EXT, int NT, bool DIRECT>
struct Loader {
  using Tile = OperandTile<T, ORDER, EXT, NT>;
  static constexpr int L = Tile::LOADS;
  Source<T> src;
  int first;                       // first output index of the tile
  const T* ptr[L];                 // inner order: the thread's rows
  u32x4 reg[DIRECT ? 1 : L];

  __device__ __forceinline__ void init(const Source<T>& s, int first_out) {
    src = s;
    first = first_out;
    if constexpr (ORDER == kInner) {
#pragma unroll
      for (int j = 0; j < L; ++j) {
        int r, c;
        Tile::slot(j * NT + (int)threadIdx.x, &r, &c);
        ptr[j] = src.row(first + r);
      }
    }
  }

  // Start the loads of summed indices k0 .. k0+BK-1.
  __device__ __forceinline__ void load(char* lds, int k0) {
    // no chunk of this tile straddles the operand's end (the same for the
    // whole workgroup)
    const bool whole = ORDER == kInner ? k0 + Tile::BK <= src.inner : first + EXT <= src.inner;
    if (DIRECT || whole) load_as<true>(lds, k0);
    else load_as<false>(lds, k0);
  }

  template <bool WHOLE>
  __device__ __forceinline__ void load_as(char* lds, int k0) {
#pragma unroll
    for (int j = 0; j < L; ++j) {
      int r, c;
      Tile::slot(j * NT + (int)threadIdx.x, &r, &c);
      const T* row;
      int at;
      if constexpr (ORDER == kInner) {
        row = ptr[j];
        at = k0 + c * Tile::V;
      } else {
        row = src.row(k0 + r);
        at = first + c * Tile::V;
      }
      if constexpr (DIRECT) {
        const void* p = row != nullptr && at < src.inner ? (const void*)(row + at)
                                                          : (const void*)&kZeroChunk;
        // a wave's 64 chunks; the same LDS base for all its lanes
        char* to = lds + (j * NT + ((int)threadIdx.x & ~63)) * 16;
        __builtin_amdgcn_global_load_lds(
            (const __attribute__((address_space(1))) void*)p,
            (__attribute__((address_space(3))) void*)to, 16, 0, 0);
      } else {
        if constexpr (WHOLE) reg[j] = load_whole(row, at);
        else reg[j] = load_guarded(row, at, src.inner);
      }
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

// Tile (tm, tn) of workgroup id: ids are regrouped so that each of the 8 XCDs
// takes a contiguous range (workgroups go round-robin over XCDs, each with its
// own L2), then walk down `GM` tile rows before the next tile column.
__device__ __forceinline__ void map_tile(int id, int tiles_m, int tiles_n, int* tm, int* tn) {
  const int total = tiles_m * tiles_n, per = total / 8, extra = total % 8;
  const int x = id % 8, at = id / 8;
  const int t = x * per + (x < extra ? x : extra) + at;
  constexpr int GM = 8;
  const int span = GM * tiles_n, band = t / span, m0 = band * GM;
  const int rows = tiles_m - m0 < GM ? tiles_m - m0 : GM;
  const int in = t - band * span;
  *tm = m0 + in % rows;
  *tn = in / rows;
}

template <typename T, int LA, int LB, int BM, int BN, int WGM, int WGN, bool DIRECT, int MODE>
__global__ __launch_bounds__(WGM* WGN * 64) void prod_tile_kernel(const ProdArgs a) {
  constexpr int NT = WGM * WGN * 64;
  constexpr int WM = BM / WGM, WN = BN / WGN, RB = WM / 16, CB = WN / 16;
  constexpr int BK = 128 / (int)sizeof(T);
  constexpr int STAGE = (BM + BN) * 128;
  constexpr int EPI_LD = WN + 4;
  constexpr int EPI = WGM * WGN * 16 * EPI_LD * 4;
  constexpr int LDS = 2 * STAGE > EPI ? 2 * STAGE : EPI;
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
  int k0 = k_lo;
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
  Loader<T, LA, BM, NT, DIRECT> la;
  Loader<T, LB, BN, NT, DIRECT> lb;
  la.init(sa, row0);
  lb.init(sb, col0);

  f32x4 acc[RB][CB];
#pragma unroll
  for (int r = 0; r < RB; ++r)
#pragma unroll
    for (int c = 0; c < CB; ++c) acc[r][c] = f32x4{0, 0, 0, 0};

  const int nk = (k_hi - k_lo + BK - 1) / BK;
  if (nk > 0) {
    la.load(lds, k0);
    lb.load(lds + BM * 128, k0);
    if constexpr (!DIRECT) {
      la.store(lds);
      lb.store(lds + BM * 128);
      if (nk > 1) {
        la.load(nullptr, k0 + BK);
        lb.load(nullptr, k0 + BK);
      }
    }
  }
  for (int kt = 0; kt < nk; ++kt) {
    char* cur = lds + (kt & 1) * STAGE;
    char* nxt = lds + ((kt + 1) & 1) * STAGE;
    // this wave's loads of tile kt have landed; then every wave's have, and
    // nobody reads the other stage any more
    if constexpr (DIRECT) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    k0 += BK;
    if constexpr (DIRECT) {
      if (kt + 1 < nk) {
        la.load(nxt, k0);
        lb.load(nxt + BM * 128, k0);
      }
    } else {
      if (kt + 1 < nk) {
        la.store(nxt);
        lb.store(nxt + BM * 128);
      }
      if (kt + 2 < nk) {
        la.load(nullptr, k0 + BK);
        lb.load(nullptr, k0 + BK);
      }
    }
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      u32x4 fa[RB], fb[CB];
#pragma unroll
      for (int c = 0; c < CB; ++c) fb[c] = TB::frag(cur + BM * 128, wn, c, kk);
#pragma unroll
      for (int r = 0; r < RB; ++r) fa[r] = TA::frag(cur, wm, r, kk);
      // B's block as the instruction's rows: a lane then holds four
      // consecutive columns of one row of D
#pragma unroll
      for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int c = 0; c < CB; ++c) acc[r][c] = Elem<T>::mfma(fb[c], fa[r], acc[r][c]);
    }
  }
  __syncthreads();   // the operands' LDS becomes the epilogue's

  // Epilogue: 16 rows of the wave tile at a time through the wave's own LDS,
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
  float* stg = reinterpret_cast<float*>(lds) + wave * 16 * EPI_LD;
  constexpr int LPR = WN / 8, RPP = 64 / LPR;   // lanes per row, rows per pass
#pragma unroll
  for (int r = 0; r < RB; ++r) {
#pragma unroll
    for (int c = 0; c < CB; ++c)
      *reinterpret_cast<f32x4*>(stg + (lane & 15) * EPI_LD + 16 * c + 4 * (lane >> 4)) = acc[r][c];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int p = 0; p < 16; p += RPP) {
      const int row = p + lane / LPR, col = (lane % LPR) * 8;
      const float* from = stg + row * EPI_LD + col;
      const f32x4 x = *reinterpret_cast<const f32x4*>(from);
      const f32x4 y = *reinterpret_cast<const f32x4*>(from + 4);
      const int m = row0 + wm + 16 * r + row, n = col0 + wn + col;
      if (m < rows && n < a.N) {
        const float v[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
        if (MODE == kDense && a.splits > 1) {
          float* to = a.partial + ((long long)blockIdx.y * a.M + m) * a.N + n;
          if (n + 8 <= a.N) {
            put8<float>(to, 0, v);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (n + j < a.N) to[j] = v[j];
          }
        } else {
          finish8<T>(a, bias, D, m, n, v);
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

}  // namespace layers
}  // namespace pgemm
