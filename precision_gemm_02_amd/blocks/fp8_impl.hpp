// Internal: the launches of 8-bit products whose left operand has type FA, with results
// of 16 bits or (WIDE) of 32 (included by fp8_*.hip).
#pragma once

#include "../layers/launch.hpp"
#include "fp8.hpp"
#include "ops.hpp"
#include "whole8.hpp"

namespace pgemm {
namespace blocks {
namespace {

template <int FA, int FB, bool COLS, bool WIDE, int KERNEL, int WGM, int WGN, bool DIRECT>
hipError_t tile8(const Prod8Args& a, dim3 grid, hipStream_t s) {
  constexpr int BM = kShape[KERNEL].bm, BN = kShape[KERNEL].bn;
  static_assert(WGM * WGN * 64 == prod_threads(KERNEL), "the checked launch");
  return launch(&prod8_tile_kernel<FA, FB, BM, BN, WGM, WGN, DIRECT, COLS, WIDE>, grid,
                WGM * WGN * 64, a, s);
}

template <int FA, int FB, bool COLS, bool TAIL>
hipError_t whole8(const Prod8Args& a, int kernel, dim3 grid, hipStream_t s) {
  if (kernel == kTile256)
    return launch(&prod8_whole_kernel<FA, FB, 256, 256, 2, 4, COLS, TAIL>, grid,
                  prod_threads(kTile256), a, s);
  if (kernel == kTile128)
    return launch(&prod8_whole_kernel<FA, FB, 128, 128, 2, 2, COLS, TAIL>, grid,
                  prod_threads(kTile128), a, s);
  return launch(&prod8_whole_kernel<FA, FB, 64, 64, 2, 2, COLS, TAIL>, grid, prod_threads(kTile64), a,
                s);
}

template <int FA, int FB, bool COLS, bool WIDE, int MB, int NB>
hipError_t rows8(const Prod8Args& a, dim3 grid, hipStream_t s) {
  static_assert(prod_threads(kFew16) == 512, "the checked launch");
  return launch(&prod8_rows_kernel<FA, FB, MB, NB, 8, COLS, WIDE>, grid, 512, a, s);
}

template <int FA, int FB, bool COLS, bool WIDE>
hipError_t prod8(const Prod8Args& a, int kernel, int loading, hipStream_t s) {
  const ProdGrid g = prod_grid(a.p, kDense, kernel);
  const dim3 grid((unsigned)g.x, (unsigned)g.y);
  hipError_t e = hipErrorInvalidValue;
  if (!WIDE && loading == kWhole && kernel <= kTile64) {
    if constexpr (!WIDE)
      e = a.p.K % 128 ? whole8<FA, FB, COLS, true>(a, kernel, grid, s)
                      : whole8<FA, FB, COLS, false>(a, kernel, grid, s);
  } else if (kernel == kTile256) {
    if constexpr (!WIDE) e = tile8<FA, FB, COLS, WIDE, kTile256, 2, 4, true>(a, grid, s);
  } else if (kernel == kTile128) {
    e = loading != kThrough ? tile8<FA, FB, COLS, WIDE, kTile128, 2, 2, true>(a, grid, s)
               : tile8<FA, FB, COLS, WIDE, kTile128, 2, 2, false>(a, grid, s);
  } else if (kernel == kTile64) {
    e = loading != kThrough ? tile8<FA, FB, COLS, WIDE, kTile64, 2, 2, true>(a, grid, s)
               : tile8<FA, FB, COLS, WIDE, kTile64, 2, 2, false>(a, grid, s);
  } else if (kernel == kFew16) {
    e = rows8<FA, FB, COLS, WIDE, 1, 1>(a, grid, s);
  } else if (kernel == kFew32) {
    e = rows8<FA, FB, COLS, WIDE, 2, 1>(a, grid, s);
  } else if (kernel == kFew16Wide) {
    e = rows8<FA, FB, COLS, WIDE, 1, 2>(a, grid, s);
  } else {
    e = rows8<FA, FB, COLS, WIDE, 2, 2>(a, grid, s);
  }
  if (e != hipSuccess || a.p.splits <= 1) return e;
  const long long items = (long long)a.p.M * ((a.p.N + 7) / 8);
  return launch(&prod8_reduce_kernel<FA, WIDE>, dim3((unsigned)((items + 255) / 256)), 256, a, s);
}

template <int FA, bool WIDE>
hipError_t prod8_of(const Prod8Args& a, int w_type, int kernel, int loading, hipStream_t s) {
  const bool cols = a.w_shift == 0;
  if (w_type == kE4M3)
    return cols ? prod8<FA, kE4M3, true, WIDE>(a, kernel, loading, s)
                : prod8<FA, kE4M3, false, WIDE>(a, kernel, loading, s);
  return cols ? prod8<FA, kE5M2, true, WIDE>(a, kernel, loading, s)
              : prod8<FA, kE5M2, false, WIDE>(a, kernel, loading, s);
}

}  // namespace
}  // namespace blocks
}  // namespace pgemm
