// Internal: the launches of gated products of one element type (included by
// gated_*.hip).
#pragma once

#include "../layers/launch.hpp"
#include "ops.hpp"
#include "whole.hpp"

namespace pgemm {
namespace blocks {
namespace {

template <typename T, int LB, int PAIR, int KERNEL, int WGM, int WGN, int LOADING>
hipError_t pair_tile(const PairArgs& a, dim3 grid, hipStream_t s) {
  constexpr int BM = kShape[KERNEL].bm, BN = kShape[KERNEL].bn;
  static_assert(WGM * WGN * 64 == prod_threads(KERNEL), "the checked launch");
  return launch(&pair_tile_kernel<T, LB, BM, BN, WGM, WGN, LOADING, PAIR>, grid, WGM * WGN * 64, a, s);
}

template <typename T, int LB, int PAIR, int LOADING>
hipError_t pair_tiles(const PairArgs& a, int kernel, dim3 grid, hipStream_t s) {
  if constexpr (LOADING == kDirect) {
    if (kernel == kTile256) return pair_tile<T, LB, PAIR, kTile256, 2, 4, LOADING>(a, grid, s);
  }
  if (kernel == kTile128) return pair_tile<T, LB, PAIR, kTile128, 2, 2, LOADING>(a, grid, s);
  if (kernel == kTile64) return pair_tile<T, LB, PAIR, kTile64, 2, 2, LOADING>(a, grid, s);
  return hipErrorInvalidValue;
}

template <typename T, int LA, int LB, int PAIR, bool TAIL>
hipError_t whole_tile(const PairArgs& a, int kernel, dim3 grid, hipStream_t s) {
  if (kernel == kTile256)
    return launch(&pair_whole_kernel<T, LA, LB, 256, 256, 2, 4, PAIR, TAIL>, grid,
                  prod_threads(kTile256), a, s);
  if (kernel == kTile128)
    return launch(&pair_whole_kernel<T, LA, LB, 128, 128, 2, 2, PAIR, TAIL>, grid,
                  prod_threads(kTile128), a, s);
  if (kernel == kTile64)
    return launch(&pair_whole_kernel<T, LA, LB, 64, 64, 2, 2, PAIR, TAIL>, grid,
                  prod_threads(kTile64), a, s);
  return hipErrorInvalidValue;
}

template <typename T, int LA, int LB, int PAIR>
hipError_t whole_tiles(const PairArgs& a, int kernel, dim3 grid, hipStream_t s) {
  const int along = PAIR == kHalves ? a.inner : a.p.K;
  return along % (int)(128 / sizeof(T)) ? whole_tile<T, LA, LB, PAIR, true>(a, kernel, grid, s)
                                        : whole_tile<T, LA, LB, PAIR, false>(a, kernel, grid, s);
}

template <typename T>
hipError_t pair_reduce(const PairArgs& a, int count, hipStream_t s) {
  const long long items = (long long)a.p.M * ((a.p.N + 7) / 8);
  return launch(&pair_reduce_kernel<T>, dim3((unsigned)((items + 255) / 256), (unsigned)count), 256, a,
                s);
}

template <typename T, int LB, int MB, int NB, int WAVES>
hipError_t gate_rows(const PairArgs& a, dim3 grid, hipStream_t s) {
  static_assert(prod_threads(kFew16) >= WAVES * 64, "the checked launch");
  return launch(&gate_rows_kernel<T, LB, MB, NB, WAVES>, grid, WAVES * 64, a, s);
}

template <typename T, int LB, int PAIR>
hipError_t pair(const PairArgs& a, int kernel, int loading, bool whole, hipStream_t s) {
  const ProdGrid g = prod_grid(a.p, kDense, kernel);
  const dim3 grid((unsigned)g.x, (unsigned)g.y);
  hipError_t e = hipErrorInvalidValue;
  if (kernel >= kFew16) {
    if constexpr (PAIR == kColumns) {
      e = kernel == kFew16       ? gate_rows<T, LB, 1, 2, 4>(a, grid, s)
          : kernel == kFew32     ? gate_rows<T, LB, 2, 2, 4>(a, grid, s)
          : kernel == kFew16Wide ? gate_rows<T, LB, 1, 4, 2>(a, grid, s)
                                 : gate_rows<T, LB, 2, 4, 2>(a, grid, s);
    }
  } else if (whole) {
    e = whole_tiles<T, kInner, LB, PAIR>(a, kernel, grid, s);
  } else if (loading == kDirect) {
    e = pair_tiles<T, LB, PAIR, kDirect>(a, kernel, grid, s);
  } else if (sizeof(T) == 2 && loading == kRagged) {
    if constexpr (sizeof(T) == 2) e = pair_tiles<T, LB, PAIR, kRagged>(a, kernel, grid, s);
  } else {
    e = pair_tiles<T, LB, PAIR, kThrough>(a, kernel, grid, s);
  }
  if (e != hipSuccess || a.p.splits <= 1) return e;
  if constexpr (PAIR == kHalves) return pair_reduce<T>(a, 1, s);
  const long long items = (long long)a.p.M * ((a.p.N + 7) / 8);
  return launch(&gate_reduce_kernel<T>, dim3((unsigned)((items + 255) / 256)), 256, a, s);
}

template <typename T>
hipError_t pair(const PairArgs& a, int lb, int pair_, int kernel, int loading, bool whole,
                hipStream_t s) {
  if (pair_ == kColumns)
    return lb == kInner ? pair<T, kInner, kColumns>(a, kernel, loading, whole, s)
                        : pair<T, kOuter, kColumns>(a, kernel, loading, whole, s);
  return lb == kInner ? pair<T, kInner, kHalves>(a, kernel, loading, whole, s)
                      : pair<T, kOuter, kHalves>(a, kernel, loading, whole, s);
}

template <typename T>
hipError_t apart(const PairArgs& a, int kernel, hipStream_t s) {
  const ProdGrid g = prod_grid(a.p, kDense, kernel);
  const dim3 grid((unsigned)(g.x * a.count), (unsigned)g.y);
  const hipError_t e = whole_tiles<T, kOuter, kOuter, kApart>(a, kernel, grid, s);
  return e != hipSuccess || a.p.splits <= 1 ? e : pair_reduce<T>(a, a.count, s);
}

template <typename T>
hipError_t slope(const GateSlopeArgs& a, bool sums32, hipStream_t s) {
  const dim3 grid((unsigned)((a.half + a.tpr * 8 - 1) / (a.tpr * 8)), (unsigned)a.chunks);
  if constexpr (sizeof(T) == 4) return launch(&gate_slope_kernel<T, kExact>, grid, 256, a, s);
  else if (sums32) return launch(&gate_slope_kernel<T, kFine>, grid, 256, a, s);
  else return launch(&gate_slope_kernel<T, kFast>, grid, 256, a, s);
}

template <typename T>
hipError_t pad(const PadRowsArgs& a, int count, hipStream_t s) {
  return launch(&pad_rows_kernel<T>, dim3(2048, (unsigned)count), 256, a, s);
}

template <typename T>
const GateOps& ops() {
  static const GateOps o = {&pair<T>, &apart<T>, &slope<T>, &pad<T>};
  return o;
}

}  // namespace
}  // namespace blocks
}  // namespace pgemm
