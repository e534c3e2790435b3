// Internal: the launches of one element type (included by prod_*.hip).
#pragma once

#include "launch.hpp"
#include "prod_rows.hpp"
#include "prod_tile.hpp"

namespace pgemm {
namespace layers {
namespace {

inline dim3 grid_of(const ProdArgs& a, int mode, int kernel) {
  const ProdGrid g = prod_grid(a, mode, kernel);
  return dim3((unsigned)g.x, (unsigned)g.y);
}

template <typename T, int LA, int LB, int KERNEL, int WGM, int WGN, int LOADING, int MODE>
hipError_t launch_tile(const ProdArgs& a, hipStream_t s) {
  constexpr int BM = kShape[KERNEL].bm, BN = kShape[KERNEL].bn;
  static_assert(WGM * WGN * 64 == prod_threads(KERNEL), "the checked launch");
  return launch(&prod_tile_kernel<T, LA, LB, BM, BN, WGM, WGN, LOADING, MODE>,
                grid_of(a, MODE, KERNEL), WGM * WGN * 64, a, s);
}

template <typename T, int LA, int LB, int MODE, int LOADING>
hipError_t prod_tile(const ProdArgs& a, int kernel, hipStream_t s) {
  if constexpr (LOADING == kDirect) {
    if (kernel == kTile256) return launch_tile<T, LA, LB, kTile256, 2, 4, LOADING, MODE>(a, s);
  }
  if (kernel == kTile128) return launch_tile<T, LA, LB, kTile128, 2, 2, LOADING, MODE>(a, s);
  if (kernel == kTile64) return launch_tile<T, LA, LB, kTile64, 2, 2, LOADING, MODE>(a, s);
  return hipErrorInvalidValue;
}

template <typename T, int LA, int LB, int MODE>
hipError_t prod_tile(const ProdArgs& a, int kernel, int loading, hipStream_t s) {
  if (loading == kDirect) return prod_tile<T, LA, LB, MODE, kDirect>(a, kernel, s);
  if constexpr (MODE != kSums && sizeof(T) == 2) {
    if (loading == kRagged) return prod_tile<T, LA, LB, MODE, kRagged>(a, kernel, s);
  }
  return prod_tile<T, LA, LB, MODE, kThrough>(a, kernel, s);
}

template <typename T, int LB, int MB, int MODE>
hipError_t prod_few(const ProdArgs& a, int kernel, hipStream_t s) {
  const dim3 grid = grid_of(a, MODE, kernel);
  static_assert(prod_threads(kFew16) == 512, "the checked launch");
  if (kernel >= kFew16Wide)
    return launch(&prod_rows_kernel<T, LB, MB, 4, 8, MODE>, grid, 512, a, s);
  return launch(&prod_rows_kernel<T, LB, MB, 1, 8, MODE>, grid, 512, a, s);
}

template <typename T, int LB, int MODE>
hipError_t prod_few(const ProdArgs& a, int kernel, hipStream_t s) {
  return kernel == kFew16 || kernel == kFew16Wide ? prod_few<T, LB, 1, MODE>(a, kernel, s)
                                                  : prod_few<T, LB, 2, MODE>(a, kernel, s);
}

template <typename T>
hipError_t reduce(const ProdArgs& a, hipStream_t s) {
  const long long items = (long long)(a.groups > 0 ? a.groups : 1) * a.M * ((a.N + 7) / 8);
  return launch(&prod_reduce_kernel<T>, dim3((unsigned)((items + 255) / 256)), 256, a, s);
}

template <typename T>
hipError_t prod(const ProdArgs& a, int la, int lb, int mode, int kernel, int loading,
                hipStream_t s) {
  hipError_t e;
  const bool few = kernel >= kFew16;
  if (mode == kDense) {
    if (few)
      e = lb == kInner ? prod_few<T, kInner, kDense>(a, kernel, s)
                       : prod_few<T, kOuter, kDense>(a, kernel, s);
    else if (la == kOuter)
      e = prod_tile<T, kOuter, kOuter, kDense>(a, kernel, loading, s);
    else
      e = lb == kInner ? prod_tile<T, kInner, kInner, kDense>(a, kernel, loading, s)
                       : prod_tile<T, kInner, kOuter, kDense>(a, kernel, loading, s);
    return e == hipSuccess && a.splits > 1 ? reduce<T>(a, s) : e;
  }
  if (mode == kRows) {
    if (few)
      return lb == kInner ? prod_few<T, kInner, kRows>(a, kernel, s)
                          : prod_few<T, kOuter, kRows>(a, kernel, s);
    return lb == kInner ? prod_tile<T, kInner, kInner, kRows>(a, kernel, loading, s)
                        : prod_tile<T, kInner, kOuter, kRows>(a, kernel, loading, s);
  }
  e = prod_tile<T, kOuter, kOuter, kSums>(a, kernel, loading, s);
  return e == hipSuccess && a.splits > 1 ? reduce<T>(a, s) : e;
}

template <typename T>
hipError_t slope(const SlopeArgs& a, int groups, hipStream_t s) {
  const unsigned cols = (unsigned)((a.n + a.tpr * 8 - 1) / (a.tpr * 8));
  const dim3 grid(cols, (unsigned)a.chunks, (unsigned)groups);
  if constexpr (sizeof(T) == 4) return launch(&slope_kernel<T, kExact>, grid, 256, a, s);
  else if (a.sums32) return launch(&slope_kernel<T, kFine>, grid, 256, a, s);
  else return launch(&slope_kernel<T, kFast>, grid, 256, a, s);
}

template <typename T>
hipError_t column_sum(const float* partial, void* out, int n, int groups, int chunks, int out32,
                      hipStream_t s) {
  void* args[] = {&partial, &out, &n, &chunks, &out32};
  return hipLaunchKernel(reinterpret_cast<const void*>(&column_sum_kernel<T>),
                         dim3((unsigned)((n + 31) / 32), (unsigned)groups), dim3(256), args, 0, s);
}

// Workgroups of 256 threads in one launch; more tokens take several (a launch
// has less than 2^32 threads).
constexpr int kMostGroups = 1 << 23;

// p moved by `rows` rows of `ld` elements of T (nullptr stays).
template <typename T, typename P>
P* rows_on(P* p, long long rows, long long ld) {
  return p == nullptr ? nullptr : (P*)((const char*)p + rows * ld * (long long)sizeof(T));
}

template <typename T>
hipError_t combine(const CombineArgs& all, hipStream_t s) {
  const int tpb = 256 / all.tpr;
  const long long part = (long long)kMostGroups * tpb;
  for (long long t0 = 0; t0 < all.m; t0 += part) {
    CombineArgs a = all;
    a.m = (int)(all.m - t0 < part ? all.m - t0 : part);
    a.slots = rows_on<int>(a.slots, t0, a.top);
    a.weights = rows_on<float>(a.weights, t0, a.top);
    a.R = rows_on<T>(a.R, t0, a.ldr);
    a.out = rows_on<T>(a.out, t0, a.ldo);
    const hipError_t e = launch(&combine_kernel<T>,
                                dim3((unsigned)((a.m + tpb - 1) / tpb),
                                     (unsigned)((a.n + a.tpr * 8 - 1) / (a.tpr * 8))),
                                256, a, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T>
hipError_t combine_back(const CombineBackArgs& all, hipStream_t s) {
  const int part = kMostGroups * 4 / all.top;
  for (long long t0 = 0; t0 < all.m; t0 += part) {
    CombineBackArgs a = all;
    a.m = (int)(all.m - t0 < part ? all.m - t0 : part);
    a.dout = rows_on<T>(a.dout, t0, a.ldo);
    a.slots = rows_on<int>(a.slots, t0, a.top);
    a.weights = rows_on<float>(a.weights, t0, a.top);
    a.dweights = rows_on<float>(a.dweights, t0, a.top);
    const long long waves = (long long)a.m * a.top;
    const hipError_t e =
        launch(&combine_back_kernel<T>, dim3((unsigned)((waves + 3) / 4)), 256, a, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Experts per lane, one class for each number of registers that pays: a class of
// three for up to 192 (16384 tokens: 160 experts 39 us, with the class of four 44;
// 192 in 6 groups 41, so 46).
template <typename T>
hipError_t route(const RouteArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.blocks);
  hipError_t e;
  if (a.experts <= 64) e = launch(&route_kernel<T, 1>, grid, 1024, a, s);
  else if (a.experts <= 128) e = launch(&route_kernel<T, 2>, grid, 1024, a, s);
  else if (a.experts <= 192) e = launch(&route_kernel<T, 3>, grid, 1024, a, s);
  else if (a.experts <= 256) e = launch(&route_kernel<T, 4>, grid, 1024, a, s);
  else if (a.experts <= 512) e = launch(&route_kernel<T, 8>, grid, 1024, a, s);
  else e = launch(&route_kernel<T, 16>, grid, 1024, a, s);
  if (e != hipSuccess || a.blocks == 1) return e;
  if (a.blocks <= 512) return launch(&route_place_kernel<T, true>, grid, 1024, a, s);
  e = launch(&route_sum_kernel<T>, dim3((unsigned)a.experts), 64, a, s);
  if (e != hipSuccess) return e;
  return launch(&route_place_kernel<T, false>, grid, 1024, a, s);
}

// Up to 256 experts a class of three would give little (16384 tokens of 192: 14 us,
// with it 13); above, the class of 16 is slow for what it does (512: 69 us, where a
// class of eight took 25) and serves for its rarity.
template <typename T>
hipError_t route_back(const RouteBackArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.m + 3) / 4));
  if (a.experts <= 64) return launch(&route_back_kernel<T, 1>, grid, 256, a, s);
  if (a.experts <= 128) return launch(&route_back_kernel<T, 2>, grid, 256, a, s);
  if (a.experts <= 256) return launch(&route_back_kernel<T, 4>, grid, 256, a, s);
  return launch(&route_back_kernel<T, 16>, grid, 256, a, s);
}

template <typename T>
const TypeOps& type_ops() {
  static const TypeOps ops = {&prod<T>,         &slope<T>, &column_sum<T>, &combine<T>,
                              &combine_back<T>, &route<T>, &route_back<T>};
  return ops;
}

}  // namespace
}  // namespace layers
}  // namespace pgemm
