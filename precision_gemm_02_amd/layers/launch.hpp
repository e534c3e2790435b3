// Internal: what the entry points launch.  One translation unit per element
// type compiles its kernels (prod_f32.hip, prod_f16.hip, prod_bf16.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "prod.hpp"
#include "rows.hpp"
#include "route.hpp"

namespace pgemm {
namespace layers {

// A kernel's launch, its arguments in one struct.
template <typename A>
hipError_t launch(void (*kernel)(const A), dim3 grid, int threads, const A& a, hipStream_t s) {
  A copy = a;
  void* args[] = {&copy};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(threads), args, 0, s);
}

// The tile classes and the few-rows kernels of the products.
enum Kernel {
  kTile256 = 0,
  kTile128 = 1,
  kTile64 = 2,
  kFew16 = 3,
  kFew32 = 4,
  kFew16Wide = 5,
  kFew32Wide = 6
};

struct KernelShape {
  int bm, bn;
};
constexpr KernelShape kShape[3] = {{256, 256}, {128, 128}, {64, 64}};

// Columns of a workgroup of the few-rows kernels.
constexpr int few_columns(int kernel) { return kernel >= kFew16Wide ? 64 : 16; }

// The launch of a product: workgroups (x, and the splits of the summed index in
// y) and the threads of each.
struct ProdGrid {
  long long x;
  int y;
};
inline ProdGrid prod_grid(const ProdArgs& a, int mode, int kernel) {
  ProdGrid g = {(long long)a.tiles_m * a.tiles_n, mode == kRows ? 1 : a.splits};
  if (kernel >= kFew16) {
    // no more groups have rows than there are rows
    if (mode == kRows) g.x *= a.groups < a.rows ? a.groups : a.rows;
  } else if (mode == kSums) {
    g.x *= a.groups;   // (tiles_m of grouped rows already counts every group's)
  }
  return g;
}
constexpr int prod_threads(int kernel) {
  return kernel == kTile128 || kernel == kTile64 ? 256 : 512;
}

struct TypeOps {
  hipError_t (*prod)(const ProdArgs& a, int la, int lb, int mode, int kernel, int loading,
                     hipStream_t s);
  hipError_t (*slope)(const SlopeArgs& a, int groups, hipStream_t s);
  hipError_t (*column_sum)(const float* partial, void* out, int n, int groups, int chunks,
                           int out32, hipStream_t s);
  hipError_t (*combine)(const CombineArgs& a, hipStream_t s);
  hipError_t (*combine_back)(const CombineBackArgs& a, hipStream_t s);
  hipError_t (*route)(const RouteArgs& a, hipStream_t s);
  hipError_t (*route_back)(const RouteBackArgs& a, hipStream_t s);
};

const TypeOps& ops_f32();
const TypeOps& ops_f16();
const TypeOps& ops_bf16();

}  // namespace layers
}  // namespace pgemm
