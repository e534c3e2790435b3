// Internal: a kernel's launch.
#pragma once

#include <hip/hip_runtime.h>

namespace pgemm {
namespace blocks {

template <typename A>
hipError_t launch(void (*kernel)(const A), dim3 grid, int threads, const A& a, hipStream_t s) {
  A copy = a;
  void* args[] = {&copy};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(threads), args, 0, s);
}

}  // namespace blocks
}  // namespace pgemm
