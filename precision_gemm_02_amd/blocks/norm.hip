// Layer norm's launches, for each type.
#include "../layers/launch.hpp"
#include "ops.hpp"
#include "pgemm_layers.h"

namespace pgemm {
namespace blocks {
namespace {

using layers::launch;

// Workgroups of up to 1024 threads in one launch; more rows take several (a launch
// has less than 2^32 threads).
constexpr int kMostGroups = 1 << 21;

template <typename T, typename P>
P* rows_on(P* p, long long rows, long long ld) {
  return p == nullptr ? nullptr : (P*)((const char*)p + rows * ld * (long long)sizeof(T));
}

template <typename T>
hipError_t norm_parts(void (*kernel)(const NormArgs), int rows, int threads, const NormArgs& all,
                      hipStream_t s) {
  const long long part = (long long)kMostGroups * rows;
  for (long long r = 0; r < all.m; r += part) {
    NormArgs a = all;
    a.m = (int)(all.m - r < part ? all.m - r : part);
    a.X = rows_on<T>(a.X, r, a.ldx);
    a.Y = rows_on<T>(a.Y, r, a.ldy);
    a.mean = rows_on<float>(a.mean, r, 1);
    a.rstd = rows_on<float>(a.rstd, r, 1);
    const hipError_t e = launch(kernel, dim3((unsigned)((a.m + rows - 1) / rows)), threads, a, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T, int TPR, int C, int NT>
hipError_t norm_as(const NormArgs& a, hipStream_t s) {
  return norm_parts<T>(&norm_kernel<T, TPR, C, NT>, NT / TPR, NT, a, s);
}

template <typename T>
hipError_t norm(const NormArgs& a, hipStream_t s) {
  if (a.n <= 128) return norm_as<T, 16, 1, 256>(a, s);
  if (a.n <= 512) return norm_as<T, 64, 1, 256>(a, s);
  if (a.n <= 1024) return norm_as<T, 64, 2, 256>(a, s);
  if (a.n <= 2048) return norm_as<T, 256, 1, 256>(a, s);
  if (a.n <= 4096) return norm_as<T, 256, 2, 256>(a, s);
  if (a.n <= 8192) return norm_as<T, 512, 2, 512>(a, s);
  if (a.n <= 16384) return norm_as<T, 1024, 2, 1024>(a, s);
  if (a.n <= kRowMost) return norm_as<T, 1024, 4, 1024>(a, s);
  return norm_parts<T>(&norm_long_kernel<T>, 1, 1024, a, s);
}

template <typename T, int TPR, int C, int NT>
hipError_t norm_back_as(const NormBackArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.groups);
  if constexpr (TPR * C * 8 <= kSumMost) {
    if (a.partial != nullptr) return launch(&norm_back_kernel<T, TPR, C, NT, true>, grid, NT, a, s);
  }
  return launch(&norm_back_kernel<T, TPR, C, NT, false>, grid, NT, a, s);
}

template <typename T>
hipError_t norm_back(const NormBackArgs& a, hipStream_t s) {
  if (a.n <= 128) return norm_back_as<T, 16, 1, 256>(a, s);
  if (a.n <= 512) return norm_back_as<T, 64, 1, 256>(a, s);
  if (a.n <= 1024) return norm_back_as<T, 64, 2, 256>(a, s);
  if (a.n <= 2048) return norm_back_as<T, 256, 1, 512>(a, s);
  if (a.n <= 4096) return norm_back_as<T, 512, 1, 1024>(a, s);
  if (a.n <= 8192) return norm_back_as<T, 1024, 1, 1024>(a, s);
  if (a.n <= kBackMost) return norm_back_as<T, 1024, 2, 1024>(a, s);
  for (long long r = 0; r < a.m; r += kMostGroups) {
    NormBackArgs b = a;
    b.m = (int)(a.m - r < kMostGroups ? a.m - r : kMostGroups);
    b.X = rows_on<T>(b.X, r, b.ldx);
    b.dY = rows_on<T>(b.dY, r, b.ldy);
    b.R = rows_on<T>(b.R, r, b.ldr);
    b.dX = rows_on<T>(b.dX, r, b.ldd);
    b.mean = rows_on<float>(b.mean, r, 1);
    b.rstd = rows_on<float>(b.rstd, r, 1);
    const hipError_t e = launch(&norm_back_long_kernel<T>, dim3((unsigned)b.m), 1024, b, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T>
hipError_t norm_sums(const NormBackArgs& a, hipStream_t s) {
  return launch(&norm_sums_kernel<T>, dim3((unsigned)((a.n + 511LL) / 512 * a.groups)), 256, a, s);
}

template <typename T>
hipError_t norm_columns(const NormColumnArgs& a, hipStream_t s) {
  const long long columns = (a.n + 63LL) / 64;
  return launch(&norm_columns_kernel<T>, dim3((unsigned)(columns < 65536 ? columns : 65536), 2), 1024,
                a, s);
}

template <typename T>
const NormOps& ops() {
  static const NormOps o = {&norm<T>, &norm_back<T>, &norm_sums<T>, &norm_columns<T>};
  return o;
}

}  // namespace

const NormOps& norm_ops(int dtype) {
  return dtype == PGEMM_F32 ? ops<float>() : dtype == PGEMM_F16 ? ops<_Float16>() : ops<__bf16>();
}

}  // namespace blocks
}  // namespace pgemm
