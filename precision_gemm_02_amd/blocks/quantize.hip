// The launches of the quantization, for each type.
#include "../layers/launch.hpp"
#include "ops.hpp"
#include "pgemm_layers.h"

namespace pgemm {
namespace blocks {
namespace {

using layers::launch;

// Workgroups of one launch (which has less than 2^32 threads).
constexpr long long kMost = 1 << 22;

template <typename T, int F>
hipError_t quantize(const QuantizeArgs& all, bool outer, hipStream_t s) {
  QuantizeArgs a = all;
  if (!outer && !all.together) {
    // as many blocks beside each other as leave less than an eighth of them without work
    a.beside = 4;
    while (a.beside > 0 && (-all.blocks & ((1 << a.beside) - 1)) > all.blocks / 8) --a.beside;
    const long long across = (all.blocks + (1 << a.beside) - 1) >> a.beside;
    const long long high = (16 >> a.beside) * kRowsAhead, total = (all.r + high - 1) / high;
    const long long most = kMost / across < 65535 ? kMost / across : 65535;
    for (a.first = 0; a.first < total; a.first += most) {
      const dim3 grid((unsigned)across, (unsigned)(total - a.first < most ? total - a.first : most));
      const hipError_t e = launch(&quantize_rows_kernel<T, F>, grid, 256, a, s);
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
  const long long total = ((long long)all.r + kScaleBlock - 1) / kScaleBlock * all.blocks;
  for (long long at = 0; at < total; at += kMost) {
    a.first = at;
    const dim3 grid((unsigned)(total - at < kMost ? total - at : kMost));
    const hipError_t e =
        !outer         ? launch(&quantize_blocks_kernel<T, F>, grid, 256, a, s)
        : a.together   ? launch(&quantize_outer_kernel<T, F, true>, grid, 256, a, s)
                       : launch(&quantize_outer_kernel<T, F, false>, grid, 256, a, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T>
hipError_t quantize_as(const QuantizeArgs& a, int type, bool outer, hipStream_t s) {
  return type == kE4M3 ? quantize<T, kE4M3>(a, outer, s) : quantize<T, kE5M2>(a, outer, s);
}

}  // namespace

hipError_t quantize_op(const QuantizeArgs& a, int dtype, int type, bool outer, hipStream_t s) {
  if (dtype == PGEMM_F32) return quantize_as<float>(a, type, outer, s);
  if (dtype == PGEMM_F16) return quantize_as<_Float16>(a, type, outer, s);
  return quantize_as<__bf16>(a, type, outer, s);
}

}  // namespace blocks
}  // namespace pgemm
