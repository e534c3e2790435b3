// 8-bit products whose left operand is e4m3, with fp32 results.
#include "fp8_impl.hpp"

namespace pgemm {
namespace blocks {

hipError_t prod8_e4m3_wide(const Prod8Args& a, int w_type, int kernel, int loading, hipStream_t s) {
  return prod8_of<kE4M3, true>(a, w_type, kernel, loading, s);
}

}  // namespace blocks
}  // namespace pgemm
