// 8-bit products whose left operand is e5m2, with fp32 results.
#include "fp8_impl.hpp"

namespace pgemm {
namespace blocks {

hipError_t prod8_e5m2_wide(const Prod8Args& a, int w_type, int kernel, int loading, hipStream_t s) {
  return prod8_of<kE5M2, true>(a, w_type, kernel, loading, s);
}

}  // namespace blocks
}  // namespace pgemm
