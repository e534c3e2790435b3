// 8-bit products whose left operand is e4m3, with 16-bit results.
#include "fp8_impl.hpp"

namespace pgemm {
namespace blocks {

hipError_t prod8_e4m3(const Prod8Args& a, int w_type, int kernel, int loading, hipStream_t s) {
  return prod8_of<kE4M3, false>(a, w_type, kernel, loading, s);
}

}  // namespace blocks
}  // namespace pgemm
