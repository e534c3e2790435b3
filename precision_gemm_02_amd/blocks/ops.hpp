// Internal: what the block operators' entry points launch.
#pragma once

#include <hip/hip_runtime.h>

#include "norm.hpp"

namespace pgemm {
namespace blocks {

struct NormOps {
  hipError_t (*norm)(const NormArgs& a, hipStream_t s);
  // dX, and with a.partial (rows of at most kSumMost) the column sums
  hipError_t (*norm_back)(const NormBackArgs& a, hipStream_t s);
  // the column sums alone
  hipError_t (*norm_sums)(const NormBackArgs& a, hipStream_t s);
  hipError_t (*norm_columns)(const NormColumnArgs& a, hipStream_t s);
};
const NormOps& norm_ops(int dtype);

}  // namespace blocks
}  // namespace pgemm
