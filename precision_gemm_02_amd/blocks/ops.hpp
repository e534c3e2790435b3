// Internal: what the block operators' entry points launch.
#pragma once

#include <hip/hip_runtime.h>

#include "fp8.hpp"
#include "gated.hpp"
#include "norm.hpp"
#include "quantize.hpp"

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

// X of `dtype`, to 8 bits of `type` (Fp8); outer: X's columns are contiguous.
hipError_t quantize_op(const QuantizeArgs& a, int dtype, int type, bool outer, hipStream_t s);

// The product of a plan (and the sum of its splits), A of the type named, W of w_type,
// for results of 16 bits and (wide) of 32, which have no tiles of 256 x 256.  loading: kDirect,
// kThrough, or kWhole where prod8_whole_kernel takes its tiles (16-bit results).
constexpr int kWhole = 3;
typedef hipError_t (*Prod8)(const Prod8Args& a, int w_type, int kernel, int loading, hipStream_t s);
hipError_t prod8_e4m3(const Prod8Args& a, int w_type, int kernel, int loading, hipStream_t s);
hipError_t prod8_e5m2(const Prod8Args& a, int w_type, int kernel, int loading, hipStream_t s);
hipError_t prod8_e4m3_wide(const Prod8Args& a, int w_type, int kernel, int loading, hipStream_t s);
hipError_t prod8_e5m2_wide(const Prod8Args& a, int w_type, int kernel, int loading, hipStream_t s);

struct GateOps {
  // a gated product (kColumns), or dX of one (kHalves), and the sum of its splits; whole: by
  // pair_whole_kernel
  hipError_t (*pair)(const PairArgs& a, int lb, int pair, int kernel, int loading, bool whole,
                     hipStream_t s);
  // one or two products of outer-order operands (kApart), whole
  hipError_t (*apart)(const PairArgs& a, int kernel, hipStream_t s);
  hipError_t (*slope)(const GateSlopeArgs& a, bool sums32, hipStream_t s);
  hipError_t (*pad)(const PadRowsArgs& a, int count, hipStream_t s);
};
const GateOps& gate_ops_f32();
const GateOps& gate_ops_f16();
const GateOps& gate_ops_bf16();
inline const GateOps& gate_ops(int dtype) {
  return dtype == 0 ? gate_ops_f32() : dtype == 1 ? gate_ops_f16() : gate_ops_bf16();
}

}  // namespace blocks
}  // namespace pgemm
