// Gated products in fp32.
#include "gated_impl.hpp"

namespace pgemm {
namespace blocks {

const GateOps& gate_ops_f32() { return ops<float>(); }

}  // namespace blocks
}  // namespace pgemm
