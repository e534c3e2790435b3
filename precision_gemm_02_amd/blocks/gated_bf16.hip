// Gated products in bf16.
#include "gated_impl.hpp"

namespace pgemm {
namespace blocks {

const GateOps& gate_ops_bf16() { return ops<__bf16>(); }

}  // namespace blocks
}  // namespace pgemm
