// Gated products in fp16.
#include "gated_impl.hpp"

namespace pgemm {
namespace blocks {

const GateOps& gate_ops_f16() { return ops<_Float16>(); }

}  // namespace blocks
}  // namespace pgemm
