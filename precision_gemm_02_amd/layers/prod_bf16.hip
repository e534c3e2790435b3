// Layer kernels for bf16.
#include "launch_impl.hpp"

namespace pgemm {
namespace layers {

const TypeOps& ops_bf16() { return type_ops<__bf16>(); }

}  // namespace layers
}  // namespace pgemm
