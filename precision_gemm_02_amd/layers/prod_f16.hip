// Layer kernels for f16.
#include "launch_impl.hpp"

namespace pgemm {
namespace layers {

const TypeOps& ops_f16() { return type_ops<_Float16>(); }

}  // namespace layers
}  // namespace pgemm
