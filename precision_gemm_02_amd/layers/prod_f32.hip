// Layer kernels for f32.
#include "launch_impl.hpp"

namespace pgemm {
namespace layers {

const TypeOps& ops_f32() { return type_ops<float>(); }

}  // namespace layers
}  // namespace pgemm
