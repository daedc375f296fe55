// Mixture of experts: f16.
#include "moe_launch.hpp"

namespace pgemm {

pgemm_status moe_f16(const MoeCall &c) { return launch_detail::moe_layer<_Float16>(c); }

}  // namespace pgemm
