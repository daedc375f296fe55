// Mixture of experts: bf16.
#include "moe_launch.hpp"

namespace pgemm {

pgemm_status moe_bf16(const MoeCall &c) { return launch_detail::moe_layer<__bf16>(c); }

}  // namespace pgemm
