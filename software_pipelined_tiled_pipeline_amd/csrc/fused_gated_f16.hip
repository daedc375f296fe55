// The gated block and its gradients: f16.
#include "gated_launch.hpp"

namespace pgemm {

pgemm_status gated_f16(const GatedCall &c) { return launch_detail::gated_forward<_Float16>(c); }
pgemm_status gated_bwd_f16(const GatedCall &c) { return launch_detail::gated_backward<_Float16>(c); }

}  // namespace pgemm
