// The gated block and its gradients: bf16.
#include "gated_launch.hpp"

namespace pgemm {

pgemm_status gated_bf16(const GatedCall &c) { return launch_detail::gated_forward<__bf16>(c); }
pgemm_status gated_bwd_bf16(const GatedCall &c) { return launch_detail::gated_backward<__bf16>(c); }

}  // namespace pgemm
