// The cross entropy over a vocabulary and its gradients: bf16.
#include "xent_launch.hpp"

namespace pgemm {

pgemm_status xent_bf16(const XentCall &c) { return launch_detail::xent_forward<__bf16>(c); }
pgemm_status xent_bwd_bf16(const XentCall &c) { return launch_detail::xent_backward<__bf16>(c); }

}  // namespace pgemm
