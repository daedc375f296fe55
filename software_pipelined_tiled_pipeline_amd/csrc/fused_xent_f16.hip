// The cross entropy over a vocabulary and its gradients: f16.
#include "xent_launch.hpp"

namespace pgemm {

pgemm_status xent_f16(const XentCall &c) { return launch_detail::xent_forward<_Float16>(c); }
pgemm_status xent_bwd_f16(const XentCall &c) { return launch_detail::xent_backward<_Float16>(c); }

}  // namespace pgemm
