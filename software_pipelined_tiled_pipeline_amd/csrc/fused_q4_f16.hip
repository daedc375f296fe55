// Products with 4-bit weights: f16 activations.
#include "q4_launch.hpp"

namespace pgemm {

pgemm_status q4_f16(const Q4Call &c) { return launch_detail::q4_product<_Float16>(c); }

}  // namespace pgemm
