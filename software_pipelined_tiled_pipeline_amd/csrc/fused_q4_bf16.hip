// Products with 4-bit weights: bf16 activations.
#include "q4_launch.hpp"

namespace pgemm {

pgemm_status q4_bf16(const Q4Call &c) { return launch_detail::q4_product<__bf16>(c); }

}  // namespace pgemm
