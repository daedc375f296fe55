// The choice of a token from logits of either type.
#include "sample.hpp"

namespace pgemm {

pgemm_status sample_f16(const SampleCall &c) { return launch_detail::sample_rows<_Float16>(c); }
pgemm_status sample_bf16(const SampleCall &c) { return launch_detail::sample_rows<__bf16>(c); }

}  // namespace pgemm
