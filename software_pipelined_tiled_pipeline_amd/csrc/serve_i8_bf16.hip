// 8-bit products and the quantization of rows: bf16.
#include "i8_launch.hpp"

namespace pgemm {

pgemm_status quant_i8_bf16(const QuantCall &c) {
  return launch_detail::quant_rows<__bf16>(c.x, c.q, c.scale, c.M, c.K, c.stream);
}
pgemm_status i8_bf16(const I8Call &c) { return launch_detail::i8_product<__bf16>(c); }

}  // namespace pgemm
