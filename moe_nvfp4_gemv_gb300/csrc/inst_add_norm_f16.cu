// The residual and norm kernel for f16.
#include "inst_add_norm.inc"

namespace fp4 {

cudaError_t launch_add_norm_f16(const AddNormParams& p, int part, int sms, int pdl, cudaStream_t stream) {
  return add_norm_half<true>(p, part, sms, pdl, stream);
}

}  // namespace fp4
