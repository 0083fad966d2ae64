// The residual and norm kernel for bf16, and the choice of the type.
#include "inst_add_norm.inc"

namespace fp4 {

cudaError_t launch_add_norm_f16(const AddNormParams& p, int part, int sms, int pdl, cudaStream_t stream);

cudaError_t launch_add_norm(const AddNormParams& p, int f16, int part, int sms, int pdl, cudaStream_t stream) {
  return f16 ? launch_add_norm_f16(p, part, sms, pdl, stream) : add_norm_half<false>(p, part, sms, pdl, stream);
}

}  // namespace fp4
