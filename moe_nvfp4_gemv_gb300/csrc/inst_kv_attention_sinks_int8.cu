// The attention kernel with first tokens that stay visible, over INT8 codes.
#include "inst_kv_attention_more.inc"

namespace fp4 {

cudaError_t launch_kv_attention_sinks_int8(const KvAttnSinksParams& p, int dim, int row_units, int sms, int pdl,
                                           cudaStream_t stream) {
  return more_format<kAttnSinks, true>(p, dim, row_units, sms, pdl, stream);
}

}  // namespace fp4
