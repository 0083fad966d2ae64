// The attention kernel over INT8 codes.
#include "inst_kv_attention.inc"

namespace fp4 {

cudaError_t launch_kv_attention_int8(const KvAttnParams& p, int dim, int row_units, int sms, int pdl,
                                     cudaStream_t stream) {
  return attn_format<true>(p, dim, row_units, sms, pdl, stream);
}

}  // namespace fp4
