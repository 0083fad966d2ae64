// The attention kernel over INT8 codes.
#include "inst_kv_attention.inc"

namespace fp4 {

cudaError_t launch_kv_attention_int8(const KvAttnParams& p, int dim, int rows_per_tile, int sms, int pdl,
                                     cudaStream_t stream) {
  return attn_format<true>(p, dim, rows_per_tile, sms, pdl, stream);
}

}  // namespace fp4
