// The attention kernel with leading strips over INT8 codes.
#include "inst_kv_attention_more.inc"

namespace fp4 {

cudaError_t launch_kv_attention_more_int8(const KvAttnMoreParams& p, int dim, int row_units, int sms, int pdl,
                                          cudaStream_t stream) {
  return more_format<true>(p, dim, row_units, sms, pdl, stream);
}

}  // namespace fp4
