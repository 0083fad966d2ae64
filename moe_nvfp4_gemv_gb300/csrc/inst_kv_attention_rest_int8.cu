// The attention kernel behind a beginning that is taken, over INT8 codes.
#include "inst_kv_attention_more.inc"

namespace fp4 {

cudaError_t launch_kv_attention_rest_int8(const KvAttnRestParams& p, int dim, int row_units, int sms, int pdl,
                                           cudaStream_t stream) {
  return more_format<kAttnRest, true>(p, dim, row_units, sms, pdl, stream);
}

}  // namespace fp4
