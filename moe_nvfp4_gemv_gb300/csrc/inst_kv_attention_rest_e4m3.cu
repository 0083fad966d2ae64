// The attention kernel behind a beginning that is taken, over E4M3 codes, and the
// choice by format.
#include "inst_kv_attention_more.inc"

namespace fp4 {

cudaError_t launch_kv_attention_rest_int8(const KvAttnRestParams& p, int dim, int row_units, int sms, int pdl,
                                           cudaStream_t stream);

cudaError_t launch_kv_attention_rest(const KvAttnRestParams& p, int dim, int int8, int row_units, int sms, int pdl,
                                      cudaStream_t stream) {
  return int8 ? launch_kv_attention_rest_int8(p, dim, row_units, sms, pdl, stream)
              : more_format<kAttnRest, false>(p, dim, row_units, sms, pdl, stream);
}

}  // namespace fp4
