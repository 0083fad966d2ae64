// The attention kernel with first tokens that stay visible, over E4M3 codes, and the
// choice by format.
#include "inst_kv_attention_more.inc"

namespace fp4 {

cudaError_t launch_kv_attention_sinks_int8(const KvAttnSinksParams& p, int dim, int row_units, int sms, int pdl,
                                           cudaStream_t stream);

cudaError_t launch_kv_attention_sinks(const KvAttnSinksParams& p, int dim, int int8, int row_units, int sms, int pdl,
                                      cudaStream_t stream) {
  return int8 ? launch_kv_attention_sinks_int8(p, dim, row_units, sms, pdl, stream)
              : more_format<kAttnSinks, false>(p, dim, row_units, sms, pdl, stream);
}

}  // namespace fp4
