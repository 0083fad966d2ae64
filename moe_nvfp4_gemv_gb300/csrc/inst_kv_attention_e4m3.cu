// The attention kernel over E4M3 codes, and the choice by format.
#include "inst_kv_attention.inc"

namespace fp4 {

cudaError_t launch_kv_attention_int8(const KvAttnParams& p, int dim, int row_units, int sms, int pdl,
                                     cudaStream_t stream);

int kv_attention_max_ctas(int sms) { return 2 * sms; }

cudaError_t launch_kv_attention(const KvAttnParams& p, int dim, int int8, int row_units, int sms, int pdl,
                                cudaStream_t stream) {
  return int8 ? launch_kv_attention_int8(p, dim, row_units, sms, pdl, stream)
              : attn_format<false>(p, dim, row_units, sms, pdl, stream);
}

}  // namespace fp4
