// The attention kernel over E4M3 codes, and the choice by format.
#include "inst_kv_attention.inc"

namespace fp4 {

cudaError_t launch_kv_attention_int8(const KvAttnParams& p, int dim, int rows_per_tile, int sms, int pdl,
                                     cudaStream_t stream);

int kv_attention_max_ctas(int sms) { return 2 * sms; }

cudaError_t launch_kv_attention(const KvAttnParams& p, int dim, int int8, int rows_per_tile, int sms, int pdl,
                                cudaStream_t stream) {
  return int8 ? launch_kv_attention_int8(p, dim, rows_per_tile, sms, pdl, stream)
              : attn_format<false>(p, dim, rows_per_tile, sms, pdl, stream);
}

}  // namespace fp4
