// The attention kernel on the 5th-generation tensor core.
#include <algorithm>

#include "decode_launch.h"
#include "k_kv_attention_tc.cuh"
#include "launch.h"

namespace fp4 {

cudaError_t launch_kv_attention_tc(const KvAttnTcParams& p, int sms, int pdl, cudaStream_t stream) {
  using C = AttnTc;
  static int configured[64];
  const size_t smem = C::smem(p.B);
  cudaError_t e = configure_kernel(kv_attention_tc_kernel, configured, smem, 1);
  if (e != cudaSuccess) return e;
  // no more CTAs than the table's width could give a tile
  const int64_t tiles = ((static_cast<int64_t>(p.max_blocks) << p.block_log2) + C::kTile - 1) / C::kTile;
  const int64_t ctas = std::min<int64_t>(sms, static_cast<int64_t>(p.B) * p.kv_heads * p.row_tiles * tiles);
  KvAttnTcParams q = p;
  q.inv_ctas = 1.0f / static_cast<float>(ctas);
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
  lc.blockDim = dim3(C::kThreads, 1, 1);
  lc.dynamicSmemBytes = smem;
  lc.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = &attr;
  lc.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&lc, kv_attention_tc_kernel, q);
}

}  // namespace fp4
