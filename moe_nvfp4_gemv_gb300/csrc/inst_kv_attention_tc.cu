// The attention kernel on the 5th-generation tensor core.
#include <algorithm>

#include "decode_launch.h"
#include "k_kv_attention_tc.cuh"
#include "launch.h"

namespace fp4 {

template <bool kSinks, class P>
static cudaError_t tc_typed(const P& p, int sms, int pdl, cudaStream_t stream) {
  using C = AttnTc;
  static int configured[64];
  const size_t smem = C::smem(p.B);
  cudaError_t e = configure_kernel(kv_attention_tc_kernel<kSinks>, configured, smem, 1);
  if (e != cudaSuccess) return e;
  // no more CTAs than the table's width could give a tile
  const int64_t tiles = ((static_cast<int64_t>(p.max_blocks) << p.block_log2) + C::kTile - 1) / C::kTile;
  const int64_t ctas = std::min<int64_t>(sms, static_cast<int64_t>(p.B) * p.kv_heads * p.row_tiles * tiles);
  P q = p;
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
  return cudaLaunchKernelEx(&lc, kv_attention_tc_kernel<kSinks>, q);
}

cudaError_t launch_kv_attention_tc(const KvAttnTcParams& p, int sms, int pdl, cudaStream_t stream) {
  return tc_typed<false>(p, sms, pdl, stream);
}

cudaError_t launch_kv_attention_tc_sinks(const KvAttnSinksParams& p, const CUtensorMap& k_map, const CUtensorMap& v_map,
                                         int skip_tile, int sms, int pdl, cudaStream_t stream) {
  KvAttnTcSinksParams q = {};
  static_cast<KvAttnSinksParams&>(q) = p;
  q.k_map = k_map;
  q.v_map = v_map;
  q.skip_tile = skip_tile;
  return tc_typed<true>(q, sms, pdl, stream);
}

}  // namespace fp4
