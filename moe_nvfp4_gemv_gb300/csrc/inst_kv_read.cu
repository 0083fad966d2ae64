// Launcher of the cache's read kernel.
#include <algorithm>

#include "decode_launch.h"
#include "k_kv_read.cuh"

namespace fp4 {

template <bool kInt8, int kOut>
static cudaError_t read_typed(const KvReadParams& p, const cudaLaunchConfig_t& lc) {
  return cudaLaunchKernelEx(&lc, kv_read_kernel<kInt8, kOut>, p);
}

cudaError_t launch_kv_read(const KvReadParams& p, int int8, int dtype, int sms, int pdl, cudaStream_t stream) {
  KvReadParams q = p;
  const int chunks = p.dim / (dtype == 2 ? 4 : 8);
  q.step = kReadThreads / chunks;
  q.chunk_magic = (65536 + chunks - 1) / chunks;  // (exact for the threads there are)
  const int block = 1 << p.block_log2;
  const int64_t units = p.cu ? (p.T >> p.block_log2) + 2ll * p.B
                             : static_cast<int64_t>(p.B) * (((p.uniform + block - 2) >> p.block_log2) + 1);
  // all heads in a CTA, as long as that leaves 64 CTAs for every SM (40001 tokens in five prompts, INT8: with 8 48.9 us, 24
  // 40.8, 64 39.9; with 64 and 256 threads 52, half the loads under way 40.8)
  int groups = 1;
  while (groups < p.heads && units * 2 * groups < 64ll * sms) groups *= 2;
  q.heads_per = (p.heads + groups - 1) / groups;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(static_cast<unsigned>(units), static_cast<unsigned>((p.heads + q.heads_per - 1) / q.heads_per), 2);
  lc.blockDim = dim3(kReadThreads, 1, 1);
  lc.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = &attr;
  lc.numAttrs = pdl ? 1 : 0;
  if (int8) return dtype == 2 ? read_typed<true, 2>(q, lc) : dtype == 1 ? read_typed<true, 1>(q, lc) : read_typed<true, 0>(q, lc);
  return dtype == 2 ? read_typed<false, 2>(q, lc) : dtype == 1 ? read_typed<false, 1>(q, lc) : read_typed<false, 0>(q, lc);
}

}  // namespace fp4
