// Launcher of the cache's append kernel.
#include "decode_launch.h"

namespace fp4 {

using AppendKernel = void (*)(KvAppendParams);

template <int kThreads, int kH>
static AppendKernel append_kernel(bool int8, bool f16) {
  return int8 ? f16 ? kv_append_kernel<true, true, kThreads, kH> : kv_append_kernel<true, false, kThreads, kH>
         : f16 ? kv_append_kernel<false, true, kThreads, kH>
               : kv_append_kernel<false, false, kThreads, kH>;
}

cudaError_t launch_kv_append(const KvAppendParams& p, int int8, int f16, int pdl, cudaStream_t stream) {
  // threads that hold a head's values of a page, kAppendChunks chunks of 8 each at most; with fewer chunks to a head
  // (small pages, or at most `uniform` tokens) several heads
  const int values = p.dim << p.block_log2, per = kAppendChunks * 8;
  const int threads = values <= 128 * per ? 128 : values <= 256 * per ? 256 : 512;
  KvAppendParams q = p;
  q.step = threads / (p.dim / 8);
  q.chunk_magic = (65536 + p.dim / 8 - 1) / (p.dim / 8);  // (exact for the threads there are)
  const int block = 1 << p.block_log2, tokens = p.cu || p.uniform > block ? block : p.uniform;
  const int slots = (tokens + q.step - 1) / q.step;
  int heads = 1;
  while (threads == 128 && 2 * heads * slots <= kAppendChunks && heads < p.heads) heads *= 2;
  const int64_t units = p.cu ? (p.T >> p.block_log2) + 2ll * p.B
                             : static_cast<int64_t>(p.B) * (((p.uniform + block - 2) >> p.block_log2) + 1);
  AppendKernel kernel;
  if (threads == 512) kernel = append_kernel<512, 1>(int8, f16);
  else if (threads == 256) kernel = append_kernel<256, 1>(int8, f16);
  else
    kernel = heads == 1   ? append_kernel<128, 1>(int8, f16)
             : heads == 2 ? append_kernel<128, 2>(int8, f16)
             : heads == 4 ? append_kernel<128, 4>(int8, f16)
                          : append_kernel<128, 8>(int8, f16);
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(static_cast<unsigned>(units), static_cast<unsigned>((p.heads + heads - 1) / heads), 2);
  lc.blockDim = dim3(threads, 1, 1);
  lc.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = &attr;
  lc.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&lc, kernel, q);
}

}  // namespace fp4
