// Launcher of the cache's append kernel.
#include "decode_launch.h"

namespace fp4 {

static auto append_kernel(bool int8, bool f16, bool large) -> void (*)(KvAppendParams) {
  if (large)
    return int8 ? f16 ? kv_append_kernel<true, true, 512> : kv_append_kernel<true, false, 512>
           : f16 ? kv_append_kernel<false, true, 512>
                 : kv_append_kernel<false, false, 512>;
  return int8 ? f16 ? kv_append_kernel<true, true, 128> : kv_append_kernel<true, false, 128>
         : f16 ? kv_append_kernel<false, true, 128>
               : kv_append_kernel<false, false, 128>;
}

cudaError_t launch_kv_append(const KvAppendParams& p, int int8, int f16, int pdl, cudaStream_t stream) {
  // enough threads to hold a full page of one head, kAppendChunks chunks of 8 each
  const int threads = p.block * p.dim <= 128 * kAppendChunks * 8 ? 128 : 512;
  const int64_t units = p.cu ? p.T / p.block + 2ll * p.B
                             : static_cast<int64_t>(p.B) * ((p.uniform + p.block - 2) / p.block + 1);
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(static_cast<unsigned>(units), static_cast<unsigned>(p.heads), 2);
  lc.blockDim = dim3(threads, 1, 1);
  lc.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = &attr;
  lc.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&lc, append_kernel(int8, f16, threads == 512), p);
}

}  // namespace fp4
