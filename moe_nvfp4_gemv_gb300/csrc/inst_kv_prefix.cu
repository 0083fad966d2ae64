// Launcher of the kernel for a beginning that sequences share.
#include "decode_launch.h"
#include "k_kv_prefix.cuh"
#include "launch.h"

namespace fp4 {

int kv_prefix_slots(int dim) { return dim == 256 ? PrefixCfg<256>::kSlots : PrefixCfg<128>::kSlots; }
int kv_prefix_tile(int dim) { return dim == 256 ? PrefixCfg<256>::kTile : PrefixCfg<128>::kTile; }

template <int kDim, bool kInt8>
static cudaError_t prefix_typed(const KvPrefixParams& p, int pdl, cudaStream_t stream) {
  using C = PrefixCfg<kDim>;
  auto kernel = kv_prefix_kernel<kDim, kInt8>;
  static int configured[64];
  cudaError_t e = configure_kernel(kernel, configured, C::kSmem, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(static_cast<unsigned>(p.line.ctas), 1, 1);
  lc.blockDim = dim3(C::kThreads, 1, 1);
  lc.dynamicSmemBytes = C::kSmem;
  lc.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = &attr;
  lc.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&lc, kernel, p);
}

cudaError_t launch_kv_prefix(const KvPrefixParams& p, int dim, int int8, int pdl, cudaStream_t stream) {
  switch (dim) {
    case 64: return int8 ? prefix_typed<64, true>(p, pdl, stream) : prefix_typed<64, false>(p, pdl, stream);
    case 96: return int8 ? prefix_typed<96, true>(p, pdl, stream) : prefix_typed<96, false>(p, pdl, stream);
    case 128: return int8 ? prefix_typed<128, true>(p, pdl, stream) : prefix_typed<128, false>(p, pdl, stream);
    default: return int8 ? prefix_typed<256, true>(p, pdl, stream) : prefix_typed<256, false>(p, pdl, stream);
  }
}

template <int kDim, int kWays>
static cudaError_t join_typed(const KvJoinParams& p, int64_t cells, int pdl, cudaStream_t stream) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(static_cast<unsigned>((cells * kWays + kJoinThreads - 1) / kJoinThreads), 1, 1);
  lc.blockDim = dim3(kJoinThreads, 1, 1);
  lc.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = &attr;
  lc.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&lc, kv_join_kernel<kDim, kWays>, p);
}

// Up to eight threads to a cell, as long as there are no more than 1024 to an SM.  28 rows on 4 KV heads of 256, 38 pieces
// of each: the call 55.2 us with one, 49.8 with eight.
template <int kDim>
static cudaError_t join_dim(const KvJoinParams& p, int sms, int pdl, cudaStream_t stream) {
  const int64_t cells = static_cast<int64_t>(p.B) * p.q_len * p.group * p.kv_heads * (kDim / 4), most = 1024ll * sms;
  if (8 * cells <= most) return join_typed<kDim, 8>(p, cells, pdl, stream);
  if (4 * cells <= most) return join_typed<kDim, 4>(p, cells, pdl, stream);
  if (2 * cells <= most) return join_typed<kDim, 2>(p, cells, pdl, stream);
  return join_typed<kDim, 1>(p, cells, pdl, stream);
}

cudaError_t launch_kv_join(const KvJoinParams& p, int dim, int sms, int pdl, cudaStream_t stream) {
  return dim == 64    ? join_dim<64>(p, sms, pdl, stream)
         : dim == 96  ? join_dim<96>(p, sms, pdl, stream)
         : dim == 128 ? join_dim<128>(p, sms, pdl, stream)
                      : join_dim<256>(p, sms, pdl, stream);
}

}  // namespace fp4
