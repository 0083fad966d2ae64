// Launchers of the routing and log-probability kernels.
#include "decode_launch.h"

namespace fp4 {

namespace {

template <typename Params>
cudaError_t launch_simple(void (*kernel)(Params), unsigned grid, unsigned threads, unsigned cluster, int pdl,
                          cudaStream_t stream, const Params& p) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(grid, 1, 1);
  lc.blockDim = dim3(threads, 1, 1);
  lc.stream = stream;
  cudaLaunchAttribute attrs[2];
  unsigned na = 0;
  if (cluster > 1) {
    attrs[na].id = cudaLaunchAttributeClusterDimension;
    attrs[na].val.clusterDim.x = cluster;
    attrs[na].val.clusterDim.y = 1;
    attrs[na].val.clusterDim.z = 1;
    ++na;
  }
  if (pdl) {
    attrs[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
  }
  lc.attrs = attrs;
  lc.numAttrs = na;
  return cudaLaunchKernelEx(&lc, kernel, p);
}

// A token on a warp (few tokens: the shortest chain), or on 8 or 16 lanes
// (many: fewer instructions per token).
template <typename T>
cudaError_t route_typed(const RouteParams& p, int sms, int pdl, cudaStream_t stream) {
  const bool many = p.M >= 16 * sms;
  int lanes = 32;
  void (*kernel)(RouteParams);
  if (many && p.E <= 64) {
    kernel = moe_route_kernel<T, 8, 8>;
    lanes = 8;
  } else if (many && p.E <= 128) {
    kernel = moe_route_kernel<T, 16, 8>;
    lanes = 16;
  } else {
    kernel = p.E <= 32    ? moe_route_kernel<T, 32, 1>
             : p.E <= 64  ? moe_route_kernel<T, 32, 2>
             : p.E <= 128 ? moe_route_kernel<T, 32, 4>
             : p.E <= 256 ? moe_route_kernel<T, 32, 8>
                          : moe_route_kernel<T, 32, 16>;
  }
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(p.M) * lanes + kRouteThreads - 1) / kRouteThreads);
  return launch_simple<RouteParams>(kernel, grid, kRouteThreads, 1, pdl, stream, p);
}

}  // namespace

cudaError_t launch_moe_route(const RouteParams& p, int dtype, int sms, int pdl, cudaStream_t stream) {
  switch (dtype) {
    case 0: return route_typed<__nv_bfloat16>(p, sms, pdl, stream);
    case 1: return route_typed<__half>(p, sms, pdl, stream);
    default: return route_typed<float>(p, sms, pdl, stream);
  }
}

template <typename T>
static cudaError_t logprobs_typed(const LogprobParams& p, int rows, int sms, int pdl, cudaStream_t stream) {
  auto kernel = token_logprobs_kernel<T>;
  // a cluster per row while the rows alone leave CTAs idle and a slice keeps 16 bytes for every thread
  unsigned c = 1;
  while (c < kLpMaxCluster && static_cast<int64_t>(rows) * c * 2 <= 4 * sms &&
         static_cast<int64_t>(p.V) * static_cast<int>(sizeof(T)) / (2 * c) >= kLpThreads * 16)
    c *= 2;
  return launch_simple<LogprobParams>(kernel, static_cast<unsigned>(rows) * c, kLpThreads, c, pdl, stream, p);
}

cudaError_t launch_token_logprobs(const LogprobParams& p, int dtype, int T, int sms, int pdl, cudaStream_t stream) {
  switch (dtype) {
    case 0: return logprobs_typed<__nv_bfloat16>(p, T, sms, pdl, stream);
    case 1: return logprobs_typed<__half>(p, T, sms, pdl, stream);
    default: return logprobs_typed<float>(p, T, sms, pdl, stream);
  }
}

}  // namespace fp4
