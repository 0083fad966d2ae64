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

// A token on a warp: the shortest chain.  On 8 lanes, with fewer instructions
// per token, where there are so many tokens that issue is what counts, and up
// to 64 experts.  Warp against 8 lanes, bf16, 60 experts, top 4, us: 2432 tokens
// 2.0 / 2.6, 4864 2.7 / 3.5, 20011 6.8 / 5.5; 16 lanes for 128 experts, top 8:
// 2.9 / 3.4, 4.0 / 4.4, 12.0 / 12.3.  Groups have to be whole lanes of 8 then
// (20011 tokens of 64 experts in 8 groups: 11.7 / 8.8).
template <typename T>
cudaError_t route_typed(const RouteParams& p, int sms, int pdl, cudaStream_t stream) {
  RouteParams q = p;
  const int size = p.E / p.n_group;  // of a group
  // Groups at lanes of their own, where 16 experts to a lane do; else they lie across lanes and are gone through one by
  // one.  Across / own, us: 1372 tokens, 8 groups of 30 7.1 / 4.2; 24094 tokens, 8 of 9, two keys each 45 / 29.
  auto group_layout = [&]() -> bool {
    int run = 32;  // lanes to a group
    while (run > 0 && run * p.n_group > 32) run /= 2;
    if (p.n_group == 1 || (size + run - 1) / run > 16) return false;
    q.group_lanes = run;
    q.lane_experts = (size + run - 1) / run;
    return true;
  };
  int lanes = 32;
  void (*kernel)(RouteParams);
  if (p.M >= 64 * sms && p.E <= 64 && (p.n_group == 1 || (size % 8 == 0 && (size & (size - 1)) == 0))) {
    kernel = moe_route_kernel<T, 8, 8>;
    lanes = 8;
    q.group_lanes = size / 8;
  } else {
    const int slots = group_layout() ? q.lane_experts : (p.E + 31) / 32;
    kernel = slots <= 1   ? moe_route_kernel<T, 32, 1>
             : slots <= 2 ? moe_route_kernel<T, 32, 2>
             : slots <= 4 ? moe_route_kernel<T, 32, 4>
             : slots <= 8 ? moe_route_kernel<T, 32, 8>
                          : moe_route_kernel<T, 32, 16>;
  }
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(p.M) * lanes + kRouteThreads - 1) / kRouteThreads);
  return launch_simple<RouteParams>(kernel, grid, kRouteThreads, 1, pdl, stream, q);
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
  // A cluster per row while the rows alone leave CTAs idle and a slice keeps 16 bytes for every thread.  Up to 2, 4 (as
  // here) or 8 CTAs per SM, us: 64 rows of 100001 fp32 10.6 / 9.4 / 9.4, 128 of 128003 bf16 13.1 / 12.7 / 15.8, 300 of
  // 32000 11.5 / 10.5 / 15.2.  Clusters of 4, 8 or 16 for one row of 128003: 6.2 / 5.6 / 9.
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
