// Launcher of the residual and norm kernel.
#include "decode_launch.h"
#include "k_add_norm.cuh"

namespace fp4 {

template <bool kF16, bool kVec, int kRow, int kChunks>
static cudaError_t add_norm_typed(const AddNormParams& p, int pdl, cudaStream_t stream) {
  constexpr int kThreads = kRow < 256 ? 256 : kRow, kRows = kThreads / kRow;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(p.M) + kRows - 1) / kRows), 1, 1);
  lc.blockDim = dim3(kThreads, 1, 1);
  lc.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = &attr;
  lc.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&lc, add_norm_kernel<kF16, kVec, kRow, kChunks>, p);
}

// The fewest threads that hold a token in one chunk each; above 1024 threads more chunks.
template <bool kF16, bool kVec>
static cudaError_t add_norm_width(const AddNormParams& p, int pdl, cudaStream_t stream) {
  if (p.H <= 256) return add_norm_typed<kF16, kVec, 32, 1>(p, pdl, stream);
  if (p.H <= 1024) return add_norm_typed<kF16, kVec, 128, 1>(p, pdl, stream);
  if (p.H <= 2048) return add_norm_typed<kF16, kVec, 256, 1>(p, pdl, stream);
  if (p.H <= 4096) return add_norm_typed<kF16, kVec, 512, 1>(p, pdl, stream);
  if (p.H <= 8192) return add_norm_typed<kF16, kVec, 1024, 1>(p, pdl, stream);
  if (p.H <= 16384) return add_norm_typed<kF16, kVec, 1024, 2>(p, pdl, stream);
  return add_norm_typed<kF16, kVec, 1024, 4>(p, pdl, stream);
}

cudaError_t launch_add_norm(const AddNormParams& p, int f16, int vec, int pdl, cudaStream_t stream) {
  if (vec) return f16 ? add_norm_width<true, true>(p, pdl, stream) : add_norm_width<false, true>(p, pdl, stream);
  return f16 ? add_norm_width<true, false>(p, pdl, stream) : add_norm_width<false, false>(p, pdl, stream);
}

}  // namespace fp4
