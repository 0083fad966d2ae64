// Launcher of the residual and norm kernel.
#include "decode_launch.h"
#include "k_add_norm.cuh"

namespace fp4 {

template <bool kF16, bool kVec, bool kX32, int kRow, int kChunks>
static cudaError_t add_norm_typed(const AddNormParams& p, int pdl, cudaStream_t stream) {
  constexpr int kThreads = norm_threads(kRow), kRows = kThreads / kRow;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(p.M) + kRows - 1) / kRows), 1, 1);
  lc.blockDim = dim3(kThreads, 1, 1);
  lc.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = &attr;
  lc.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&lc, add_norm_kernel<kF16, kVec, kX32, kRow, kChunks>, p);
}

// As many tokens as SMs hold at once with a chunk to a thread (1024 threads): that, the shortest chain.  More: two chunks
// each, so that a thread has twice the loads under way and an SM holds twice the tokens.  One / two chunks, us: 300 tokens
// of 4096 3.0 / 3.7, 450 5.1 / 3.8; 608 of 2048 3.0 / 3.5; 1 of 4096 2.4 / 2.8.
template <bool kF16, bool kVec, bool kX32>
static cudaError_t add_norm_width(const AddNormParams& p, int sms, int pdl, cudaStream_t stream) {
  const int threads = p.H <= 1024 ? 128 : p.H <= 2048 ? 256 : p.H <= 4096 ? 512 : 1024;
  const bool many = static_cast<int64_t>(p.M) * threads > 1024ll * sms;
  if (p.H <= 64) return add_norm_typed<kF16, kVec, kX32, 8, 1>(p, pdl, stream);
  if (p.H <= 128) return add_norm_typed<kF16, kVec, kX32, 16, 1>(p, pdl, stream);
  if (p.H <= 256) return add_norm_typed<kF16, kVec, kX32, 32, 1>(p, pdl, stream);
  if (many) {
    if (p.H <= 512) return add_norm_typed<kF16, kVec, kX32, 32, 2>(p, pdl, stream);
    if (p.H <= 1024) return add_norm_typed<kF16, kVec, kX32, 64, 2>(p, pdl, stream);
    if (p.H <= 2048) return add_norm_typed<kF16, kVec, kX32, 128, 2>(p, pdl, stream);
    if (p.H <= 4096) return add_norm_typed<kF16, kVec, kX32, 256, 2>(p, pdl, stream);
    if (p.H <= 5120) return add_norm_typed<kF16, kVec, kX32, 320, 2>(p, pdl, stream);
    if (p.H <= 6144) return add_norm_typed<kF16, kVec, kX32, 384, 2>(p, pdl, stream);
    if (p.H <= 8192) return add_norm_typed<kF16, kVec, kX32, 512, 2>(p, pdl, stream);
    if (p.H <= 10240) return add_norm_typed<kF16, kVec, kX32, 320, 4>(p, pdl, stream);
    if (p.H <= 16384) return add_norm_typed<kF16, kVec, kX32, 512, 4>(p, pdl, stream);
  }
  if (p.H <= 1024) return add_norm_typed<kF16, kVec, kX32, 128, 1>(p, pdl, stream);
  if (p.H <= 2048) return add_norm_typed<kF16, kVec, kX32, 256, 1>(p, pdl, stream);
  if (p.H <= 4096) return add_norm_typed<kF16, kVec, kX32, 512, 1>(p, pdl, stream);
  if (p.H <= 8192) return add_norm_typed<kF16, kVec, kX32, 1024, 1>(p, pdl, stream);
  if (p.H <= 16384) return add_norm_typed<kF16, kVec, kX32, 1024, 2>(p, pdl, stream);
  return add_norm_typed<kF16, kVec, kX32, 1024, 4>(p, pdl, stream);
}

template <bool kF16>
static cudaError_t add_norm_half(const AddNormParams& p, int vec, int sms, int pdl, cudaStream_t stream) {
  if (!vec) return add_norm_width<kF16, false, false>(p, sms, pdl, stream);  // (its loads go by the types at run time)
  return p.x_type == 2 ? add_norm_width<kF16, true, true>(p, sms, pdl, stream)
                       : add_norm_width<kF16, true, false>(p, sms, pdl, stream);
}

cudaError_t launch_add_norm(const AddNormParams& p, int f16, int vec, int sms, int pdl, cudaStream_t stream) {
  return f16 ? add_norm_half<true>(p, vec, sms, pdl, stream) : add_norm_half<false>(p, vec, sms, pdl, stream);
}

}  // namespace fp4
