// k_add_norm.cuh -- a block's output into the residual stream and the next
// block's norm (fp4gemv_add_norm).
//
// The mathematics, per token, binary32 throughout:
//   u = y, or y / sqrt(mean y^2 + eps) (offset + post)
//   r = x + scale g u         (g: 1, the gate, or its logistic function)
//   h = r / sqrt(mean r^2 + eps) (offset + weight)
// h comes from r before r is rounded to the stream's type.
//
// A token's values stay in the registers of one group of threads from the
// first read to the last write: every input is read once and every output
// written once, with one sum over the group for each norm.
//
// What bounds it: HBM for many tokens, the launch and two dependent trips to L2 for few.  Loads of x, y and gates are all
// under way before the first sum, two chunks of 8 values to a thread, 1024 threads to an SM.  Of the measured copy
// bandwidth: 20011 tokens of 4096, bf16, norms on both sides and a gate for each value 132 us, 0.93 (loads as they come to
// be used, a chunk to a thread: 254); without the gate 0.88, the next norm alone 0.98, an fp32 stream 1.0; 5120 0.77, 6144
// 0.67, 8192 0.80, 10240 0.79, 16384 0.65 (one CTA to an SM: nothing fills in between its phases).  Rows that are not
// aligned go value by value: 4099 0.32.  One token of 4096: 3.2 us a call, 37 of 6144 3.6.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace fp4 {

struct AddNormParams {
  const void* x;
  const void* y;        // NULL: no block, the norm of x alone
  const void* weight;
  const void* post;     // NULL: no norm behind the block
  const void* gate;     // NULL: none
  void* residual;
  void* out;
  int64_t ldx, ldy, ldg, ldr, ldo;  // ldg 0: one row of gates for all tokens
  int M, H;
  int x_type, w_type, g_type;  // fp4gemv_dtype; y and out are of the kernel's half type
  int gate_scalar;             // one gate per token
  int sigmoid;
  float scale, eps, offset;
};

constexpr int kNormMaxWidth = 32768;

// Eight values of a row, as fp32.  kVec: neighbours, 16-byte aligned; else kStep apart, those before `left` only.
template <bool kVec, int kStep>
__device__ __forceinline__ void norm_load(const void* p, int type, int64_t at, int left, float (&v)[8]) {
  if constexpr (kVec) {
    if (type == 2) {
      const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
      const float4 a = s[0], b = s[1];
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (type == 1) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
          v[2 * k] = f.x, v[2 * k + 1] = f.y;
        } else {
          v[2 * k] = __uint_as_float(w[k] << 16), v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = 0.0f;
      if (j * kStep < left) {
        const int64_t i = at + j * kStep;
        if (type == 2) v[j] = static_cast<const float*>(p)[i];
        else if (type == 1) v[j] = __half2float(static_cast<const __half*>(p)[i]);
        else v[j] = __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
      }
    }
  }
}
template <bool kVec, int kStep>
__device__ __forceinline__ void norm_store(void* p, int type, int64_t at, int left, const float (&v)[8]) {
  if constexpr (kVec) {
    if (type == 2) {
      float4* d = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
      d[0] = make_float4(v[0], v[1], v[2], v[3]);
      d[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (type == 1) {
          const __half2 h = __floats2half2_rn(v[2 * k], v[2 * k + 1]);
          w[k] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
          w[k] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j * kStep < left) {
        const int64_t i = at + j * kStep;
        if (type == 2) static_cast<float*>(p)[i] = v[j];
        else if (type == 1) static_cast<__half*>(p)[i] = __float2half_rn(v[j]);
        else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v[j]);
      }
  }
}

// Eight values as they lie (kVec): of a half type in `a`, of fp32 in both.
struct NormRaw {
  uint4 a, b;
};
__device__ __forceinline__ void norm_fetch(const void* p, bool f32, int64_t at, NormRaw& r) {
  if (f32) {
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at);
    r.a = s[0], r.b = s[1];
  } else {
    r.a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
  }
}
template <bool kF16>
__device__ __forceinline__ void norm_values(const NormRaw& r, bool f32, float (&v)[8]) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
  if (f32) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(w[k]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (kF16) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
        v[2 * k] = f.x, v[2 * k + 1] = f.y;
      } else {
        v[2 * k] = __uint_as_float(w[k] << 16), v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
      }
    }
  }
}
__device__ __forceinline__ float norm_gate(float g, int sigmoid) { return sigmoid ? __fdividef(1.0f, 1.0f + __expf(-g)) : g; }

// Threads of a CTA: whole tokens, 256 threads or more where that comes out even.
__host__ __device__ constexpr int norm_threads(int row) { return row < 256 && 256 % row == 0 ? 256 : row; }
// CTAs per SM that registers are kept for: 1024 threads of two chunks, 640 of four.
__host__ __device__ constexpr int norm_ctas(int row, int chunks) {
  return chunks == 1 || row > 512 ? 1 : (chunks == 2 ? 1024 : 640) / norm_threads(row) < 1 ? 1 : (chunks == 2 ? 1024 : 640) / norm_threads(row);
}

// kRow threads to a token, kChunks times eight values each.  kX32: the stream is fp32.
template <bool kF16, bool kVec, bool kX32, int kRow, int kChunks>
__global__ void __launch_bounds__(norm_threads(kRow), norm_ctas(kRow, kChunks)) add_norm_kernel(const AddNormParams p) {
  constexpr int kThreads = norm_threads(kRow), kRows = kThreads / kRow, kWarps = kRow / 32;
  constexpr int kHalf = kF16 ? 1 : 0;
  __shared__ float sums[2][kThreads / 32];
  const int tid = threadIdx.x % kRow, group = threadIdx.x / kRow;
  if (threadIdx.x == 0) pdl_launch_dependents();
  pdl_wait();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + group;
  // the sum over the token's threads, in a fixed order
  auto total = [&](float s, int which) -> float {
#pragma unroll
    for (int o = kRow < 32 ? kRow / 2 : 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if constexpr (kWarps > 1) {
      if ((threadIdx.x & 31) == 0) sums[which][threadIdx.x >> 5] = s;
      __syncthreads();
      s = 0.0f;
      if constexpr (kWarps <= 8) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += sums[which][group * kWarps + w];
      } else {
        const int lane = threadIdx.x & 31;
        if (lane < kWarps) s = sums[which][group * kWarps + lane];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
      }
    }
    return s;
  };
  // chunk i of the thread: its first value, and whether the row has any from there
  auto first = [&](int i) -> int { return kVec ? (tid + i * kRow) * 8 : i * 8 * kRow + tid; };
  auto live = [&](int i) -> bool { return row < p.M && first(i) < p.H; };
  // what the row needs of HBM, under way at once (not kVec: as it comes to be used)
  NormRaw xr[kChunks], yr[kChunks], gr[kChunks];
  const bool gated = p.gate && !p.gate_scalar, g32 = p.g_type == 2;
  if constexpr (kVec) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      if (!live(i)) continue;
      if (p.y) norm_fetch(p.y, false, row * p.ldy + first(i), yr[i]);
      norm_fetch(p.x, kX32, row * p.ldx + first(i), xr[i]);
      if (gated && !g32) norm_fetch(p.gate, false, row * p.ldg + first(i), gr[i]);
    }
  }
  float r[kChunks][8];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) r[i][j] = 0.0f;
    if (!live(i)) continue;
    if (p.y) {
      if constexpr (kVec) norm_values<kF16>(yr[i], false, r[i]);
      else norm_load<kVec, kRow>(p.y, kHalf, row * p.ldy + first(i), p.H - first(i), r[i]);
    } else {
      if constexpr (kVec) norm_values<kF16>(xr[i], kX32, r[i]);
      else norm_load<kVec, kRow>(p.x, p.x_type, row * p.ldx + first(i), p.H - first(i), r[i]);
    }
  }
  if (p.y) {
    float factor = p.scale;
    if (p.gate && p.gate_scalar && row < p.M) {
      float g;
      if (g32) g = static_cast<const float*>(p.gate)[row * p.ldg];
      else if (kF16) g = __half2float(static_cast<const __half*>(p.gate)[row * p.ldg]);
      else g = __bfloat162float(static_cast<const __nv_bfloat16*>(p.gate)[row * p.ldg]);
      factor *= norm_gate(g, p.sigmoid);
    }
    if (p.post) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < kChunks; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(r[i][j], r[i][j], s);
      factor *= rsqrtf(total(s, 0) / static_cast<float>(p.H) + p.eps);
    }
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      if (!live(i)) continue;
      const int left = p.H - first(i);
      float f[8], x[8];
      if constexpr (kVec) norm_values<kF16>(xr[i], kX32, x);
      else norm_load<kVec, kRow>(p.x, p.x_type, row * p.ldx + first(i), left, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = factor;
      if (p.post) {
        float w[8];
        norm_load<kVec, kRow>(p.post, p.w_type, first(i), left, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= w[j] + p.offset;
      }
      if (gated) {
        float g[8];
        if (kVec && !g32) norm_values<kF16>(gr[i], false, g);
        else norm_load<kVec, kRow>(p.gate, p.g_type, row * p.ldg + first(i), left, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= norm_gate(g[j], p.sigmoid);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) r[i][j] = kVec || j * kRow < left ? fmaf(r[i][j], f[j], x[j]) : 0.0f;
      norm_store<kVec, kRow>(p.residual, p.x_type, row * p.ldr + first(i), left, r[i]);
    }
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kChunks; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) s = fmaf(r[i][j], r[i][j], s);
  const float f = rsqrtf(total(s, 1) / static_cast<float>(p.H) + p.eps);
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    if (!live(i)) continue;
    const int left = p.H - first(i);
    float w[8];
    norm_load<kVec, kRow>(p.weight, p.w_type, first(i), left, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = r[i][j] * f * (w[j] + p.offset);
    norm_store<kVec, kRow>(p.out, kHalf, row * p.ldo + first(i), left, w);
  }
}

}  // namespace fp4
