// k_add_norm.cuh -- a block's output into the residual stream and the next
// block's norm (fp4gemv_add_norm).
//
// The mathematics, per token, binary32 throughout:
//   u = y, or y / sqrt(mean y^2 + eps) (offset + post)
//   r = x + scale g u         (g: 1, the gate, or its logistic function)
//   h = r / sqrt(mean r^2 + eps) (offset + weight)
// h comes from r before r is rounded to the stream's type.
//
// A token's values stay with one group of threads from the first read to the
// last write: every input is read once and every output written once, with one
// sum over the group for each norm.  They are in registers, but for part of a
// row above 16384 values (1024 threads of 32: 160 to 500 bytes of a thread spill
// to L1) and 4 to 80 bytes of fp32 streams' and of some narrow forms.
//
// What bounds it: HBM for many tokens, the launch and two dependent trips to L2 for few.  Loads of x, y and gates are all
// under way before the first sum, two chunks of 8 values to a thread, 1024 threads to an SM.  Of the measured copy
// bandwidth: 20011 tokens of 4096, bf16, norms on both sides and a gate for each value 132 us, 0.93 (loads as they come to
// be used, a chunk to a thread: 254); without the gate 0.88, the next norm alone 0.98, an fp32 stream 1.0; 5120 0.77, 6144
// 0.67, 8192 0.80, 10240 0.79, 16384 0.64, 32768 0.56 (one CTA to an SM: nothing fills in between its phases).  Rows off these
// boundaries go by pairs or by values, each a load of its own, neighbours in neighbouring threads, and are bound by the
// number of these: 4144 of 6892, norms on both sides, 56 us, 0.61 (by values 107), 20011 of 4098 with gates 188, 0.65 (593);
// 3000 of 10001 110, 0.33.  (Loads of places past the row's end instead of branches around them: 68, 257, 123.)
// One token of 4096: 3.2 us a call, 37 of 6144 3.6.
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

// Eight values of a row as they lie, in parts of kPart neighbours that are kStep values apart; those at `left` and behind
// it are zeros.  Values of a half type by twos in a word each; where a part is one value, a word each.
template <int kPart, int kStep>
__device__ __forceinline__ void norm_fetch(const void* p, bool f32, int64_t at, int left, uint32_t (&w)[8]) {
#pragma unroll
  for (int q = 0; q < 8 / kPart; ++q) {
    const bool live = kPart == 8 || q * kStep < left;
    const int64_t from = at + q * kStep;
    if (f32) {
      const float* const s = static_cast<const float*>(p) + from;
      if constexpr (kPart == 8) {
        const uint4 a = reinterpret_cast<const uint4*>(s)[0], b = reinterpret_cast<const uint4*>(s)[1];
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
      } else if constexpr (kPart == 2) {
        const uint2 a = live ? *reinterpret_cast<const uint2*>(s) : make_uint2(0, 0);
        w[2 * q] = a.x, w[2 * q + 1] = a.y;
      } else {
        w[q] = live ? *reinterpret_cast<const uint32_t*>(s) : 0u;
      }
    } else {
      const uint16_t* const s = static_cast<const uint16_t*>(p) + from;
      if constexpr (kPart == 8) {
        const uint4 a = *reinterpret_cast<const uint4*>(s);
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
      } else if constexpr (kPart == 2) {
        w[q] = live ? *reinterpret_cast<const uint32_t*>(s) : 0u;
      } else {
        w[q] = live ? *s : 0u;
      }
    }
  }
}
template <int kPart, bool kF16>
__device__ __forceinline__ void norm_values(const uint32_t (&w)[8], bool f32, float (&v)[8]) {
  if (f32) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(w[k]);
  } else if constexpr (kPart == 1) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      v[k] = kF16 ? __half2float(__ushort_as_half(static_cast<uint16_t>(w[k]))) : __uint_as_float(w[k] << 16);
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
template <int kPart, int kStep, bool kF16>
__device__ __forceinline__ void norm_load(const void* p, bool f32, int64_t at, int left, float (&v)[8]) {
  uint32_t w[8];
  norm_fetch<kPart, kStep>(p, f32, at, left, w);
  norm_values<kPart, kF16>(w, f32, v);
}
template <int kPart, int kStep, bool kF16>
__device__ __forceinline__ void norm_store(void* p, bool f32, int64_t at, int left, const float (&v)[8]) {
  uint32_t w[4];
  if (!f32) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (kF16) {
        const __half2 h = __floats2half2_rn(v[2 * k], v[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < 8 / kPart; ++q) {
    if (kPart != 8 && q * kStep >= left) continue;
    const int64_t to = at + q * kStep;
    if (f32) {
      float* const d = static_cast<float*>(p) + to;
      if constexpr (kPart == 8) {
        reinterpret_cast<float4*>(d)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(d)[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else if constexpr (kPart == 2) {
        *reinterpret_cast<float2*>(d) = make_float2(v[2 * q], v[2 * q + 1]);
      } else {
        *d = v[q];
      }
    } else {
      uint16_t* const d = static_cast<uint16_t*>(p) + to;
      if constexpr (kPart == 8) *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
      else if constexpr (kPart == 2) *reinterpret_cast<uint32_t*>(d) = w[q];
      else *d = static_cast<uint16_t>(w[q / 2] >> (16 * (q & 1)));
    }
  }
}
// The logistic function is e / (1 + e) below 0 and 1 / (1 + e) above, e = 2^(-|g| log2(e)): the divisor is within 1 .. 2, and
// small results keep their digits.  e is a square, so that it may be subnormal.
__device__ __forceinline__ float norm_gate(float g, int sigmoid) {
  if (!sigmoid) return g;
  float root, inv;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(root) : "f"(fabsf(g) * -0.7213475204444817f));
  const float e = root * root;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(1.0f + e));
  return (g < 0.0f ? e : 1.0f) * inv;
}

// Threads of a CTA: whole tokens, 256 threads or more where that comes out even.
__host__ __device__ constexpr int norm_threads(int row) { return row < 256 && 256 % row == 0 ? 256 : row; }
// CTAs per SM that registers are kept for: 1024 threads of two chunks, 640 of four.
__host__ __device__ constexpr int norm_ctas(int row, int chunks) {
  return chunks == 1 || row > 512 ? 1 : (chunks == 2 ? 1024 : 640) / norm_threads(row) < 1 ? 1 : (chunks == 2 ? 1024 : 640) / norm_threads(row);
}

// kRow threads to a token, kChunks times eight values each, in parts of kPart neighbours.  kX32: the stream is fp32.
template <bool kF16, int kPart, bool kX32, int kRow, int kChunks>
__global__ void __launch_bounds__(norm_threads(kRow), norm_ctas(kRow, kPart == 1 ? 2 * kChunks : kChunks))
    add_norm_kernel(const AddNormParams p) {
  constexpr int kThreads = norm_threads(kRow), kRows = kThreads / kRow, kWarps = kRow / 32, kStep = kRow * kPart;
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
  auto first = [&](int i) -> int { return tid * kPart + i * 8 * kRow; };
  auto live = [&](int i) -> bool { return row < p.M && first(i) < p.H; };
  // what the row needs of HBM, under way at once
  uint32_t xr[kChunks][8], yr[kChunks][8], gr[kChunks][8];
  const bool gated = p.gate && !p.gate_scalar, g32 = p.g_type == 2, w32 = p.w_type == 2;
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    if (!live(i)) continue;
    const int left = p.H - first(i);
    if (p.y) norm_fetch<kPart, kStep>(p.y, false, row * p.ldy + first(i), left, yr[i]);
    norm_fetch<kPart, kStep>(p.x, kX32, row * p.ldx + first(i), left, xr[i]);
    if (gated && !g32) norm_fetch<kPart, kStep>(p.gate, false, row * p.ldg + first(i), left, gr[i]);
  }
  float r[kChunks][8];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) r[i][j] = 0.0f;
    if (!live(i)) continue;
    if (p.y) norm_values<kPart, kF16>(yr[i], false, r[i]);
    else norm_values<kPart, kF16>(xr[i], kX32, r[i]);
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
      norm_values<kPart, kF16>(xr[i], kX32, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = factor;
      if (p.post) {
        float w[8];
        norm_load<kPart, kStep, kF16>(p.post, w32, first(i), left, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= w[j] + p.offset;
      }
      if (gated) {
        float g[8];
        if (g32) norm_load<kPart, kStep, kF16>(p.gate, true, row * p.ldg + first(i), left, g);
        else norm_values<kPart, kF16>(gr[i], false, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= norm_gate(g[j], p.sigmoid);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) r[i][j] = kPart == 8 || j / kPart * kStep < left ? fmaf(r[i][j], f[j], x[j]) : 0.0f;
      norm_store<kPart, kStep, kF16>(p.residual, kX32, row * p.ldr + first(i), left, r[i]);
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
    norm_load<kPart, kStep, kF16>(p.weight, w32, first(i), left, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = r[i][j] * f * (w[j] + p.offset);
    norm_store<kPart, kStep, kF16>(p.out, false, row * p.ldo + first(i), left, w);
  }
}

}  // namespace fp4
