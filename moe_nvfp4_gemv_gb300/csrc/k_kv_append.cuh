// k_kv_append.cuh -- new keys and values into the paged 8-bit cache
// (fp4gemv_kv_append; the formats are in include/fp4gemv_decode.h).
//
// One CTA per (touched page, KV head, K or V): it holds the page's new values
// in registers (a chunk of 8 in each of at most 8 tokens per thread), takes their largest
// finite magnitude, settles the page's scale, rounds the older codes again
// where the scale grew, and stores codes and scale.  Every value is read
// once and every code written once; no two CTAs write the same page and head.
//
// Units are numbered without the lengths at hand: sequence b may touch at
// most n / block_size + 2 pages, so with new tokens [cu[b], cu[b + 1]) its
// units start at cu[b] / block_size + 2 b, and a unit finds its sequence by
// bisection; numbers no page answers to return at once.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace fp4 {

struct KvAppendParams {
  const uint16_t* src[2];  // k, v
  int64_t ld[2];
  uint8_t* codes[2];
  float* scale[2];
  const int32_t* cu;       // NULL: `uniform` tokens each
  const int32_t* table;
  const int32_t* lens;
  uint32_t* err;
  int uniform, B, T;
  int max_blocks, num_blocks, heads, block, dim;
};

constexpr float kKvMinScale = 7.888609052210118e-31f;  // 2^-100
constexpr int kAppendChunks = 8;                       // chunks of 8 values per thread

// The scale of a page whose largest magnitude is amax (finite).
template <bool kInt8>
__device__ __forceinline__ float kv_scale(float amax) {
  if (kInt8) return fmaxf(__fmul_rn(amax, 1.0f / 127.0f), kKvMinScale);
  // the least 2^e with amax <= 1.75 * 2^(e + 8): the exponent, one more when
  // the mantissa is above 1.75
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u);
  return __uint_as_float(static_cast<uint32_t>(max(e, 27)) << 23);
}

__device__ __forceinline__ uint32_t e4m3x2_codes(float lo, float hi) {
  unsigned short d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
// x / s to the nearest code (int8: ties to even, NaN to 0; E4M3: saturating).
template <bool kInt8>
__device__ __forceinline__ uint32_t kv_codes4(const float (&x)[4]) {
  if (kInt8) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = __float2int_rn(fminf(fmaxf(x[i], -127.0f), 127.0f));
      w |= static_cast<uint32_t>(x[i] == x[i] ? q & 0xFF : 0) << (8 * i);
    }
    return w;
  }
  return e4m3x2_codes(x[0], x[1]) | (e4m3x2_codes(x[2], x[3]) << 16);
}

template <bool kInt8>
__device__ __forceinline__ void kv_values4(uint32_t w, float (&x)[4]) {
  if (kInt8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t h;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<unsigned short>(w >> (16 * i))));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

template <bool kInt8, bool kF16, int kThreads>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvAppendParams p) {
  __shared__ float warp_max[kThreads / 32];
  const int tid = threadIdx.x;
  if (tid == 0) pdl_launch_dependents();
  pdl_wait();
  // the unit's sequence, and its page
  const int unit = blockIdx.x, head = blockIdx.y, part = blockIdx.z;
  int b, page_no, first_new, count;
  if (p.cu) {
    int lo = 0, hi = p.B - 1;  // the last sequence that starts at or before the unit
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(p.cu + mid) / p.block + 2 * mid <= unit) lo = mid;
      else hi = mid - 1;
    }
    b = lo;
    first_new = __ldg(p.cu + b);
    count = __ldg(p.cu + b + 1) - first_new;
    page_no = unit - (first_new / p.block + 2 * b);
  } else {
    const int per = (p.uniform + p.block - 2) / p.block + 1;
    b = unit / per;
    page_no = unit - b * per;
    first_new = b * p.uniform;
    count = p.uniform;
  }
  if (count <= 0 || page_no < 0 || first_new < 0 || count > p.T - first_new) {
    if (tid == 0 && (first_new < 0 || count < 0 || count > p.T - first_new)) raise_error(p.err, FP4_ERR_BADIDX);
    return;
  }
  const int64_t start = static_cast<int64_t>(__ldg(p.lens + b)) - count;  // position of the first new token
  const int64_t cap = static_cast<int64_t>(p.max_blocks) * p.block;
  if (page_no == 0 && tid == 0 && (start < 0 || start + count > cap)) raise_error(p.err, FP4_ERR_BADIDX);
  // positions that lie on the table
  const int64_t from = start > 0 ? start : 0, to = start + count < cap ? start + count : cap;
  const int64_t page = from / p.block + page_no;
  if (from >= to || page * p.block >= to) return;
  const int64_t begin = page * p.block > from ? page * p.block : from;
  const int64_t end = (page + 1) * p.block < to ? (page + 1) * p.block : to;
  const int id = __ldg(p.table + static_cast<int64_t>(b) * p.max_blocks + page);
  if (id < 0 || id >= p.num_blocks) {
    if (tid == 0) raise_error(p.err, FP4_ERR_BADIDX);
    return;
  }
  const int slot = static_cast<int>(begin - page * p.block);  // the first new token's place on the page
  // A thread takes chunk `col` of tokens first, first + step, ...
  const int chunks = p.dim / 8, step = kThreads / chunks, first = tid / chunks, col = tid - first * chunks;
  const int count_here = static_cast<int>(end - begin);
  const int left = first < step ? count_here - first : 0;  // (threads past the last whole row of chunks do nothing)
  const int64_t token0 = first_new + (begin - start);
  const int64_t ld = part ? p.ld[1] : p.ld[0];
  const uint16_t* src = (part ? p.src[1] : p.src[0]) + (token0 + first) * ld + static_cast<int64_t>(head) * p.dim + col * 8;
  const int64_t src_step = step * ld;
  const int64_t tile = static_cast<int64_t>(id) * p.heads + head;
  uint8_t* codes = (part ? p.codes[1] : p.codes[0]) + tile * p.block * p.dim;
  float* scale_at = (part ? p.scale[1] : p.scale[0]) + tile;

  uint4 raw[kAppendChunks];
  auto unpack = [&](uint32_t w) -> float2 {
    return kF16 ? __half22float2(*reinterpret_cast<const __half2*>(&w))
                 : make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  };
#pragma unroll
  for (int i = 0; i < kAppendChunks; ++i) {
    raw[i] = make_uint4(0, 0, 0, 0);
    if (i * step < left) raw[i] = __ldg(reinterpret_cast<const uint4*>(src + i * src_step));
  }
  // magnitudes of both types are ordered like their bits; anything from `bound` on is not finite
  const uint32_t bound = kF16 ? 0x7C00u : 0x7F80u;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kAppendChunks; ++i)
    top = __vmaxu2(top, __vmaxu2(__vmaxu2(raw[i].x & 0x7FFF7FFFu, raw[i].y & 0x7FFF7FFFu),
                                 __vmaxu2(raw[i].z & 0x7FFF7FFFu, raw[i].w & 0x7FFF7FFFu)));
  const bool odd = max(top & 0xFFFFu, top >> 16) >= bound;  // some value of this thread is not finite
  float amax;
  if (odd) {
    amax = 0.0f;
#pragma unroll
    for (int i = 0; i < kAppendChunks; ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = unpack(w[j]);
        const float a0 = fabsf(f.x), a1 = fabsf(f.y);
        if (a0 < __builtin_huge_valf()) amax = fmaxf(amax, a0);
        if (a1 < __builtin_huge_valf()) amax = fmaxf(amax, a1);
      }
    }
  } else {
    const float2 f = unpack(top);
    amax = fmaxf(f.x, f.y);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  if ((tid & 31) == 0) warp_max[tid >> 5] = amax;
  const float old = slot > 0 ? *scale_at : 0.0f;
  __syncthreads();  // (the scale is read by every thread before it is written)
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) amax = fmaxf(amax, warp_max[i]);
  const float scale = fmaxf(old, kv_scale<kInt8>(amax));
  if (tid == 0 && scale != old) *scale_at = scale;

  if (old > 0.0f && scale > old) {  // older codes, to the larger scale
    uint32_t* w = reinterpret_cast<uint32_t*>(codes);
    for (int i = tid; i < slot * p.dim / 4; i += kThreads) {
      float x[4];
      kv_values4<kInt8>(w[i], x);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = __fdiv_rn(__fmul_rn(x[j], old), scale);
      w[i] = kv_codes4<kInt8>(x);
    }
  }
  const float inv = __fdiv_rn(1.0f, scale);  // (E4M3: an exact power of two)
  uint2* dst = reinterpret_cast<uint2*>(codes + static_cast<int64_t>(slot + first) * p.dim) + col;
  const int dst_step = step * chunks;
  uint32_t again = kInt8 && odd ? 0xFFu : 0u;  // chunks that need the division itself
#pragma unroll
  for (int i = 0; i < kAppendChunks; ++i) {
    if (i * step >= left) continue;
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack(w[j]);
      x[2 * j] = __fmul_rn(f.x, inv), x[2 * j + 1] = __fmul_rn(f.y, inv);
    }
    uint32_t o[2];
    if (!kInt8) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float v[4] = {x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]};
        o[h] = kv_codes4<kInt8>(v);
      }
    } else {
      // round(x / scale) from y = x (1 / scale): within 128 2^-22 of the rounded quotient, so its nearest integer is
      // the quotient's unless y lies that near to a half; then, and for what is not finite, the division itself,
      // below.  Adding 1.5 2^23 rounds to an integer and leaves it in the low bits.
      float far = 0.0f;
      uint32_t bits[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = __fadd_rn(x[j], 12582912.0f);
        bits[j] = __float_as_uint(n);
        far = fmaxf(far, fabsf(__fsub_rn(x[j], __fsub_rn(n, 12582912.0f))));
      }
      if (far > 0.49995f) again |= 1u << i;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        o[h] = __byte_perm(__byte_perm(bits[4 * h], bits[4 * h + 1], 0x0040),
                           __byte_perm(bits[4 * h + 2], bits[4 * h + 3], 0x0040), 0x5410);
    }
    dst[i * dst_step] = make_uint2(o[0], o[1]);
  }
  if (kInt8) {
#pragma unroll 1
    for (int i = 0; i * step < left; ++i) {
      if (!((again >> i) & 1u)) continue;
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(src + i * src_step));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t o[2];
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        const float2 a = unpack(h ? w[2] : w[0]), d = unpack(h ? w[3] : w[1]);
        const float q[4] = {__fdiv_rn(a.x, scale), __fdiv_rn(a.y, scale), __fdiv_rn(d.x, scale), __fdiv_rn(d.y, scale)};
        const uint32_t c = kv_codes4<kInt8>(q);
        if (h) o[1] = c;
        else o[0] = c;
      }
      dst[i * dst_step] = make_uint2(o[0], o[1]);
    }
  }
}

}  // namespace fp4
