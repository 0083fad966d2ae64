// k_kv_append.cuh -- new keys and values into the paged 8-bit cache
// (fp4gemv_kv_append; the formats are in include/fp4gemv_decode.h).
//
// One CTA per (touched page, kH KV heads, K or V): it holds the new values of
// its heads in registers (kAppendChunks chunks of 8 per thread, kAppendChunks /
// kH of each head, every chunk in another token), takes each head's largest
// finite magnitude, settles the page's scales, rounds older codes again where
// a scale grew, and stores codes and scales.  Every value is read once and
// every code written once; no two CTAs write the same page and head.  Small
// pages or few tokens put several heads into one CTA, so that the search below
// and the loads' latency are paid once for them.
//
// Units are numbered without the lengths at hand: sequence b may touch at
// most n / block_size + 2 pages, so with new tokens [cu[b], cu[b + 1]) its
// units start at cu[b] / block_size + 2 b, and a unit finds its sequence by a
// 32-way search (every warp for itself); numbers no page answers to return at
// once.
//
// What bounds it.  Long prompts: HBM (five prompts of up to 64001 tokens, 8
// heads of 128, pages of 64: E4M3 58 us, 1.0 of the measured copy bandwidth;
// INT8 70, 0.84, where rounding takes 5 instructions a value against 2.5); of
// 16001 17.7 (0.83) and 23.1 us (0.64): two to three waves of CTAs that load,
// then round, then store; pages of 16 26.0, of 128 24.9.  One token each for 64
// sequences: 3.3 us, one dependent chain (lengths, table, scale).  Measured and
// not taken: one CTA per page and head for small pages (39.6 us for pages of
// 16), divisions for INT8's rounding (32.8 us instead of 23.7), several rounds of
// heads in a CTA (2: 23.8 us, 4: 26.4).
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
  int max_blocks, num_blocks, heads, block_log2, dim;
  int step, chunk_magic;   // tokens that a pass of all threads covers; ceil(2^16 / (dim / 8))
};

constexpr float kKvMinScale = 7.888609052210118e-31f;  // 2^-100
constexpr int kAppendChunks = 8;                       // chunks of 8 values per thread, of all its heads

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

// (64 registers: 1024 threads per SM)
template <bool kInt8, bool kF16, int kThreads, int kH>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) kv_append_kernel(const KvAppendParams p) {
  constexpr int kWarps = kThreads / 32, kSlots = kAppendChunks / kH;  // chunks of a head
  __shared__ float warp_max[kWarps][kH];
  const int tid = threadIdx.x;
  if (tid == 0) pdl_launch_dependents();
  pdl_wait();
  // the unit's sequence, and its page (positions are below 2^30)
  const int unit = blockIdx.x, head0 = blockIdx.y * kH, part = blockIdx.z, lane = tid & 31;
  int b, page_no, first_new, count;
  if (p.cu) {
    // the last sequence that starts at or before the unit: starts do not fall, so votes count them
    b = 0;
    for (int stride = p.B > 32 ? 32 : 1; stride; stride = stride > 1 ? 1 : 0) {
      const int at = b + lane * stride;
      const bool starts = at < p.B && (__ldg(p.cu + at) >> p.block_log2) + 2 * at <= unit;
      b += max(__popc(__ballot_sync(0xFFFFFFFFu, starts)) - 1, 0) * stride;
    }
    first_new = __ldg(p.cu + b);
    count = __ldg(p.cu + b + 1) - first_new;
    page_no = unit - ((first_new >> p.block_log2) + 2 * b);
  } else {
    const int per = ((p.uniform + (1 << p.block_log2) - 2) >> p.block_log2) + 1;
    b = per == 1 ? unit : unit / per;
    page_no = unit - b * per;
    first_new = b * p.uniform;
    count = p.uniform;
  }
  if (count <= 0 || page_no < 0 || first_new < 0 || count > p.T - first_new) {
    if (tid == 0 && (first_new < 0 || count < 0 || count > p.T - first_new)) raise_error(p.err, FP4_ERR_BADIDX);
    return;
  }
  const int length = min(max(__ldg(p.lens + b), -(1 << 30)), 1 << 30);
  const int start = length - count;  // position of the first new token
  const int cap = p.max_blocks << p.block_log2;
  if (page_no == 0 && tid == 0 && (start < 0 || length > cap)) raise_error(p.err, FP4_ERR_BADIDX);
  // positions that lie on the table
  const int from = max(start, 0), to = min(length, cap);
  const int page = (from >> p.block_log2) + page_no;
  if (from >= to || page >= p.max_blocks || (page << p.block_log2) >= to) return;
  const int begin = max(page << p.block_log2, from), end = min((page + 1) << p.block_log2, to);
  const int id = __ldg(p.table + static_cast<int64_t>(b) * p.max_blocks + page);
  if (id < 0 || id >= p.num_blocks) {
    if (tid == 0) raise_error(p.err, FP4_ERR_BADIDX);
    return;
  }
  const int slot = begin - (page << p.block_log2);  // the first new token's place on the page
  // A thread takes chunk `col` of tokens first, first + step, ...
  const int chunks = p.dim >> 3, step = p.step, first = (tid * p.chunk_magic) >> 16, col = tid - first * chunks;
  const int left = first < step ? end - begin - first : 0;  // (threads past the last whole row of chunks do nothing)
  const int64_t ld = part ? p.ld[1] : p.ld[0];
  const uint16_t* src = (part ? p.src[1] : p.src[0]) + (static_cast<int64_t>(first_new) + (begin - start) + first) * ld +
                        head0 * p.dim + col * 8;
  const int64_t src_step = step * ld;
  const int64_t tile0 = static_cast<int64_t>(id) * p.heads + head0;
  const int64_t page_bytes = static_cast<int64_t>(p.dim) << p.block_log2;
  uint8_t* const codes = (part ? p.codes[1] : p.codes[0]) + tile0 * page_bytes;
  float* const scale_at = (part ? p.scale[1] : p.scale[0]) + tile0;
  const int here = min(kH, p.heads - head0);  // heads of this CTA

  auto unpack = [&](uint32_t w) -> float2 {
    return kF16 ? __half22float2(*reinterpret_cast<const __half2*>(&w))
                : make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  };
  uint4 raw[kH][kSlots];
  float old[kH];
#pragma unroll
  for (int h = 0; h < kH; ++h)
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      raw[h][i] = make_uint4(0, 0, 0, 0);
      if (i * step < left && h < here)
        raw[h][i] = __ldg(reinterpret_cast<const uint4*>(src + i * src_step + h * p.dim));
    }
#pragma unroll
  for (int h = 0; h < kH; ++h) old[h] = slot > 0 && h < here ? scale_at[h] : 0.0f;
  // magnitudes of both types are ordered like their bits; anything from `bound` on is not finite
  const uint32_t bound = kF16 ? 0x7C00u : 0x7F80u;
  bool odd = false;  // some value of this thread is not finite
#pragma unroll
  for (int h = 0; h < kH; ++h) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(raw[h][i].x & 0x7FFF7FFFu, raw[h][i].y & 0x7FFF7FFFu),
                                   __vmaxu2(raw[h][i].z & 0x7FFF7FFFu, raw[h][i].w & 0x7FFF7FFFu)));
    top = max(top & 0xFFFFu, top >> 16);
    if (top >= bound) {
      odd = true;
      top = 0;
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        const uint32_t w[4] = {raw[h][i].x, raw[h][i].y, raw[h][i].z, raw[h][i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t lo = w[j] & 0x7FFFu, hi = (w[j] >> 16) & 0x7FFFu;
          top = max(top, max(lo < bound ? lo : 0u, hi < bound ? hi : 0u));
        }
      }
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (lane == 0) warp_max[tid >> 5][h] = unpack(top).x;
  }
  __syncthreads();  // (scales are read by every thread before they are written)
#pragma unroll
  for (int h = 0; h < kH; ++h) {
    if (h >= here) break;
    float amax = warp_max[0][h];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) amax = fmaxf(amax, warp_max[i][h]);
    const float scale = fmaxf(old[h], kv_scale<kInt8>(amax));
    if (tid == 0 && scale != old[h]) scale_at[h] = scale;
    uint8_t* const tile = codes + h * page_bytes;
    if (old[h] > 0.0f && scale > old[h]) {  // older codes, to the larger scale
      uint32_t* w = reinterpret_cast<uint32_t*>(tile);
#pragma unroll 1
      for (int i = tid; i < slot * p.dim / 4; i += kThreads) {
        float x[4];
        kv_values4<kInt8>(w[i], x);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = __fdiv_rn(__fmul_rn(x[j], old[h]), scale);
        w[i] = kv_codes4<kInt8>(x);
      }
    }
    const float inv = __fdiv_rn(1.0f, scale);  // (E4M3: an exact power of two)
    uint2* const dst = reinterpret_cast<uint2*>(tile + (slot + first) * p.dim) + col;
    const int dst_step = step * chunks;
    uint32_t again = kInt8 && odd ? 0xFFu : 0u;  // chunks that need the division itself
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      const uint32_t w[4] = {raw[h][i].x, raw[h][i].y, raw[h][i].z, raw[h][i].w};
      uint32_t o[2];
      if (!kInt8) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float2 a = unpack(w[2 * q]), d = unpack(w[2 * q + 1]);
          const float v[4] = {__fmul_rn(a.x, inv), __fmul_rn(a.y, inv), __fmul_rn(d.x, inv), __fmul_rn(d.y, inv)};
          o[q] = kv_codes4<kInt8>(v);
        }
      } else {
        // round(x / scale) as the integer nearest to x (1 / scale), which is within 128 2^-22 of the rounded quotient:
        // the same unless it lies that near to a half; then, and for what is not finite, the division itself, below.
        // Adding 1.5 2^23 in the fused product rounds to an integer and leaves it in the low bits.
        float far = 0.0f;
        uint32_t bits[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = unpack(w[j]);
          const uint64_t x = pair(f.x, f.y), round = pair(12582912.0f, 12582912.0f), inv2 = pair(inv, inv);
          const uint64_t near = fma2(x, inv2, round);
          const float2 n = unpair(near), rest = unpair(fma2(x, inv2, fma2(near, pair(-1.0f, -1.0f), round)));
          bits[2 * j] = __float_as_uint(n.x), bits[2 * j + 1] = __float_as_uint(n.y);
          far = fmaxf(far, fmaxf(fabsf(rest.x), fabsf(rest.y)));
        }
        if (far > 0.49995f) again |= 1u << i;
#pragma unroll
        for (int q = 0; q < 2; ++q)
          o[q] = __byte_perm(__byte_perm(bits[4 * q], bits[4 * q + 1], 0x0040),
                             __byte_perm(bits[4 * q + 2], bits[4 * q + 3], 0x0040), 0x5410);
      }
      if (i * step < left) dst[i * dst_step] = make_uint2(o[0], o[1]);
    }
    if (kInt8 && again != 0) {
#pragma unroll 1
      for (int i = 0; i * step < left; ++i) {
        if (!((again >> i) & 1u)) continue;
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(src + i * src_step + h * p.dim));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t o[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float2 a = unpack(w[2 * q]), d = unpack(w[2 * q + 1]);
          const float r[4] = {__fdiv_rn(a.x, scale), __fdiv_rn(a.y, scale), __fdiv_rn(d.x, scale),
                              __fdiv_rn(d.y, scale)};
          o[q] = kv_codes4<kInt8>(r);
        }
        dst[i * dst_step] = make_uint2(o[0], o[1]);
      }
    }
  }
}

}  // namespace fp4
