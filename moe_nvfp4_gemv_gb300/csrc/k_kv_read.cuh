// k_kv_read.cuh -- the last tokens of sequences out of the paged 8-bit cache
// again (fp4gemv_kv_read): value = code * scale in binary32, rounded once to
// the output's type.
//
// A CTA takes a page's tokens of one sequence, K or V, of some heads.  Units
// are numbered without the lengths at hand, as k_kv_append.cuh does it:
// sequence b's start at cu[b] / block_size + 2 b, and a unit finds its sequence
// by a 32-way search.  A thread keeps to one chunk column (16 bytes of output)
// and has kReadDepth loads in flight; a warp's loads and stores are contiguous
// runs of a head's row.
//
// What bounds it: HBM.  40001 tokens in five uneven prompts, 8 heads of 128, INT8 pages of 64 to bf16: 39.9 us, 0.92 of the
// measured copy bandwidth on codes and outputs; 33 tokens of one sequence 2.7 us, the launch and one dependent chain.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "k_kv_append.cuh"

namespace fp4 {

struct KvReadParams {
  const uint8_t* codes[2];  // k, v
  const float* scale[2];
  void* dst[2];
  int64_t ld[2];
  const int32_t* cu;        // NULL: `uniform` tokens each
  const int32_t* table;
  const int32_t* lens;
  uint32_t* err;
  int uniform, B, T;
  int max_blocks, num_blocks, heads, block_log2, dim;
  int heads_per;            // heads of a CTA
  int step, chunk_magic;    // tokens that a pass of all threads covers; ceil(2^16 / chunks of a row)
};

constexpr int kReadThreads = 128;
constexpr int kReadDepth = 8;

// kOut: fp4gemv_dtype of the output
template <bool kInt8, int kOut>
__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(const KvReadParams p) {
  constexpr int kValues = kOut == 2 ? 4 : 8;  // of a chunk
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid == 0) pdl_launch_dependents();
  pdl_wait();
  const int unit = blockIdx.x, head0 = blockIdx.y * p.heads_per, part = blockIdx.z;
  int b, page_no, row0, count;
  if (p.cu) {
    // the last sequence that starts at or before the unit: starts do not fall, so votes count them
    b = 0;
    for (int stride = p.B > 32 ? 32 : 1; stride; stride = stride > 1 ? 1 : 0) {
      const int at = b + lane * stride;
      const bool starts = at < p.B && (__ldg(p.cu + at) >> p.block_log2) + 2 * at <= unit;
      b += max(__popc(__ballot_sync(0xFFFFFFFFu, starts)) - 1, 0) * stride;
    }
    row0 = __ldg(p.cu + b);
    count = __ldg(p.cu + b + 1) - row0;
    page_no = unit - ((row0 >> p.block_log2) + 2 * b);
  } else {
    const int per = ((p.uniform + (1 << p.block_log2) - 2) >> p.block_log2) + 1;
    b = per == 1 ? unit : unit / per;
    page_no = unit - b * per;
    row0 = b * p.uniform;
    count = p.uniform;
  }
  if (count <= 0 || page_no < 0 || row0 < 0 || count > p.T - row0) {
    if (tid == 0 && (row0 < 0 || count < 0 || count > p.T - row0)) raise_error(p.err, FP4_ERR_BADIDX);
    return;
  }
  const int length = min(max(__ldg(p.lens + b), -(1 << 30)), 1 << 30);
  const int start = length - count;  // position of the first token (below 0: there is none)
  const int page = (start >> p.block_log2) + page_no;
  const int64_t begin = max(static_cast<int64_t>(page) << p.block_log2, static_cast<int64_t>(start));
  const int64_t end = min((static_cast<int64_t>(page) + 1) << p.block_log2, static_cast<int64_t>(length));
  if (begin >= end) return;
  int id = -1;
  if (page >= 0 && page < p.max_blocks) id = __ldg(p.table + static_cast<int64_t>(b) * p.max_blocks + page);
  const bool good = id >= 0 && id < p.num_blocks;  // (else: zeros)
  if (!good && tid == 0) raise_error(p.err, FP4_ERR_BADIDX);

  const int chunks = p.dim / kValues, first = (tid * p.chunk_magic) >> 16, col = tid - first * chunks;
  const int rows = static_cast<int>(end - begin), slot = static_cast<int>(begin - (static_cast<int64_t>(page) << p.block_log2));
  const int passes = (rows + p.step - 1) / p.step;
  const int here = min(p.heads_per, p.heads - head0);
  const int64_t tile0 = (good ? static_cast<int64_t>(id) : 0) * p.heads + head0;
  const uint8_t* const codes = (part ? p.codes[1] : p.codes[0]) + ((tile0 << p.block_log2) + slot + first) * p.dim + col * kValues;
  const float* const scale = (part ? p.scale[1] : p.scale[0]) + tile0;
  const int64_t ld = part ? p.ld[1] : p.ld[0];
  const int64_t out0 = (row0 + (begin - start) + first) * ld + static_cast<int64_t>(head0) * p.dim + col * kValues;
  char* const dst = static_cast<char*>(part ? p.dst[1] : p.dst[0]) + out0 * (16 / kValues);
  const int64_t head_codes = static_cast<int64_t>(p.dim) << p.block_log2;
  const bool mine = first < p.step;  // (threads past the last whole row of chunks do nothing)

  for (int k0 = 0, h0 = 0, i0 = 0; k0 < here * passes; k0 += kReadDepth) {
    uint2 raw[kReadDepth];
    float s[kReadDepth];
    int h = h0, i = i0;
#pragma unroll
    for (int u = 0; u < kReadDepth; ++u) {
      raw[u] = make_uint2(0, 0);
      s[u] = 0.0f;
      if (good && mine && h < here && first + i * p.step < rows) {
        const uint8_t* src = codes + h * head_codes + i * p.step * p.dim;
        if (kValues == 8) raw[u] = __ldg(reinterpret_cast<const uint2*>(src));
        else raw[u].x = __ldg(reinterpret_cast<const uint32_t*>(src));
        s[u] = __ldg(scale + h);
      }
      if (++i == passes) i = 0, ++h;
    }
    h = h0, i = i0;
#pragma unroll
    for (int u = 0; u < kReadDepth; ++u) {
      if (mine && h < here && first + i * p.step < rows) {
        float x[8];
        kv_values4<kInt8>(raw[u].x, reinterpret_cast<float(&)[4]>(x[0]));
        if (kValues == 8) kv_values4<kInt8>(raw[u].y, reinterpret_cast<float(&)[4]>(x[4]));
#pragma unroll
        for (int j = 0; j < kValues; ++j) x[j] = __fmul_rn(x[j], s[u]);
        uint4 w;
        if (kOut == 2) {
          w = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
        } else {
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (kOut == 1) {
              const __half2 t = __floats2half2_rn(x[2 * j], x[2 * j + 1]);
              o[j] = *reinterpret_cast<const uint32_t*>(&t);
            } else {
              const __nv_bfloat162 t = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
              o[j] = *reinterpret_cast<const uint32_t*>(&t);
            }
          }
          w = make_uint4(o[0], o[1], o[2], o[3]);
        }
        *reinterpret_cast<uint4*>(dst + (i * p.step * ld + static_cast<int64_t>(h) * p.dim) * (16 / kValues)) = w;
      }
      if (++i == passes) i = 0, ++h;
    }
    h0 = h, i0 = i;
  }
}

}  // namespace fp4
