// k_kv_attention.cuh -- attention of a few newest tokens per sequence over
// the paged 8-bit cache (fp4gemv_kv_attention).
//
// The mathematics.  A page's scales leave the inner loops: with K = ks kc and
// V = vs vc (codes kc, vc) the score in base 2 is
//   s = (q . kc) ks sm_scale log2(e),
// and instead of p = 2^(s - max s) the kernel weighs codes directly with
//   w = 2^(s + log2 vs - m),   m the running maximum of s + log2 vs,
// so that out = (sum w vc) / (sum w / vs) with w of one size whatever the
// scales: w is rounded to f16 for the product with vc, sums stay fp32.  The
// codes are exact in f16.  Queries are made exact f16 operands by a power of
// two for each row.
//
// The work.  KV bytes are read once, 16 tokens (a strip) of K and V of one
// head at a time, by mma.sync m16n8k16 in the transposed form: the codes are
// the A operand (S^T = K Q^T with tokens as rows, out^T = V^T w^T with
// head_dim as rows), the query rows that share the KV head (heads of the group
// x new tokens) are the N side, in tiles of 8, so a group of up to 8 pays for
// 8 rows and not for 16.  Codes are converted from 8 bits to f16 in registers
// right before use: shared memory and HBM see 8 bits only.  The contraction
// over head_dim is permuted so that a thread's share of a K row is contiguous
// bytes, V's pairs of tokens are joined by byte permutes before the
// conversion, and the weights turn from accumulator to operand by movmatrix.
//
// m follows the maximum lazily: weights may grow to 2^kAttnSlack before m
// moves (f16 holds them, fp32 sums do), so the usual strip costs one vote and
// no shuffles; a strip that would exceed it reduces its maxima over the warp
// and rescales.
//
// Every warp streams its own strips through its own ring of cp.async stages
// and keeps its own m, sums and accumulators: no barrier in the loop.  The
// strips of all (sequence, KV head, row tile) items form one line which is
// cut into equal lengths, one for each CTA, wherever the cuts fall; at an
// item's end the warps' results are joined through shared memory.  An item
// that several CTAs share is joined from fp32 partials in the workspace by the
// last of them to arrive (a counter that it leaves at zero).  Nothing waits on
// another CTA.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace fp4 {

struct KvAttnParams {
  const uint8_t* k_codes;
  const uint8_t* v_codes;
  const float* k_scale;
  const float* v_scale;
  const uint16_t* q;
  int64_t ldq;
  uint16_t* out;
  int64_t ldo;
  float* lse;
  const int32_t* table;
  const int32_t* lens;
  uint32_t* err;
  float* partial;      // [CTAs][2][rows][dim + 2]
  uint32_t* arrived;   // [CTAs], zero between calls
  int B, max_blocks, num_blocks, block_log2;
  int kv_heads, group, q_len, row_tiles;  // row tiles of 8 kN rows
  int window;
  int f16;             // element type of q and out
  float sm_scale;
};

constexpr int kAttnMaxBatch = 1024;
constexpr float kAttnFloor = -1e30f;  // the running maximum before any token
constexpr float kAttnSlack = 8.0f;    // log2 of the largest weight before the running maximum moves

__device__ __forceinline__ float attn_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float attn_lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// C += A B; A 16 x 16 (rows g and g + 8), B 16 x 8, f16; C fp32.
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The transpose of an 8 x 8 matrix of 16-bit values, two adjacent columns of
// row g per thread.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Two codes (the low 16 bits of w) as two f16.
template <bool kInt8>
__device__ __forceinline__ uint32_t codes2_lo(uint32_t w) {
  uint32_t h;
  if (kInt8) {  // 1024 + (code + 128) as f16 bits, minus 1152
    const uint32_t u = __byte_perm(w ^ 0x80808080u, 0x64646464u, 0x4140);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(h) : "r"(u), "r"(0x64806480u));
  } else {
    asm("{ .reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l; }" : "=r"(h) : "r"(w));
  }
  return h;
}
// The high 16 bits.
template <bool kInt8>
__device__ __forceinline__ uint32_t codes2_hi(uint32_t w) {
  uint32_t h;
  if (kInt8) {
    const uint32_t u = __byte_perm(w ^ 0x80808080u, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(h) : "r"(u), "r"(0x64806480u));
  } else {
    asm("{ .reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, h; }" : "=r"(h) : "r"(w));
  }
  return h;
}

// How a strip of 16 rows of kDim code bytes lies in shared memory and which
// bytes a thread (g = lane / 4, t = lane % 4) takes.  Rows are cut into
// blocks of 64, 96 or 128 bytes.  A thread's K words of a block: kWords
// consecutive 4-byte words of row g or g + 8, the k-steps' operands.  Its V
// words: kWords / 2 words of each of the token rows 2t, 2t + 1, 2t + 8,
// 2t + 9; bytes 2 j and 2 j + 1 of word i are rows g and g + 8 of the output
// tile 2 i + j.
template <int kDim>
struct AttnLayout {
  static constexpr int kBlk = kDim % 128 == 0 ? 128 : kDim;  // 64, 96 or 128
  static constexpr int kBlocks = kDim / kBlk;
  static constexpr int kWords = kBlk / 16;   // K words per thread, row and block
  static constexpr int kVWords = kBlk / 32;  // V words per thread, token and block
  static constexpr int kSteps = kDim / 16;   // k-steps of 16
  static constexpr int kTiles = kDim / 16;   // output tiles of 16 dims
  static constexpr int kStripBytes = 16 * kDim;

  // Byte offset of 16-byte chunk c of token row r: chunks of a 128-byte line
  // change places by row, so that the accesses below meet no bank twice.
  static __device__ __forceinline__ int chunk(int r, int c) {
    if (kBlk == 128) return r * kDim + (c >> 3) * 128 + (((c & 7) ^ (r & 7)) << 4);
    if (kBlk == 64) return r * kDim + ((c ^ (r & 2)) << 4);
    return r * kDim + (c << 4);
  }
  // head_dim index of the first of the four values of K word i (block blk)
  static __device__ __forceinline__ int k_dim(int blk, int i, int t) {
    if (kBlk == 96) return 32 * (i >> 1) + 8 * t + 4 * (i & 1);
    return blk * kBlk + t * (kBlk / 4) + 4 * i;
  }
  static __device__ __forceinline__ void k_words(uint32_t base, int r, int blk, int t, uint32_t (&w)[kWords]) {
    if constexpr (kBlk == 128) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 v = lds128(base + chunk(r, blk * 8 + 2 * t + i));
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
    } else if constexpr (kBlk == 64) {
      const uint4 v = lds128(base + chunk(r, t));
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                     : "=r"(w[2 * i]), "=r"(w[2 * i + 1])
                     : "r"(base + r * kDim + 32 * i + 8 * t));
    }
  }
  // head_dim index of the first byte of thread row g's V word i (block blk)
  static __device__ __forceinline__ int v_dim(int blk, int i, int g) {
    if (kBlk == 96) return 32 * i + 4 * g;
    return blk * kBlk + g * (kBlk / 8) + 4 * i;
  }
  static __device__ __forceinline__ void v_words(uint32_t base, int r, int blk, int g, uint32_t (&w)[kVWords]) {
    if constexpr (kBlk == 128) {
      const uint4 v = lds128(base + chunk(r, blk * 8 + g));
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (kBlk == 64) {
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                   : "=r"(w[0]), "=r"(w[1])
                   : "r"(base + chunk(r, g >> 1) + 8 * (g & 1)));
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i) w[i] = lds32(base + r * kDim + 32 * i + 4 * g);
    }
  }
};

// kN: tiles of 8 query rows that a pass over the codes serves.
template <int kDim, int kN>
struct AttnCfg {
  using L = AttnLayout<kDim>;
  static constexpr int kWarps = 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kRows = 8 * kN;
  static constexpr int kResident = kDim <= 128 && kN <= 2 ? 2 : 1;  // CTAs per SM (registers, shared memory)
  static constexpr bool kQInRegs = kN == 1 && kDim <= 128;     // queries stay in registers
  static constexpr int kStageBytes = 2 * L::kStripBytes + 16;  // K, V, the two scales
  static constexpr int kStages = kDim >= 128 ? 3 : kDim == 96 ? 4 : 5;
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  static constexpr int kQBytes = kN * L::kSteps * 32 * 8;
  static constexpr int kSlabBytes = kWarps * 8 * 32 * 4;  // a joining pass: 8 rows, 32 dims of every warp
  // the joining passes come when the item's queries are no longer needed
  static constexpr int kQSlabBytes = kQBytes > kSlabBytes ? kQBytes : kSlabBytes;
  static constexpr int kSmem = kRingBytes + kQSlabBytes + kWarps * kRows * 8 + kRows * 8 + kRows * 4;
};

// One place on the line of all strips.
struct AttnCursor {
  int b, head, tile;  // sequence, KV head, row tile
  int strip, strips;  // within the item; the item's number of strips
  int first;          // the sequence's first strip that any query sees (its token / 16)
};

template <int kDim, bool kInt8, int kN>
__global__ void __launch_bounds__(AttnCfg<kDim, kN>::kThreads, AttnCfg<kDim, kN>::kResident)
    kv_attention_kernel(const KvAttnParams p) {
  using C = AttnCfg<kDim, kN>;
  using L = AttnLayout<kDim>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int line_of[kAttnMaxBatch + 1];  // strips of the sequences before each
  __shared__ int warp_sum[C::kWarps];
  __shared__ int last_flag;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  if (tid == 0) pdl_launch_dependents();
  pdl_wait();

  const int rows = p.q_len * p.group;      // query rows of an item's head
  const int items = p.kv_heads * p.row_tiles;
  const int64_t cap = static_cast<int64_t>(p.max_blocks) << p.block_log2;
  auto length = [&](int b) -> int {
    const int n = __ldg(p.lens + b);
    return n < 0 ? 0 : n > cap ? static_cast<int>(cap) : n;
  };
  auto first_strip = [&](int n) -> int {
    const int at = n - p.q_len;  // the first query's position
    return p.window > 0 && at >= p.window ? (at - p.window + 1) >> 4 : 0;
  };
  // ---- the line: an exclusive scan of the sequences' strips ----
  int base = 0;
  for (int b0 = 0; b0 < p.B; b0 += C::kThreads) {
    const int b = b0 + tid;
    int mine = 0;
    if (b < p.B) {
      const int n = length(b);
      if (n != __ldg(p.lens + b) && blockIdx.x == 0) raise_error(p.err, FP4_ERR_BADIDX);
      mine = (((n + 15) >> 4) - first_strip(n)) * items;
    }
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    int before = base, whole = base;
#pragma unroll
    for (int i = 0; i < C::kWarps; ++i) {
      before += i < warp ? warp_sum[i] : 0;
      whole += warp_sum[i];
    }
    if (b < p.B) line_of[b] = before + sum - mine;
    base = whole;
    __syncthreads();
  }
  const int total = base;
  if (tid == 0) line_of[p.B] = total;
  __syncthreads();

  // sequences nobody visits: zeros, lse -inf
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (line_of[b + 1] != line_of[b]) continue;
    const int heads = p.kv_heads * p.group;
    for (int i = tid; i < p.q_len * heads * (kDim / 8); i += C::kThreads) {
      const int64_t row = i / (kDim / 8);
      const int64_t tok = static_cast<int64_t>(b) * p.q_len + row / heads;
      reinterpret_cast<uint4*>(p.out + tok * p.ldo + (row % heads) * kDim)[i % (kDim / 8)] = make_uint4(0, 0, 0, 0);
      if (p.lse && i % (kDim / 8) == 0) p.lse[tok * heads + row % heads] = -__builtin_huge_valf();
    }
  }
  // this CTA's share, in whole rounds of its warps
  const int rounds = (total + C::kWarps - 1) / C::kWarps;
  const int per = (rounds + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x) * C::kWarps;
  const int64_t begin64 = static_cast<int64_t>(per) * blockIdx.x;
  if (begin64 >= total) return;
  const int begin = static_cast<int>(begin64);
  const int end = min(total, begin + per);

  auto seek = [&](int at) -> AttnCursor {  // the cursor of strip `at` of the line (at < total)
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (line_of[mid] <= at) lo = mid;
      else hi = mid - 1;
    }
    AttnCursor c;
    c.b = lo;  // (the last that starts at or before: never an empty one)
    const int n = length(lo);
    c.first = first_strip(n);
    c.strips = ((n + 15) >> 4) - c.first;
    const int item = (at - line_of[lo]) / c.strips;
    c.strip = (at - line_of[lo]) - item * c.strips;
    c.head = item / p.row_tiles;
    c.tile = item - c.head * p.row_tiles;
    return c;
  };
  auto advance = [&](AttnCursor& c, int by) {  // (towards a place before `total`)
    c.strip += by;
    while (c.strip >= c.strips) {
      c.strip -= c.strips;
      if (++c.tile == p.row_tiles) {
        c.tile = 0;
        if (++c.head == p.kv_heads) {
          c.head = 0;
          do ++c.b;
          while (line_of[c.b + 1] == line_of[c.b]);
          const int n = length(c.b);
          c.first = first_strip(n);
          c.strips = ((n + 15) >> 4) - c.first;
        }
      }
    }
  };

  // ---- the warp's ring ----
  const uint32_t sm = smem_u32(smem);
  const uint32_t ring = sm + warp * C::kStages * C::kStageBytes;
  const uint32_t q_base = sm + C::kRingBytes;
  float* const slab = reinterpret_cast<float*>(smem + C::kRingBytes);
  float2* const ml = reinterpret_cast<float2*>(smem + C::kRingBytes + C::kQSlabBytes);  // [warp][row]
  float2* const ml_all = ml + C::kWarps * C::kRows;                                     // [row]
  float* const row_scale = reinterpret_cast<float*>(ml_all + C::kRows);

  AttnCursor ahead{};
  int ahead_at = begin + warp;
  if (ahead_at < end) ahead = seek(ahead_at);
  const int block_mask = (1 << p.block_log2) - 1;
  auto page_of = [&](const AttnCursor& c) -> int {
    const int tok = (c.first + c.strip) << 4;
    return __ldg(p.table + static_cast<int64_t>(c.b) * p.max_blocks + (tok >> p.block_log2));
  };
  int page = ahead_at < end ? page_of(ahead) : 0;
  auto issue = [&](int stage) {
    if (ahead_at < end) {
      const uint32_t dst = ring + stage * C::kStageBytes;
      int id = page;
      const bool good = id >= 0 && id < p.num_blocks;
      if (!good) {
        if (lane == 0) raise_error(p.err, FP4_ERR_BADIDX);
        id = 0;
      }
      const uint32_t bytes = good ? 16u : 0u;
      const int64_t tile = static_cast<int64_t>(id) * p.kv_heads + ahead.head;
      const int64_t at = ((tile << p.block_log2) + (((ahead.first + ahead.strip) << 4) & block_mask)) * kDim;
#pragma unroll
      for (int i = 0; i < kDim / 32; ++i) {
        const int c = i * 32 + lane;  // 16-byte chunk of the strip
        const int r = c / (kDim / 16), o = L::chunk(r, c - r * (kDim / 16));
        cp_async16(dst + o, p.k_codes + at + c * 16, bytes);
        cp_async16(dst + L::kStripBytes + o, p.v_codes + at + c * 16, bytes);
      }
      if (lane < 2) {
        const float* s = (lane ? p.v_scale : p.k_scale) + tile;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + 2 * L::kStripBytes + 4 * lane), "l"(s),
                     "r"(good ? 4u : 0u)
                     : "memory");
      }
      ahead_at += C::kWarps;
      if (ahead_at < end) {
        advance(ahead, C::kWarps);
        page = page_of(ahead);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < C::kStages - 1; ++s) issue(s);

  // ---- segments: the parts of items in this CTA's share ----
  AttnCursor cur = seek(begin);
  int at = begin;
  int stage = 0;
  float acc[kN][L::kTiles][4];  // dims by rows: thread's rows 2t, 2t + 1 of every tile of 8
  float m[kN][2], sum[kN][2];
  while (at < end) {
    const int seg_end = min(end, at + cur.strips - cur.strip);
    const int n = length(cur.b);
    const int row0 = cur.tile * C::kRows;
    // the item's queries as f16 operands, scaled by a power of two per row
    for (int r = warp; r < C::kRows; r += C::kWarps) {
      const int row = row0 + r;
      float amax = 0.0f;
      uint32_t w[(kDim + 63) / 64];
      const bool live = row < rows;
      const uint32_t* src = nullptr;
      if (live) {
        const int64_t tok = static_cast<int64_t>(cur.b) * p.q_len + row / p.group;
        src = reinterpret_cast<const uint32_t*>(p.q + tok * p.ldq +
                                                (static_cast<int64_t>(cur.head) * p.group + row % p.group) * kDim);
      }
      auto two = [&](uint32_t v) -> float2 {
        return p.f16 ? __half22float2(*reinterpret_cast<const __half2*>(&v))
                     : make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
      };
      // (lane takes words lane, lane + 32, ...; kDim / 2 words a row)
#pragma unroll
      for (int i = 0; i < (kDim + 63) / 64; ++i) {
        const int k = i * 32 + lane;
        const uint32_t v = live && k < kDim / 2 ? __ldg(src + k) : 0u;
        w[i] = v;
        const float2 f = two(v);
        amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
      // 2^-e brings amax to [2^14, 2^15)
      const int field = static_cast<int>(__float_as_uint(amax) >> 23);
      const int e = field == 0 ? 0 : min(max(field - 127 - 14, -126), 126);
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      if (lane == 0)
        row_scale[r] = p.sm_scale * 1.4426950408889634f * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
      for (int i = 0; i < (kDim + 63) / 64; ++i) {
        const int k = i * 32 + lane;
        if (k >= kDim / 2) break;
        const float2 f = two(w[i]);
        // where the pair (2k, 2k + 1) stands: operand word `reg` of thread (r % 8, tt) in step `st`
        const int d = 2 * k, blk = d / L::kBlk, o = d - blk * L::kBlk;
        int tt, i4;
        if (L::kBlk == 96) {
          tt = (o & 31) >> 3;
          i4 = 2 * (o >> 5) + ((o & 7) >> 2);
        } else {
          tt = o / (L::kBlk / 4);
          i4 = (o - tt * (L::kBlk / 4)) >> 2;
        }
        const int st = blk * L::kWords + i4;
        const uint32_t dst = q_base + ((((r >> 3) * L::kSteps + st) >> 1) * 32 + (r & 7) * 4 + tt) * 16 + (st & 1) * 8 +
                             ((o & 2) ? 4 : 0);
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst), "r"(pack_f16(f.x * down, f.y * down)) : "memory");
      }
    }
    __syncthreads();
    auto q_frag = [&](int nt, int pair) -> uint4 {  // k-steps 2 pair and 2 pair + 1
      return lds128(q_base + ((nt * (L::kSteps / 2) + pair) * 32 + lane) * 16);
    };
    uint4 qr[C::kQInRegs ? L::kSteps / 2 : 1];
    if constexpr (C::kQInRegs) {
#pragma unroll
      for (int i = 0; i < L::kSteps / 2; ++i) qr[i] = q_frag(0, i);
    }
    float rs[kN][2];
#pragma unroll
    for (int nt = 0; nt < kN; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        rs[nt][h] = row_scale[nt * 8 + 2 * t + h];
        m[nt][h] = kAttnFloor;
        sum[nt][h] = 0.0f;
#pragma unroll
        for (int j = 0; j < L::kTiles; ++j) acc[nt][j][h] = acc[nt][j][2 + h] = 0.0f;
      }
    const int tokens_all = n - p.q_len + 1;                          // every row sees those before this one
    const int tokens_low = p.window > 0 ? max(0, n - p.window) : 0;  // ... from this one on

    // this warp's strips of the segment: line places begin + warp + k kWarps
    int i = at + ((begin + warp - at) % C::kWarps + C::kWarps) % C::kWarps;
    for (; i < seg_end; i += C::kWarps) {
      asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 2) : "memory");
      __syncwarp();
      {  // the stage read last is free: every lane is past it
        const int next = stage == 0 ? C::kStages - 1 : stage - 1;
        issue(next);
      }
      const uint32_t kb = ring + stage * C::kStageBytes, vb = kb + L::kStripBytes;
      const int tok = (cur.first + cur.strip + (i - at)) << 4;
      float sc[kN][4];  // tokens g (0, 1) and g + 8 (2, 3) by rows 2t and 2t + 1
#pragma unroll
      for (int nt = 0; nt < kN; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.0f;
#pragma unroll
      for (int blk = 0; blk < L::kBlocks; ++blk) {
        uint32_t w[2][L::kWords];
        L::k_words(kb, g, blk, t, w[0]);
        L::k_words(kb, g + 8, blk, t, w[1]);
#pragma unroll
        for (int s = 0; s < L::kWords; s += 2) {
          uint32_t a[2][4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            a[e][0] = codes2_lo<kInt8>(w[0][s + e]);
            a[e][1] = codes2_lo<kInt8>(w[1][s + e]);
            a[e][2] = codes2_hi<kInt8>(w[0][s + e]);
            a[e][3] = codes2_hi<kInt8>(w[1][s + e]);
          }
#pragma unroll
          for (int nt = 0; nt < kN; ++nt) {
            uint4 b;
            if constexpr (C::kQInRegs) b = qr[(blk * L::kWords + s) / 2];
            else b = q_frag(nt, (blk * L::kWords + s) / 2);
            mma_f16(sc[nt], a[0], b.x, b.y);
            mma_f16(sc[nt], a[1], b.z, b.w);
          }
        }
      }
      const float ks = ldsf(kb + 2 * L::kStripBytes);
      const float lv = attn_lg2(fmaxf(ldsf(kb + 2 * L::kStripBytes + 4), 7.888609052210118e-31f));
      const float inv_vs = attn_ex2(-lv);
      const bool masked = tok + 16 > tokens_all || tok < tokens_low;
      uint32_t pb[kN][2];
#pragma unroll
      for (int nt = 0; nt < kN; ++nt) {
        const float f0 = rs[nt][0] * ks, f1 = rs[nt][1] * ks;
        const float b0 = lv - m[nt][0], b1 = lv - m[nt][1];
        float x[4] = {fmaf(sc[nt][0], f0, b0), fmaf(sc[nt][1], f1, b1), fmaf(sc[nt][2], f0, b0),
                      fmaf(sc[nt][3], f1, b1)};
        bool dead[4] = {false, false, false, false};
        if (masked) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = min(row0 + nt * 8 + 2 * t + (e & 1), rows - 1), at_tok = tok + (e >> 1) * 8 + g;
            const int see_to = n - p.q_len + row / p.group + 1;
            dead[e] = at_tok >= see_to || (p.window > 0 && at_tok < see_to - p.window);
            if (dead[e]) x[e] = -__builtin_huge_valf();
          }
        }
        if (__any_sync(0xFFFFFFFFu, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) > kAttnSlack)) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float f = h ? f1 : f0;
            const float r0 = dead[h] ? -__builtin_huge_valf() : fmaf(sc[nt][h], f, lv);
            const float r1 = dead[2 + h] ? -__builtin_huge_valf() : fmaf(sc[nt][2 + h], f, lv);
            float top = fmaxf(r0, r1);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            const float mn = fmaxf(m[nt][h], top);
            const float fall = attn_ex2(m[nt][h] - mn);
            m[nt][h] = mn;
            sum[nt][h] *= fall;
#pragma unroll
            for (int j = 0; j < L::kTiles; ++j) {
              acc[nt][j][h] *= fall;
              acc[nt][j][2 + h] *= fall;
            }
            x[h] = r0 - mn;
            x[2 + h] = r1 - mn;
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = attn_ex2(x[e]);
        sum[nt][0] = fmaf(x[0] + x[2], inv_vs, sum[nt][0]);
        sum[nt][1] = fmaf(x[1] + x[3], inv_vs, sum[nt][1]);
        pb[nt][0] = transpose8x8(pack_f16(x[0], x[1]));
        pb[nt][1] = transpose8x8(pack_f16(x[2], x[3]));
      }
      const int left = n - tok;  // tokens of the sequence in this strip
#pragma unroll
      for (int blk = 0; blk < L::kBlocks; ++blk) {
        uint32_t w[4][L::kVWords];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int r = 2 * t + (c & 1) + (c >> 1) * 8;
          L::v_words(vb, r, blk, g, w[c]);
          if (left < 16 && r >= left) {  // past the end: whatever lies there counts nothing
#pragma unroll
            for (int k = 0; k < L::kVWords; ++k) w[c][k] = 0u;
          }
        }
#pragma unroll
        for (int k = 0; k < L::kVWords; ++k) {
          const uint32_t lo[2] = {__byte_perm(w[0][k], w[1][k], 0x5140), __byte_perm(w[0][k], w[1][k], 0x7362)};
          const uint32_t hi[2] = {__byte_perm(w[2][k], w[3][k], 0x5140), __byte_perm(w[2][k], w[3][k], 0x7362)};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t a[4] = {codes2_lo<kInt8>(lo[j]), codes2_hi<kInt8>(lo[j]), codes2_lo<kInt8>(hi[j]),
                                   codes2_hi<kInt8>(hi[j])};
#pragma unroll
            for (int nt = 0; nt < kN; ++nt)
              mma_f16(acc[nt][(blk * L::kVWords + k) * 2 + j], a, pb[nt][0], pb[nt][1]);
          }
        }
      }
      __syncwarp();
      stage = stage + 1 == C::kStages ? 0 : stage + 1;
    }

    // ---- the segment's end: join the warps ----
#pragma unroll
    for (int nt = 0; nt < kN; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) sum[nt][h] += __shfl_xor_sync(0xFFFFFFFFu, sum[nt][h], o);
        if (g == 0) ml[warp * C::kRows + nt * 8 + 2 * t + h] = make_float2(m[nt][h], sum[nt][h]);
      }
    __syncthreads();
    if (tid < C::kRows) {
      float top = kAttnFloor, l = 0.0f;
#pragma unroll
      for (int w = 0; w < C::kWarps; ++w) top = fmaxf(top, ml[w * C::kRows + tid].x);
#pragma unroll
      for (int w = 0; w < C::kWarps; ++w) {
        const float2 v = ml[w * C::kRows + tid];
        l += attn_ex2(v.x - top) * v.y;
      }
      ml_all[tid] = make_float2(top, l);
    }
    __syncthreads();
    const bool starts = cur.strip == 0, ends = at - cur.strip + cur.strips == seg_end;
    const bool whole = starts && ends;
    const int used = min(C::kRows, rows - row0);
    float* const part = p.partial + (static_cast<int64_t>(blockIdx.x) * 2 + (starts ? 1 : 0)) * C::kRows * (kDim + 2);
    auto store = [&](int r, int d, float4 v) {  // four outputs of local row r, dims d .. d + 3
      const int row = row0 + r;
      const int64_t tok_out = static_cast<int64_t>(cur.b) * p.q_len + row / p.group;
      uint16_t* o = p.out + tok_out * p.ldo + (static_cast<int64_t>(cur.head) * p.group + row % p.group) * kDim + d;
      uint2 w;
      if (p.f16) {
        w.x = pack_f16(v.x, v.y);
        w.y = pack_f16(v.z, v.w);
      } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
        w.x = *reinterpret_cast<const uint32_t*>(&a);
        w.y = *reinterpret_cast<const uint32_t*>(&b);
      }
      *reinterpret_cast<uint2*>(o) = w;
    };
    auto store_lse = [&](int r, float top, float l) {
      if (!p.lse) return;
      const int row = row0 + r;
      const int64_t tok_out = static_cast<int64_t>(cur.b) * p.q_len + row / p.group;
      p.lse[tok_out * (p.kv_heads * p.group) + cur.head * p.group + row % p.group] =
          l > 0.0f ? 0.6931471805599453f * (top + log2f(l)) : l == l ? -__builtin_huge_valf() : l;
    };
#pragma unroll
    for (int nt = 0; nt < kN; ++nt) {  // eight rows at a time
      if (nt * 8 >= used) break;
#pragma unroll
      for (int k = 0; k < L::kTiles / 2; ++k) {  // and a V word's 32 dims
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float4*>(slab + ((warp * 8 + 2 * t + h) * 8 + g) * 4) = make_float4(
              acc[nt][2 * k][h], acc[nt][2 * k][2 + h], acc[nt][2 * k + 1][h], acc[nt][2 * k + 1][2 + h]);
        __syncthreads();
        if (tid < 64 && nt * 8 + (tid >> 3) < used) {
          const int r = nt * 8 + (tid >> 3), col = tid & 7;
          const float2 tot = ml_all[r];
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int w = 0; w < C::kWarps; ++w) {
            const float f = attn_ex2(ml[w * C::kRows + r].x - tot.x);
            const float4 a = *reinterpret_cast<const float4*>(slab + ((w * 8 + (tid >> 3)) * 8 + col) * 4);
            v.x = fmaf(a.x, f, v.x), v.y = fmaf(a.y, f, v.y), v.z = fmaf(a.z, f, v.z), v.w = fmaf(a.w, f, v.w);
          }
          const int d = L::v_dim(k / L::kVWords, k % L::kVWords, col);
          if (whole) {
            const float inv = tot.y != 0.0f ? 1.0f / tot.y : 0.0f;
            store(r, d, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
          } else {
            __stcg(reinterpret_cast<float2*>(part + r * (kDim + 2) + d), make_float2(v.x, v.y));
            __stcg(reinterpret_cast<float2*>(part + r * (kDim + 2) + d + 2), make_float2(v.z, v.w));
          }
        }
        __syncthreads();
      }
    }
    if (whole) {
      if (tid < used) store_lse(tid, ml_all[tid].x, ml_all[tid].y);
    } else {
      if (tid < used)
        __stcg(reinterpret_cast<float2*>(part + tid * (kDim + 2) + kDim), ml_all[tid]);
      // the CTAs that share the item; the last to arrive joins their partials
      const int item0 = at - cur.strip;
      const int c0 = item0 / per, c1 = (item0 + cur.strips - 1) / per;
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const uint32_t before = atomicAdd(p.arrived + c0, 1u);
        last_flag = before == static_cast<uint32_t>(c1 - c0);
        if (last_flag) p.arrived[c0] = 0u;
      }
      __syncthreads();
      if (last_flag) {
        __threadfence();
        const int64_t stride = static_cast<int64_t>(2) * C::kRows * (kDim + 2);
        // (the first CTA's part starts the item: its slot 1; the others' slot 0)
        auto part_of = [&](int c) { return p.partial + c * stride + (c == c0 ? C::kRows * (kDim + 2) : 0); };
        // A thread takes four dims of a row and every `ways`-th partial, kBatch
        // of them in flight; the ways meet in shared memory.
        constexpr int kBatch = 8;
        const int cells = used * (kDim / 4), parts = c1 - c0 + 1;
        int ways = 1;
        while (2 * ways * cells <= C::kThreads && ways * kBatch < parts) ways *= 2;
        for (int x0 = 0; x0 < cells; x0 += C::kThreads / ways) {
          const int way = tid / (C::kThreads / ways), x = x0 + tid - way * (C::kThreads / ways);
          const bool live = x < cells;
          const int r = live ? x / (kDim / 4) : 0, d = live ? (x - r * (kDim / 4)) * 4 : 0;
          float top = kAttnFloor, l = 0.0f;
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          for (int c = c0 + way; live && c <= c1; c += kBatch * ways) {
            float2 cm[kBatch], a[kBatch], b[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
              const int cc = c + j * ways;
              cm[j] = make_float2(kAttnFloor, 0.0f);
              a[j] = b[j] = make_float2(0.0f, 0.0f);
              if (cc <= c1) {
                const float* s = part_of(cc) + r * (kDim + 2);
                cm[j] = __ldcg(reinterpret_cast<const float2*>(s + kDim));
                a[j] = __ldcg(reinterpret_cast<const float2*>(s + d));
                b[j] = __ldcg(reinterpret_cast<const float2*>(s + d + 2));
              }
            }
            float mn = top;
#pragma unroll
            for (int j = 0; j < kBatch; ++j) mn = fmaxf(mn, cm[j].x);
            const float fall = attn_ex2(top - mn);
            v.x *= fall, v.y *= fall, v.z *= fall, v.w *= fall, l *= fall;
            top = mn;
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
              const float f = attn_ex2(cm[j].x - mn);
              v.x = fmaf(a[j].x, f, v.x), v.y = fmaf(a[j].y, f, v.y);
              v.z = fmaf(b[j].x, f, v.z), v.w = fmaf(b[j].y, f, v.w);
              l = fmaf(cm[j].y, f, l);
            }
          }
          if (ways > 1) {
            float* const mine = slab + tid * 6;  // (6 kThreads floats: within the joining buffer)
            *reinterpret_cast<float2*>(mine) = make_float2(v.x, v.y);
            *reinterpret_cast<float2*>(mine + 2) = make_float2(v.z, v.w);
            *reinterpret_cast<float2*>(mine + 4) = make_float2(top, l);
            __syncthreads();
            if (way == 0) {
              for (int w = 1; w < ways; ++w) {
                const float* o = slab + (tid + w * (C::kThreads / ways)) * 6;
                const float mn = fmaxf(top, o[4]);
                const float f = attn_ex2(top - mn), fo = attn_ex2(o[4] - mn);
                v.x = v.x * f + o[0] * fo, v.y = v.y * f + o[1] * fo;
                v.z = v.z * f + o[2] * fo, v.w = v.w * f + o[3] * fo;
                l = l * f + o[5] * fo;
                top = mn;
              }
            }
            __syncthreads();
          }
          if (live && way == 0) {
            const float inv = l != 0.0f ? 1.0f / l : 0.0f;
            store(r, d, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
            if (d == 0) store_lse(r, top, l);
          }
        }
      }
    }
    // on to the next item (the loop's end leaves it past the share)
    at = seg_end;
    if (at < end) advance(cur, cur.strips - cur.strip);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

}  // namespace fp4
