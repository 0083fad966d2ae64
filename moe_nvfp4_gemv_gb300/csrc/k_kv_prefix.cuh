// k_kv_prefix.cuh -- the common beginning of fp4gemv_kv_attention_shared: the
// attention of all rows of a KV head (every sequence's new tokens, the heads of
// the group) over the tokens that the sequences share, on the 5th-generation
// tensor core.
//
// The mathematics is k_kv_attention.cuh's: weights 2^(s + log2 vs - m) of codes,
// f16 for the product with V, m following the maximum lazily, sums fp32; queries
// are exact f16 operands by a power of two for each row.  m moves by whole
// numbers here, so weights that are already made move exactly with it.  What is
// left per row and share are m, the sum of weights and the sums of V.  A last
// kernel joins them with those of each sequence's own tokens, which
// k_kv_attention.cuh leaves before this one starts.
//
// The beginning is cut at a multiple of 128 tokens that no sequence's first
// query comes before, so that nothing is masked here: every row sees every
// token.
//
// The layout.  Rows are the M side: blocks of 128 (a row per TMEM lane), tokens
// the N side of S = Q K^T and the K side of out = P V.  Codes become f16 on
// their way into shared memory (128-byte swizzle, blocks of 64 dims: K-major for
// K, the same bytes N-major for V), once for all rows.  P is written over S in
// tensor memory and is the A operand from there.  Two threads take a row, half a
// tile's tokens each; they compare their m once a unit.
//
// The work.  A CTA per SM.  Items are (KV head, two blocks of rows) and stand on
// a line, each as long as the beginning has tiles; the line is cut into equal
// shares.  Two slots, eight warps, an S and an accumulator each, take turns on
// the tensor core: one makes weights while the other's products run.  An item
// with two blocks gives each slot a block; with one, the slots take its tiles by
// turns.  Heads of 256 have room for one accumulator alone: one slot, with two S
// in front of it.  Seven warps move codes, a job of 16 tokens of K or V at a
// time; one warp issues the products.
//
// What bounds it.  64 sequences on 32768 common tokens, 64 heads on 8 of 128, E4M3: the call 98 to 101 us, of them 53 for the
// tiles here, 1.95 us for a tile of 128 tokens and 256 rows (the products alone 1.2 at the measured bf16 rate).  The chain
// from scores over weights to the next scores holds it: the tensor pipe is active 41 percent, and products and movers move
// some 70 bytes a cycle through shared memory, whose 128 Q K^T alone would take (a mapping that loads half lines still
// costs 10 percent).  The remaining 45: the own tokens' kernel 17 to 24, the start up to the first scores 6.5 (lengths,
// queries, pages, codes), the sums' way out 4, the join 5, launches.  7 sequences on 65536, heads of 256: 49 us, 1.0 us for
// 64 tokens, 0.7 of the HBM rate; 24 on 8191, 4 new tokens, INT8 heads of 64: 35, the chain of launches.
// Steps to it, us: weights in two passes over the scores by one thread a row, the join at the ends of the own tokens' items
// 177.7; the join's loads out of their loops (registers) 145; scores read once, movers by jobs 121; own tokens first, a kernel for the
// join 116; two threads a row 97.  Measured and not taken: tiles of 64 tokens with the queries in tensor memory for heads of 128 (112), 11
// movers (102), one thread for all steps of the products (100), 32 tokens at once per weigher (100), movers without the
// lanes' exchange of halves (102).
//
// Every wait is bounded.  After a failed one (the error word holds
// FP4_ERR_TIMEOUT) the waits that follow are skipped and the rows' sums are NaN.
#pragma once

#include "k_kv_attention.cuh"

namespace fp4 {

// The tiles of a beginning that the sequences share (k_kv_prefix.cuh) on their line, and what their sums are.
struct KvPrefixLine {
  int32_t* tokens;        // [1]: how many tokens were taken together
  float* sums;            // [piece][slot][128 rows][dim]
  float2* ml;             // [piece][slot][128 rows]: m, the sum of weights
  int ctas;
  int blocks;             // of 128 rows
  int items;              // of a KV head
  int slots;
  int tile;               // tokens
};

// A share of the line: pieces are numbered by CTA + item, which never repeats.
__host__ __device__ inline int prefix_share(int tiles, int ctas) { return (tiles + ctas - 1) / ctas; }

struct KvPrefixParams {
  const uint8_t* k_codes;
  const uint8_t* v_codes;
  const float* k_scale;
  const float* v_scale;
  const uint16_t* q;
  int64_t ldq;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* prefix_len;
  uint32_t* err;
  KvPrefixLine line;
  int B, max_blocks, num_blocks, block_log2;
  int kv_heads, group, q_len;
  int group_magic;  // KvAttnParams'
  int skip_tile;    // test hook: V of this tile of every CTA is not said to be there (-1: of none)
  int f16;
  float inv_rows;   // 1 / (q_len group)
  float sm_scale;
};

template <int kDim>
struct PrefixCfg {
  static constexpr int kTile = kDim == 256 ? 64 : 128;  // tokens
  // Queries lie in tensor memory where there is room: the products then read K alone from shared memory, whose bandwidth
  // they share with the movers.  (128 dims with room made by tiles of 64 tokens: 86 us instead of 72.5, 64 sequences on
  // 32768 tokens; 256 dims 41 instead of 43, 7 sequences on 65536.)
  static constexpr bool kQInTmem = kDim == 64 || kDim == 256;
  static constexpr int kSlots = kDim == 256 ? 1 : 2;    // accumulators
  static constexpr int kWeighers = kSlots * 256;        // two to a row, half a tile's tokens each
  static constexpr int kMovers = 7;                     // warps
  static constexpr int kThreads = kWeighers + kMovers * 32 + 32;
  static constexpr int kDimBlocks = (kDim + 63) / 64;
  static constexpr int kBlockBytes = kTile * 128;       // a tile's 64 dims
  static constexpr int kTileBytes = kDimBlocks * kBlockBytes;
  static constexpr int kStages = kDim == 256 ? 3 : kDim == 64 ? 4 : 2;
  static constexpr int kQBytes = kQInTmem ? 0 : kDimBlocks * 128 * 128;  // of a slot
  static constexpr int kGroups = kTile / 16;            // of 16 tokens: no page is smaller
  static constexpr int kHalf = kTile / 2;               // a weigher's tokens of a tile
  static constexpr int kParts = kHalf / 16;             // of 16 tokens, which share a page
  static constexpr int kSplit = (kDim / 32 + 1) / 2 * 32;  // a row's dims up to here are its first weigher's to move
  // Movers' jobs: 16 tokens of K or of V, K's of a tile first.
  static constexpr int kJobs = 2 * kGroups;
  static constexpr int kChunks = kDim / 32;             // of 16 codes, per lane and job
  // Q | K ring | V ring | 4 KB for each weighing warp (of Q, where it is here) | scales [stage][group of 16](K factor, log2 vs, 1 / vs, -) | what a row's
  // two weighers tell each other [slot][half][row]
  static constexpr int kKOff = kSlots * kQBytes;
  static constexpr int kVOff = kKOff + kStages * kTileBytes;
  static constexpr int kSpareOff = kVOff + kStages * kTileBytes;
  static constexpr int kScaleOff = kSpareOff + (kQInTmem ? kWeighers / 32 * 4096 : 0);
  static constexpr int kRowOff = kScaleOff + kStages * kGroups * 16;
  static constexpr int kSmem = 1024 + kRowOff + kSlots * 256 * 4;
  // TMEM columns: two S, the slots' queries, their sums
  static constexpr uint32_t kCols = 512, kQCol = 2 * kTile, kOCol = 512 - kSlots * kDim;
  static_assert(kSmem <= 232448, "shared memory");
  static_assert(kQCol + (kQInTmem ? kSlots * kDim / 2 : 0) <= kOCol, "room for all");
};

// kind::f16, f16 A and B, fp32 D; B K-major, or N-major
__host__ __device__ constexpr uint32_t idesc_f16_f32(uint32_t M, uint32_t N, bool b_n_major) {
  return (1u << 4) | (b_n_major ? 1u << 16 : 0u) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
// N-major operand of 2-byte elements in 128-byte lines, one for each k, swizzled in atoms of 8 lines; blocks of 64
// elements of N `block_bytes` apart.
__device__ __forceinline__ uint64_t sdesc_n_major_f16(uint32_t saddr, uint32_t block_bytes) {
  return (sdesc_sw128(saddr) & ~(static_cast<uint64_t>(0x3FFF) << 16)) | (static_cast<uint64_t>(block_bytes >> 4) << 16);
}

// 16 consecutive columns of the lane, on their way until tmem_here.
__device__ __forceinline__ void tmem_fetch16(uint32_t taddr, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(taddr)
      : "memory");
}
// (the values pass through the wait, so that nothing that uses them moves before it)
__device__ __forceinline__ void tmem_here(float (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
                 "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// Barrier `id` of two warps: whether v holds for any of their threads.
__device__ __forceinline__ bool named_any_of(int id, bool v) {
  uint32_t r;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 p, %2, 0; barrier.cta.red.or.pred.aligned q, %1, 64, p; selp.u32 %0, 1, 0, q; }"
      : "=r"(r)
      : "r"(id), "r"(static_cast<uint32_t>(v))
      : "memory");
  return r != 0;
}
// `columns` (a multiple of 16) sums of the lane times f.
inline __device__ __noinline__ void prefix_rescale(uint32_t cols, int columns, float f) {
#pragma unroll 1
  for (int c = 0; c < columns; c += 16) {
    float o[16];
    uint32_t w[16];
    tmem_fetch16(cols + c, o);
    tmem_here(o);
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(o[i] * f);
    tmem_st16(cols + c, w);
  }
  tmem_wait_st();
}
// `parts` times 16 weights (two to a column) of the lane times f, a power of two, as two f16 numbers: f itself may be below
// f16's range where a weight of 2^15 times f is not.
inline __device__ __noinline__ void prefix_rescale_weights(uint32_t cols, int parts, float f) {
  tmem_wait_st();  // (they may be on their way)
  const __half2 f0 = __float2half2_rn(fmaxf(f, 0x1p-24f)), f1 = __float2half2_rn(fminf(f * 0x1p24f, 1.0f));
#pragma unroll 1
  for (int c = 0; c < parts; ++c) {
    uint32_t w[8];
    tmem_ld8(cols + 8 * c, w);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __half2 x = __hmul2(__hmul2(*reinterpret_cast<const __half2*>(&w[i]), f0), f1);
      w[i] = *reinterpret_cast<const uint32_t*>(&x);
    }
    tmem_st8(cols + 8 * c, w);
  }
  tmem_wait_st();
}

template <int kDim, bool kInt8>
__global__ void __launch_bounds__(PrefixCfg<kDim>::kThreads, 1) kv_prefix_kernel(const KvPrefixParams p) {
  using C = PrefixCfg<kDim>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[4 * C::kStages + 2 * 3 + 2];
  __shared__ uint32_t tmem_slot;
  __shared__ int together_s, owner_s;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  uint8_t* const smem = smem_raw + (-smem_u32(smem_raw) & 1023u);  // (swizzle atoms of 1024 bytes)
  const uint32_t sm = smem_u32(smem), bar0 = smem_u32(bars);
  auto k_full = [&](int s) -> uint32_t { return bar0 + 8 * s; };
  auto k_empty = [&](int s) -> uint32_t { return bar0 + 8 * (C::kStages + s); };
  auto v_full = [&](int s) -> uint32_t { return bar0 + 8 * (2 * C::kStages + s); };
  auto v_empty = [&](int s) -> uint32_t { return bar0 + 8 * (3 * C::kStages + s); };
  auto scored = [&](int b) -> uint32_t { return bar0 + 8 * (4 * C::kStages + b); };       // S is there
  auto weighed = [&](int b) -> uint32_t { return bar0 + 8 * (4 * C::kStages + 2 + b); };  // P is there, S is read
  auto added = [&](int b) -> uint32_t { return bar0 + 8 * (4 * C::kStages + 4 + b); };    // the sums are
  const uint32_t q_there = bar0 + 8 * (4 * C::kStages + 6), idle = bar0 + 8 * (4 * C::kStages + 7);

  if (tid == 0) {
    pdl_launch_dependents();
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(k_full(s), C::kGroups);
      mbar_init(k_empty(s), 1);
      mbar_init(v_full(s), C::kGroups);
      mbar_init(v_empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(scored(b), 1);
      mbar_init(weighed(b), 256);
      mbar_init(added(b), 1);
    }
    mbar_init(q_there, C::kWeighers);
    mbar_init(idle, 1);
    mbar_fence_init();
  }
  // What this kernel reads was there before the one in front of it (the rest of the sequences) let it start; it is waited
  // for at the end, for those who follow.  Reads go to L2, since no wait has made the first-level cache's lines new.
  if (warp == 0) {
    int owner;
    const int n = attn_together<true>(__ldcg(p.prefix_len), p.lens, p.B, p.q_len, static_cast<int64_t>(p.max_blocks) << p.block_log2,
                                &owner);
    if (lane == 0) {
      together_s = n;
      owner_s = owner;
      if (blockIdx.x == 0) *p.line.tokens = n;
    }
  }
  __syncthreads();
  const int together = together_s, owner = owner_s;
  const int tiles_each = together / C::kTile, total = tiles_each * p.kv_heads * p.line.items;
  const int per = prefix_share(total, static_cast<int>(gridDim.x));
  const int begin = static_cast<int>(min(static_cast<int64_t>(per) * blockIdx.x, static_cast<int64_t>(total)));
  const int end = min(begin + per, total);
  if (begin >= end) {
    pdl_wait();
    return;
  }
  if (warp == C::kThreads / 32 - 1) {
    tmem_alloc(smem_u32(&tmem_slot), C::kCols);
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  bool ok = true;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (ok) ok = mbar_wait(bar, parity, p.err);
    __syncwarp();
  };
  const int rows = p.q_len * p.group, all_rows = p.B * rows;
  // segments: the parts of items in this CTA's share.  Units are a slot's turn on a tile: with two blocks of rows both
  // slots take every tile, else they take turns.
  auto paired = [&](int item) -> bool {
    return C::kSlots == 2 && 2 * (item % p.line.items) + 1 < p.line.blocks;
  };

  if (warp < C::kWeighers / 32) {
    // ---- weights and sums: two threads to a row of the slot's block, half a tile's tokens each ----
    const int slot = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter) << 21;
    const uint32_t o_cols = tmem + C::kOCol + slot * kDim + lanes, q_cols = tmem + C::kQCol + slot * (kDim / 2) + lanes;
    float* const row_said = reinterpret_cast<float*>(smem + C::kRowOff) + slot * 256;  // [half][row]
    const uint32_t q_base = sm + slot * C::kQBytes;
    const uint32_t spare = C::kQInTmem ? sm + C::kSpareOff + warp * 4096 : q_base + (warp & 7) * 4096;  // 32 rows of 128 bytes
    // the two warps of the same rows; whether `v` holds for any of them
    auto both_any = [&](bool v) -> bool { return named_any_of(2 + slot * 4 + quarter, v); };
    int turns[2] = {0, 0};  // units of each S before the segment
    int tile_no = 0;        // tiles before the segment
    for (int at = begin; at < end;) {
      const int item = at / tiles_each, seg_end = min(end, (item + 1) * tiles_each), tiles = seg_end - at;
      const bool both = paired(item);
      const int units = both ? 2 * tiles : tiles;
      const int head = item / p.line.items, number = item - head * p.line.items;
      const int block = C::kSlots == 1 ? number : 2 * number + (both ? slot : 0);
      // (no slot without work runs ahead to arrive twice in a segment's count)
      asm volatile("barrier.cta.sync 1, %0;" ::"n"(C::kWeighers) : "memory");
      // ---- queries: four lanes to a row and 32 dims, all loads under way at once; to tensor memory through shared memory,
      // since a lane there is a row ----
      float factor = fabsf(p.sm_scale) * 1.4426950408889634f;
      if (C::kSlots == 1 || units > slot) {
        const uint32_t flip = p.sm_scale < 0.0f ? 0x80008000u : 0u;  // (scores' factors are not negative)
        constexpr int kRuns = C::kSplit / 32;                        // of 32 dims, at most
        const int runs = half ? (kDim - C::kSplit) / 32 : kRuns, part = lane & 3;
        uint4 raw[kRuns][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int gr = block * 128 + quarter * 32 + t * 8 + (lane >> 2);
          int b = static_cast<int>(static_cast<float>(gr) * p.inv_rows);  // gr / rows (below 2^20: at most one off)
          b -= b * rows > gr;
          b += b * rows + rows <= gr;
          const int in = gr - b * rows, i = (in * p.group_magic) >> 16;
          const uint16_t* const src = p.q + (static_cast<int64_t>(b) * p.q_len + i) * p.ldq +
                                      (head * p.group + in - i * p.group) * kDim + half * C::kSplit + part * 8;
#pragma unroll
          for (int k = 0; k < kRuns; ++k) {
            raw[k][t] = make_uint4(0, 0, 0, 0);
            if (gr < all_rows && k < runs) raw[k][t] = __ldcg(reinterpret_cast<const uint4*>(src + k * 32));
          }
        }
        float down[4] = {1.0f, 1.0f, 1.0f, 1.0f};
        if (!p.f16) {  // 2^-e brings a row's largest to [2^14, 2^15): exact f16 values
          uint32_t* const tops = reinterpret_cast<uint32_t*>(row_said);
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < kRuns; ++k)
              top = __vmaxu2(top, __vmaxu2(__vmaxu2(raw[k][t].x & 0x7FFF7FFFu, raw[k][t].y & 0x7FFF7FFFu),
                                           __vmaxu2(raw[k][t].z & 0x7FFF7FFFu, raw[k][t].w & 0x7FFF7FFFu)));
            top = max(top & 0xFFFFu, top >> 16);
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            if (part == 0) tops[half * 128 + quarter * 32 + t * 8 + (lane >> 2)] = top;
          }
          both_any(false);
          auto exponent = [&](int r) -> int {
            const int field = static_cast<int>(max(tops[quarter * 32 + r], tops[128 + quarter * 32 + r]) >> 7);
            return field == 0 ? 0 : min(max(field - 127 - 14, -126), 126);
          };
#pragma unroll
          for (int t = 0; t < 4; ++t)
            down[t] = __uint_as_float(static_cast<uint32_t>(127 - exponent(t * 8 + (lane >> 2))) << 23);
          factor *= __uint_as_float(static_cast<uint32_t>(127 + exponent(lane)) << 23);
        }
#pragma unroll
        for (int k = 0; k < kRuns; ++k) {
          if (k >= runs) break;
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            uint32_t w[4] = {raw[k][t].x, raw[k][t].y, raw[k][t].z, raw[k][t].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (!p.f16)
                w[j] = pack_f16(__uint_as_float(w[j] << 16) * down[t], __uint_as_float(w[j] & 0xFFFF0000u) * down[t]);
              w[j] ^= flip;
            }
            const int r = t * 8 + (lane >> 2);
            if (C::kQInTmem) {
              sts128(spare + r * 64 + ((part ^ ((r >> 1) & 3)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
            } else {
              const int c = (half * C::kSplit + k * 32) / 8 + part;  // of 16 bytes
              sts128(q_base + (c >> 3) * (128 * 128) + (quarter * 32 + r) * 128 + (((c & 7) ^ (r & 7)) << 4),
                     make_uint4(w[0], w[1], w[2], w[3]));
            }
          }
          if (!C::kQInTmem) continue;
          __syncwarp();
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 v = lds128(spare + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4));
            w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
          }
          tmem_st16(q_cols + (half * C::kSplit + k * 32) / 2, w);
          __syncwarp();
        }
        if (C::kQInTmem) {
          tmem_wait_st();
          tc_fence_before();
        } else {
          fence_proxy_async_smem();
        }
      }
      mbar_arrive(q_there);
      // (the warp has a row that is one)
      const bool live = block * 128 + quarter * 32 < all_rows;
      // weights are 2^(x - m), x = s + log2 vs; m moves by whole numbers, so that weights already made move exactly; at a
      // unit's end a row's two weighers have the same
      float m = 0.0f, l = 0.0f;
      bool fresh = true;  // no m yet
      int last = -1;      // the slot's last unit's S
      for (int u = C::kSlots == 1 ? 0 : slot, k = 0; u < units; u += C::kSlots, ++k) {
        const int b = u & 1;
        const int tile = tile_no + (both ? u >> 1 : u), stage = tile % C::kStages;
        const int turn = turns[b] + (u >> 1);
        const uint32_t s_cols = tmem + b * C::kTile + half * C::kHalf + lanes;
        const uint32_t scales = sm + C::kScaleOff + stage * (C::kGroups * 16) + half * (C::kParts * 16);
        wait(scored(b), turn & 1);
        wait(v_full(stage), (tile / C::kStages) & 1);  // the scales
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
        const bool go = live && ok;
        const float m_before = m;
        const bool first = fresh;
        bool moved = false;
        if (go) {
          float x[2][16];
          tmem_fetch16(s_cols, x[0]);
#pragma unroll
          for (int c = 0; c < C::kParts; ++c) {
            float(&v)[16] = x[c & 1];
            tmem_here(v);
            if (c + 1 < C::kParts) tmem_fetch16(s_cols + 16 * (c + 1), x[(c + 1) & 1]);
            const uint4 g = lds128(scales + c * 16);
            const float f = factor * __uint_as_float(g.x);
            float sum;
            auto weigh = [&]() {
              const float base = __uint_as_float(g.y) - m;
              const uint64_t f2 = pair(f, f), base2 = pair(base, base);
              uint64_t total[2] = {0ull, 0ull};
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                const float2 e = unpair(fma2(pair(v[i], v[i + 1]), f2, base2));
                v[i] = attn_ex2(e.x), v[i + 1] = attn_ex2(e.y);
                total[(i >> 1) & 1] = add2(total[(i >> 1) & 1], pair(v[i], v[i + 1]));
              }
              const float2 t = unpair(add2(total[0], total[1]));
              sum = t.x + t.y;
            };
            if (!fresh) weigh();
            float inv_vs = __uint_as_float(g.z);
            const bool small = __uint_as_float(g.y) < kAttnSmallScale;  // (all lanes alike)
            // (a sum below f16's largest value has no weight above it)
            if (fresh || __any_sync(0xFFFFFFFFu, sum > 65000.0f || small)) {
              // (no values are held across the call: the scores are fetched again behind it)
              if (c + 1 < C::kParts) tmem_here(x[(c + 1) & 1]);
              tmem_fetch16(s_cols + 16 * c, v);
              tmem_here(v);
              float most = v[0];
#pragma unroll
              for (int i = 1; i < 16; ++i) most = fmaxf(most, v[i]);
              const float want = fmaxf(ceilf(fmaf(most, f, __uint_as_float(g.y)) - kAttnLift), kAttnFloor);
              const float now = fresh ? want : fmaxf(m, want);
              if (!fresh) {
                l = attn_halves(l, m - now);
                prefix_rescale_weights(s_cols, c, attn_ex2(m - now));
              }
              m = now;
              fresh = false;
              moved = true;
              tmem_fetch16(s_cols + 16 * c, v);
              tmem_here(v);
              if (c + 1 < C::kParts) tmem_fetch16(s_cols + 16 * (c + 1), x[(c + 1) & 1]);
              if (small) {
#pragma unroll
                for (int i = 0; i < 16; ++i) l += attn_ex2(fmaf(v[i], f, -m));
                inv_vs = 0.0f;
              }
              weigh();
            }
            l = fmaf(sum, inv_vs, l);
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = pack_f16(v[2 * i], v[2 * i + 1]);
            tmem_st8(s_cols + 8 * c, w);  // (over columns that are read)
          }
          tmem_wait_st();
        }
        if (both_any(moved)) {
          // one of the row's weighers has another m: the larger one for both
          row_said[half * 128 + row] = m;
          both_any(false);
          const float now = fmaxf(m, row_said[(half ^ 1) * 128 + row]);
          if (go) {
            l = attn_halves(l, m - now);
            prefix_rescale_weights(s_cols, C::kParts, attn_ex2(m - now));
            if (!first) {
              if (C::kSlots == 1) {  // (one accumulator for both S: the other's sums may be under way)
                wait(added(b ^ 1), (turns[b ^ 1] + ((u - 1) >> 1)) & 1);
                tc_fence_after();
              }
              prefix_rescale(o_cols + half * C::kSplit, half ? kDim - C::kSplit : C::kSplit, attn_ex2(m_before - now));
            }
          }
          m = now;
        }
        tc_fence_before();
        if (ok) mbar_arrive(weighed(b));
        last = b;
      }
      // ---- the segment's end: the piece's sums ----
      const int64_t piece = (static_cast<int64_t>(blockIdx.x) + item) * C::kSlots + slot;
      if (last >= 0) {
        const int n_last = last == 0 ? (units + 1) / 2 : units / 2;
        wait(added(last), (turns[last] + n_last - 1) & 1);
      }
      ok = __all_sync(0xFFFFFFFFu, ok);
      tc_fence_after();
      if (half == 1) row_said[128 + row] = ok ? l : __int_as_float(0x7FC00000);
      both_any(false);
      if (live) {
        float* const sums = p.line.sums + (piece * 128 + quarter * 32) * kDim;
        if (last >= 0) {
#pragma unroll 1
          for (int c = half ? C::kSplit : 0; c < (half ? kDim : C::kSplit); c += 32) {
            float o[2][16];
            tmem_fetch16(o_cols + c, o[0]);
            tmem_fetch16(o_cols + c + 16, o[1]);
            tmem_here(o[0]);
            tmem_here(o[1]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float* v = &o[i >> 2][4 * (i & 3)];
              sts128(spare + lane * 128 + ((i ^ (lane & 7)) << 4),
                     make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r = i * 4 + (lane >> 3);
              const uint4 v = lds128(spare + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
              __stcg(reinterpret_cast<uint4*>(sums + r * kDim + c) + (lane & 7), v);
            }
            __syncwarp();
          }
        }
        if (half == 0)
          __stcg(p.line.ml + piece * 128 + row,
                 make_float2(fresh ? kAttnFloor : m, ok ? l + row_said[128 + row] : __int_as_float(0x7FC00000)));
      }
      tc_fence_before();
      turns[0] += (units + 1) / 2;
      turns[1] += units / 2;
      tile_no += tiles;
      at = seg_end;
    }
  } else if (warp < C::kWeighers / 32 + C::kMovers) {
    // ---- movers: codes to f16, a job of 16 tokens at a time, the next one's loads on their way ----
    const int first = warp - C::kWeighers / 32, jobs = (end - begin) * C::kJobs;
    const int32_t* const table = p.table + static_cast<int64_t>(owner) * p.max_blocks;
    // Lane l looks up the warp's l-th next job: its strip of 16 tokens in the cache, -1 past the share, -2 for a bad page.
    int looked = first + lane * C::kMovers;
    auto look_up = [&]() -> int {
      int found = -1;
      if (looked < jobs) {
        const int at = begin + looked / C::kJobs, item = at / tiles_each, head = item / p.line.items;
        const int strip = (at - item * tiles_each) * C::kGroups + looked % C::kGroups, per_page = p.block_log2 - 4;
        const int id = __ldcg(table + (strip >> per_page));
        found = id >= 0 && id < p.num_blocks
                    ? ((id * p.kv_heads + head) << per_page) + (strip & ((1 << per_page) - 1))
                    : -2;
      }
      looked += 32 * C::kMovers;
      return found;
    };
    int batch = look_up(), batch_next = look_up();
    struct Job {
      uint4 raw[C::kChunks];
      float scale;  // lane 0: of K, lane 1: of V
      int strip;
    };
    // the strip of the warp's n-th job, n within this batch or the next
    auto strip_of = [&](int n, int now) -> int {
      return __shfl_sync(0xFFFFFFFFu, (n ^ now) & 32 ? batch_next : batch, n & 31);
    };
    auto source = [&](int n, int strip) -> const uint8_t* {
      const bool v = (first + n * C::kMovers) % C::kJobs >= C::kGroups;
      return (v ? p.v_codes : p.k_codes) + static_cast<int64_t>(strip) * (16 * kDim);
    };
    auto load = [&](Job& job, int n, int now) {
      job.strip = strip_of(n, now);
      job.scale = 0.0f;
      const uint8_t* const src = source(n, max(job.strip, 0)) + lane * 16;
#pragma unroll
      for (int i = 0; i < C::kChunks; ++i) {
        job.raw[i] = make_uint4(0, 0, 0, 0);
        if (job.strip >= 0) job.raw[i] = __ldcg(reinterpret_cast<const uint4*>(src + i * 512));
      }
      if (job.strip >= 0 && lane < 2) job.scale = __ldcg((lane ? p.v_scale : p.k_scale) + (job.strip >> (p.block_log2 - 4)));
      // further on, to L2: the job after three more
      const int far = strip_of(n + 3, now);
      if (far >= 0 && lane < kDim / 8) asm volatile("prefetch.global.L2 [%0];" ::"l"(source(n + 3, far) + lane * 128));
    };
    auto convert = [&](const Job& job, int n) {
      const int j = first + n * C::kMovers, tile = j / C::kJobs, kind = j % C::kJobs, stage = tile % C::kStages;
      const bool v = kind >= C::kGroups;
      const int group = kind % C::kGroups;
      if (tile >= C::kStages) wait(v ? v_empty(stage) : k_empty(stage), (tile / C::kStages - 1) & 1);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) return;
      const uint32_t dst = sm + (v ? C::kVOff : C::kKOff) + stage * C::kTileBytes;
      constexpr int kCols = kDim / 16;
#pragma unroll
      for (int i = 0; i < C::kChunks; ++i) {
        const int chunk = lane + 32 * i, r = chunk / kCols, c = chunk - r * kCols, row = group * 16 + r;
        const uint32_t w[4] = {job.raw[i].x, job.raw[i].y, job.raw[i].z, job.raw[i].w};
        const uint4 lo = make_uint4(codes2_lo<kInt8>(w[0]), codes2_hi<kInt8>(w[0]), codes2_lo<kInt8>(w[1]),
                                    codes2_hi<kInt8>(w[1]));
        const uint4 hi = make_uint4(codes2_lo<kInt8>(w[2]), codes2_hi<kInt8>(w[2]), codes2_lo<kInt8>(w[3]),
                                    codes2_hi<kInt8>(w[3]));
        // (neighbours whose chunks lie in different blocks of 64 dims store their halves in the other order: no two of
        // eight lanes meet a bank)
        const bool swap = (c >> 2) & 1;
        const uint32_t to = dst + (c >> 2) * C::kBlockBytes + row * 128 + (((2 * (c & 3)) ^ (r & 7)) << 4);
        sts128(swap ? to ^ 16 : to, swap ? hi : lo);
        sts128(swap ? to : to ^ 16, swap ? lo : hi);
      }
      if (v) {
        const uint32_t at = sm + C::kScaleOff + stage * (C::kGroups * 16) + group * 16;
        if (lane == 0) {
          stsf(at, job.scale);
          if (job.strip < 0) raise_error(p.err, FP4_ERR_BADIDX);
        } else if (lane == 1) {
          const float lv = attn_lg2(fmaxf(job.scale, 7.888609052210118e-31f));
          stsf(at + 4, lv);
          stsf(at + 8, attn_ex2(-lv));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && !(v && tile == p.skip_tile)) mbar_arrive(v ? v_full(stage) : k_full(stage));
    };
    const int count = first < jobs ? (jobs - first + C::kMovers - 1) / C::kMovers : 0;  // of the warp
    Job job[2];
    if (count > 0) load(job[0], 0, 0);
    for (int n = 0; n < count; n += 2) {
      if (n > 0 && (n & 31) == 0) {
        batch = batch_next;
        batch_next = look_up();
      }
      load(job[1], n + 1, n);
      convert(job[0], n);
      load(job[0], n + 2, n);
      if (n + 1 < count) convert(job[1], n + 1);
      if (!ok) break;
    }
  } else {
    // ---- MMA warp ----
    constexpr uint32_t id_s = idesc_f16_f32(128, C::kTile, false), id_o = idesc_f16_f32(128, kDim, true);
    int turns[2] = {0, 0}, tile_no = 0, segment = 0;
    for (int at = begin; at < end; ++segment) {
      const int item = at / tiles_each, seg_end = min(end, (item + 1) * tiles_each), tiles = seg_end - at;
      const bool both = paired(item);
      const int units = both ? 2 * tiles : tiles;
      wait(q_there, segment & 1);
      tc_fence_after();
      auto score = [&](int u) {
        const int b = u & 1, tile = tile_no + (both ? u >> 1 : u), stage = tile % C::kStages;
        wait(k_full(stage), (tile / C::kStages) & 1);
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
        if (ok && elect_one()) {
          const int q_slot = C::kSlots == 2 ? b : 0;
          const uint64_t k_desc = sdesc_sw128(sm + C::kKOff + stage * C::kTileBytes);
          const uint64_t q_desc = sdesc_sw128(sm + q_slot * C::kQBytes);
          const uint32_t q = tmem + C::kQCol + q_slot * (kDim / 2);
#pragma unroll
          for (int k = 0; k < kDim / 16; ++k) {
            const uint64_t from = k_desc + (k >> 2) * (C::kBlockBytes >> 4) + 2 * (k & 3);
            if (C::kQInTmem) mma_ts(tmem + b * C::kTile, q + 8 * k, from, id_s, k > 0);
            else mma_ss(tmem + b * C::kTile, q_desc + (k >> 2) * (128 * 128 >> 4) + 2 * (k & 3), from, id_s, k > 0);
          }
          mma_commit(scored(b));
          if (!both || b == 1) mma_commit(k_empty(stage));
        }
        __syncwarp();
      };
      score(0);
      if (units > 1) score(1);
      for (int u = 0; u < units; ++u) {
        const int b = u & 1, tile = tile_no + (both ? u >> 1 : u), stage = tile % C::kStages;
        const uint64_t v_desc = sdesc_n_major_f16(sm + C::kVOff + stage * C::kTileBytes, C::kBlockBytes);
        const uint32_t o = tmem + C::kOCol + (C::kSlots == 2 ? b : 0) * kDim;
        const bool more = C::kSlots == 2 ? u > 1 : u > 0;  // (there are sums to add to)
        wait(v_full(stage), (tile / C::kStages) & 1);
        wait(weighed(b), (turns[b] + (u >> 1)) & 1);
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
        if (ok && elect_one()) {
#pragma unroll
          for (int k = 0; k < C::kTile / 16; ++k)  // 16 tokens each, 2048 bytes; P of a half lies where its S did
            mma_ts(o, tmem + b * C::kTile + k / C::kParts * C::kHalf + 8 * (k % C::kParts), v_desc + 128 * k, id_o, more || k > 0);
          mma_commit(added(b));
          if (!both || b == 1) mma_commit(v_empty(stage));
        }
        __syncwarp();
        if (u + 2 < units) score(u + 2);
      }
      turns[0] += (units + 1) / 2;
      turns[1] += units / 2;
      tile_no += tiles;
      at = seg_end;
    }
    if (elect_one()) mma_commit(idle);
    __syncwarp();
    mbar_wait(idle, 0, p.err);
  }
  __syncthreads();
  if (warp == C::kThreads / 32 - 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
  pdl_wait();
}

struct KvJoinParams {
  KvPrefixLine line;
  const float* sums;  // of the sequences' own tokens (KvAttnRestParams)
  const float2* ml;
  const int32_t* lens;
  uint16_t* out;
  int64_t ldo;
  float* lse;
  int B, kv_heads, group, q_len, f16;
};
constexpr int kJoinThreads = 256;

// Own sums and the pieces of the beginning's to outputs: four dims of a row are a cell, of one thread or of kWays that
// share its pieces out (a warp's lanes by pieces, then by cells), kBatch pieces' loads of each under way.
template <int kDim, int kWays>
__global__ void __launch_bounds__(kJoinThreads) kv_join_kernel(const KvJoinParams p) {
  constexpr int kBatch = 8, kCells = kDim / 4;
  if (threadIdx.x == 0) pdl_launch_dependents();
  pdl_wait();
  const KvPrefixLine& line = p.line;
  const int rows = p.q_len * p.group, all_rows = p.B * rows;
  constexpr int kPerWarp = 32 / kWays;
  const int lane = threadIdx.x & 31, way = lane / kPerWarp;
  const int64_t x = (static_cast<int64_t>(blockIdx.x) * (kJoinThreads / 32) + (threadIdx.x >> 5)) * kPerWarp + lane % kPerWarp;
  const bool live = x < static_cast<int64_t>(all_rows) * p.kv_heads * kCells;
  const int64_t at = live ? x / kCells : 0;
  const int d = live ? static_cast<int>(x - at * kCells) * 4 : 0;
  const int head = static_cast<int>(at / all_rows), all = static_cast<int>(at - static_cast<int64_t>(head) * all_rows);
  const int b = all / rows, in = all - b * rows, i = in / p.group;
  // (all under way at once; what an empty sequence's row says is not looked at)
  const int length = __ldg(p.lens + b), taken = __ldcg(line.tokens);
  const float2 own = __ldcg(p.ml + at);
  const float4 sums_own = __ldcg(reinterpret_cast<const float4*>(p.sums + at * kDim + d));
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float top = kAttnFloor, l = 0.0f;
  if (length > 0) {
    if (way == 0) v = sums_own, top = own.x, l = own.y;
    const int tiles = taken / line.tile;
    if (tiles > 0) {
      const int per = prefix_share(tiles * p.kv_heads * line.items, line.ctas), block = all >> 7;
      const int number = line.slots == 1 ? block : block >> 1;
      const bool both = line.slots == 2 && 2 * number + 1 < line.blocks;  // (else: slots that took the tiles by turns)
      const int item = head * line.items + number, c0 = item * tiles / per, c1 = ((item + 1) * tiles - 1) / per;
      const int64_t piece = ((static_cast<int64_t>(c0) + item) * line.slots + (both ? block & 1 : 0)) * 128 + (all & 127);
      const int step = both ? 2 : 1, pieces = (c1 - c0 + 1) * (line.slots == 1 || both ? 1 : 2);
      const float2* const ml = line.ml + piece;
      const float* const sums = line.sums + piece * kDim + d;
#pragma unroll 1
      for (int k = way; k < pieces; k += kBatch * kWays) {
        float2 cm[kBatch];
        float4 a[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int kk = k + j * kWays;
          cm[j] = make_float2(kAttnFloor, 0.0f);
          a[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (kk < pieces) {
            cm[j] = __ldcg(ml + static_cast<int64_t>(kk) * step * 128);
            a[j] = __ldcg(reinterpret_cast<const float4*>(sums + static_cast<int64_t>(kk) * step * (128 * kDim)));
          }
        }
        float mn = top;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) mn = fmaxf(mn, cm[j].x);
        const float fall = attn_ex2(top - mn);
        v.x *= fall, v.y *= fall, v.z *= fall, v.w *= fall;
        l = attn_halves(l, top - mn);
        top = mn;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          if (cm[j].y == 0.0f) a[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);  // (a slot that had no tile wrote no sums)
          const float f = attn_ex2(cm[j].x - mn);
          v.x = fmaf(a[j].x, f, v.x), v.y = fmaf(a[j].y, f, v.y);
          v.z = fmaf(a[j].z, f, v.z), v.w = fmaf(a[j].w, f, v.w);
          l += attn_halves(cm[j].y, cm[j].x - mn);
        }
      }
    }
  }
#pragma unroll
  for (int o = kPerWarp; o < 32; o <<= 1) {
    const float to = __shfl_xor_sync(0xFFFFFFFFu, top, o), lo = __shfl_xor_sync(0xFFFFFFFFu, l, o);
    const float4 u = make_float4(__shfl_xor_sync(0xFFFFFFFFu, v.x, o), __shfl_xor_sync(0xFFFFFFFFu, v.y, o),
                                 __shfl_xor_sync(0xFFFFFFFFu, v.z, o), __shfl_xor_sync(0xFFFFFFFFu, v.w, o));
    const float mn = fmaxf(top, to), f = attn_ex2(top - mn), fo = attn_ex2(to - mn);
    v.x = v.x * f + u.x * fo, v.y = v.y * f + u.y * fo, v.z = v.z * f + u.z * fo, v.w = v.w * f + u.w * fo;
    l = attn_halves(l, top - mn) + attn_halves(lo, to - mn);
    top = mn;
  }
  if (!live || way != 0) return;
  const int64_t token = static_cast<int64_t>(b) * p.q_len + i;
  const int head_out = head * p.group + in - i * p.group;
  attn_put(v, top, l, p.out + token * p.ldo + head_out * kDim + d,
           d == 0 && p.lse ? p.lse + token * (p.kv_heads * p.group) + head_out : nullptr, p.f16);
}

}  // namespace fp4
