// k_kv_prefix.cuh -- the common beginning of fp4gemv_kv_attention_shared: the
// attention of all rows of a KV head (every sequence's new tokens, the heads of
// the group) over the tokens that the sequences share, on the 5th-generation
// tensor core.
//
// The mathematics is k_kv_attention.cuh's: weights 2^(s + log2 vs - m) of codes,
// f16 for the product with V, m following the maximum lazily, sums fp32; queries
// are exact f16 operands by a power of two for each row.  What is left per row
// are m, the sum of weights and the sums of V, which k_kv_attention.cuh joins
// with those of the sequence's own tokens.
//
// The beginning is cut at a multiple of 128 tokens that no sequence's first
// query comes before, so that nothing is masked here: every row sees every
// token.
//
// The layout.  Rows are the M side: blocks of 128 (a row per TMEM lane and per
// thread, so a row's maximum and sum are registers), tokens the N side of
// S = Q K^T and the K side of out = P V.  Codes become f16 on their way into
// shared memory (128-byte swizzle, blocks of 64 dims: K-major for K, the same
// bytes M-major for V), once for all rows.  P is written over S in tensor memory
// and is the A operand from there.
//
// The work.  A CTA per SM.  Items are (KV head, two blocks of rows) and stand on
// a line, each as long as the beginning has tiles; the line is cut into equal
// shares.  Two slots, a warpgroup, an S and an accumulator each, take turns on
// the tensor core: one makes weights while the other's products run.  An item
// with two blocks gives each slot a block; with one, the slots take its tiles by
// turns.  Heads of 256 have room for one accumulator alone: one warpgroup, with
// the two S in front of it.
//
// Every wait is bounded.  After a failed one (the error word holds
// FP4_ERR_TIMEOUT) the waits that follow are skipped and the rows' sums are NaN.
#pragma once

#include "k_kv_attention.cuh"

namespace fp4 {

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
  int32_t* tokens;  // KvPrefixLine's
  KvPrefixLine line;
  int B, max_blocks, num_blocks, block_log2;
  int kv_heads, group, q_len;
  int f16;
  float sm_scale;
};

template <int kDim>
struct PrefixCfg {
  static constexpr int kTile = kDim == 256 ? 64 : 128;  // tokens
  static constexpr int kSlots = kDim == 256 ? 1 : 2;    // accumulators
  static constexpr int kWeighers = kSlots * 128;
  static constexpr int kMovers = 256;                   // 128 threads for K, 128 for V
  static constexpr int kThreads = kWeighers + kMovers + 32;
  static constexpr int kDimBlocks = (kDim + 63) / 64;
  static constexpr int kBlockBytes = kTile * 128;       // a tile's 64 dims
  static constexpr int kTileBytes = kDimBlocks * kBlockBytes;
  static constexpr int kQBytes = kDimBlocks * 128 * 128;
  static constexpr int kStages = 2;
  static constexpr int kGroups = kTile / 16;            // of 16 tokens: no page is smaller
  // Q | K ring | V ring | scales [stage][K factor, log2 vs, 1 / vs][group of 16] | row factors
  static constexpr int kKOff = kSlots * kQBytes;
  static constexpr int kVOff = kKOff + kStages * kTileBytes;
  static constexpr int kScaleOff = kVOff + kStages * kTileBytes;
  static constexpr int kRowOff = kScaleOff + kStages * 3 * 8 * 4;
  static constexpr int kSmem = 1024 + kRowOff + kSlots * 128 * 4;
  static constexpr uint32_t kCols = 512;                // TMEM: S of 128 columns twice, accumulators from 256 on
  static constexpr int kChunks = kTile * (kDim / 16) / 128;  // of 16 codes, per mover
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

template <int kDim, bool kInt8>
__global__ void __launch_bounds__(PrefixCfg<kDim>::kThreads, 1) kv_prefix_kernel(const KvPrefixParams p) {
  using C = PrefixCfg<kDim>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[4 * C::kStages + 2 * 3 + 2];
  __shared__ uint32_t tmem_slot;
  __shared__ int least, first_alive;
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
      mbar_init(k_full(s), 128);
      mbar_init(k_empty(s), 1);
      mbar_init(v_full(s), 128);
      mbar_init(v_empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(scored(b), 1);
      mbar_init(weighed(b), 128);
      mbar_init(added(b), 1);
    }
    mbar_init(q_there, C::kWeighers);
    mbar_init(idle, 1);
    mbar_fence_init();
    least = 0x7FFFFFFF;
    first_alive = 0x7FFFFFFF;
  }
  pdl_wait();
  __syncthreads();
  // ---- how many tokens are taken together, and whose pages hold them ----
  {
    const int64_t cap = static_cast<int64_t>(p.max_blocks) << p.block_log2;
    int low = 0x7FFFFFFF, who = 0x7FFFFFFF;
    for (int b = tid; b < p.B; b += C::kThreads) {
      const int raw = __ldg(p.lens + b);
      const int n = raw < 0 ? 0 : raw > cap ? static_cast<int>(cap) : raw;
      if (n > 0) {
        low = min(low, n - p.q_len);  // (before the first query: every row sees them, and some token is left)
        who = min(who, b);
      }
    }
    low = __reduce_min_sync(0xFFFFFFFFu, low);
    who = __reduce_min_sync(0xFFFFFFFFu, who);
    if (lane == 0 && who != 0x7FFFFFFF) {
      atomicMin(&least, low);
      atomicMin(&first_alive, who);
    }
  }
  __syncthreads();
  const int owner = first_alive;
  const int together = owner == 0x7FFFFFFF ? 0 : max(min(least, __ldg(p.prefix_len)), 0) & ~127;
  if (blockIdx.x == 0 && tid == 0) *p.tokens = together;
  const int tiles_each = together / C::kTile, total = tiles_each * p.kv_heads * p.line.items;
  const int per = prefix_share(total, static_cast<int>(gridDim.x));
  const int begin = static_cast<int>(min(static_cast<int64_t>(per) * blockIdx.x, static_cast<int64_t>(total)));
  const int end = min(begin + per, total);
  if (begin >= end) return;
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
    // ---- weights and sums: thread = row of the slot's block ----
    const int slot = warp >> 2, row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    const uint32_t o_cols = tmem + 256 + slot * 128 + lanes;
    float* const row_factor = reinterpret_cast<float*>(smem + C::kRowOff) + slot * 128;
    const uint32_t q_base = sm + slot * C::kQBytes;
    int turns[2] = {0, 0};  // units of each S before the segment
    int tile_no = 0;        // tiles before the segment
    for (int at = begin; at < end;) {
      const int item = at / tiles_each, seg_end = min(end, (item + 1) * tiles_each), tiles = seg_end - at;
      const bool pair = paired(item);
      const int units = pair ? 2 * tiles : tiles;
      const int head = item / p.line.items, number = item - head * p.line.items;
      const int block = C::kSlots == 1 ? number : 2 * number + (pair ? slot : 0);
      const bool works = C::kSlots == 1 || units > slot;
      // (no slot without work runs ahead to arrive twice in a segment's count)
      asm volatile("barrier.cta.sync 1, %0;" ::"n"(C::kWeighers) : "memory");
      // ---- queries: eight lanes to a row, four rows of the warp at a time ----
      if (works) {
        const float sign = p.sm_scale < 0.0f ? -1.0f : 1.0f;
        constexpr int kQChunks = kDim / 8;              // of 16 bytes
        constexpr int kPer = (kQChunks + 7) / 8;        // of a lane
#pragma unroll 2
        for (int r0 = 0; r0 < 32; r0 += 4) {
          const int r = (warp & 3) * 32 + r0 + (lane >> 3), part = lane & 7;
          const int gr = block * 128 + r;
          uint4 raw[kPer];
#pragma unroll
          for (int k = 0; k < kPer; ++k) raw[k] = make_uint4(0, 0, 0, 0);
          if (gr < all_rows) {
            const int b = gr / rows, in = gr - b * rows, i = in / p.group;
            const uint16_t* src = p.q + (static_cast<int64_t>(b) * p.q_len + i) * p.ldq +
                                  (head * p.group + in - i * p.group) * kDim;
#pragma unroll
            for (int k = 0; k < kPer; ++k)
              if (part + 8 * k < kQChunks) raw[k] = __ldg(reinterpret_cast<const uint4*>(src) + part + 8 * k);
          }
          float factor = fabsf(p.sm_scale) * 1.4426950408889634f;
          if (!p.f16) {  // 2^-e brings the largest to [2^14, 2^15): exact f16 values
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < kPer; ++k)
              top = __vmaxu2(top, __vmaxu2(__vmaxu2(raw[k].x & 0x7FFF7FFFu, raw[k].y & 0x7FFF7FFFu),
                                           __vmaxu2(raw[k].z & 0x7FFF7FFFu, raw[k].w & 0x7FFF7FFFu)));
            top = max(top & 0xFFFFu, top >> 16);
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            const int field = static_cast<int>(top >> 7);
            const int e = field == 0 ? 0 : min(max(field - 127 - 14, -126), 126);
            const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
              uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
              for (int j = 0; j < 4; ++j)
                w[j] = pack_f16(__uint_as_float(w[j] << 16) * down, __uint_as_float(w[j] & 0xFFFF0000u) * down);
              raw[k] = make_uint4(w[0], w[1], w[2], w[3]);
            }
            factor *= __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
          }
          const uint32_t flip = sign < 0.0f ? 0x80008000u : 0u;  // (scores' factors are not negative)
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
            const int c = part + 8 * k;
            if (c < kQChunks)
              sts128(q_base + (c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                     make_uint4(raw[k].x ^ flip, raw[k].y ^ flip, raw[k].z ^ flip, raw[k].w ^ flip));
          }
          if (part == 0) row_factor[r] = factor;
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
      const float factor = row_factor[row];
      mbar_arrive(q_there);
      // (the warp has a row that is one)
      const bool live = block * 128 + (row & ~31) < all_rows;
      float m = kAttnFloor, l = 0.0f;
      int last = -1;  // the slot's last unit's S
      for (int u = C::kSlots == 1 ? 0 : slot, k = 0; u < units; u += C::kSlots, ++k) {
        const int b = u & 1;
        const int tile = tile_no + (pair ? u >> 1 : u), stage = tile % C::kStages;
        const int turn = turns[b] + (u >> 1);
        const uint32_t s_cols = tmem + b * 128 + lanes;
        wait(scored(b), turn & 1);
        wait(v_full(stage), (tile / C::kStages) & 1);  // the scales
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
        if (live && ok) {
          const float* const scales = reinterpret_cast<const float*>(smem + C::kScaleOff) + stage * 24;
          float top = kAttnFloor;
#pragma unroll
          for (int c = 0; c < C::kTile / 32; ++c) {
            float x[32];
            tmem_get32(s_cols + 32 * c, x);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float most = x[16 * h];
#pragma unroll
              for (int i = 1; i < 16; ++i) most = fmaxf(most, x[16 * h + i]);
              top = fmaxf(top, fmaf(most, factor * scales[2 * c + h], scales[8 + 2 * c + h]));
            }
          }
          if (__any_sync(0xFFFFFFFFu, top - m > kAttnLift + kAttnSlack)) {
            const float now = fmaxf(m, top - kAttnLift), fall = attn_ex2(m - now);
            l = attn_lower<true>(l, m - now);
            m = now;
            if (k > 0) {
              // (one accumulator for both S: the other's sums may be under way)
              if (C::kSlots == 1) {
                wait(added(b ^ 1), (turns[b ^ 1] + ((u - 1) >> 1)) & 1);
                tc_fence_after();
              }
#pragma unroll 1
              for (int c = 0; c < kDim; c += 32) {
                float o[32];
                uint32_t w[16];
                tmem_get32(o_cols + c, o);
#pragma unroll
                for (int h = 0; h < 32; h += 16) {
#pragma unroll
                  for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(o[h + i] * fall);
                  tmem_st16(o_cols + c + h, w);
                }
              }
              tmem_wait_st();
            }
          }
#pragma unroll
          for (int c = 0; c < C::kTile / 32; ++c) {
            float x[32];
            tmem_get32(s_cols + 32 * c, x);
            uint32_t w[16];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float f = factor * scales[2 * c + h], base = scales[8 + 2 * c + h] - m;
              float part = 0.0f;
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                const float a = attn_ex2(fmaf(x[16 * h + i], f, base)), d = attn_ex2(fmaf(x[16 * h + i + 1], f, base));
                part += a + d;
                w[8 * h + i / 2] = pack_f16(a, d);
              }
              l = fmaf(part, scales[16 + 2 * c + h], l);
            }
            tmem_st16(s_cols + 16 * c, w);  // (over columns that are read)
          }
          tmem_wait_st();
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
      if (live) {
        float* const sums = p.line.sums + (piece * 128 + (warp & 3) * 32) * kDim;
        const uint32_t spare = q_base + (warp & 3) * 4096;  // (the queries are of no use any more) 32 rows of 32 floats
        if (last >= 0) {
#pragma unroll 1
          for (int c = 0; c < kDim; c += 32) {
            float o[32];
            tmem_get32(o_cols + c, o);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              sts128(spare + lane * 128 + ((i ^ (lane & 7)) << 4),
                     make_uint4(__float_as_uint(o[4 * i]), __float_as_uint(o[4 * i + 1]), __float_as_uint(o[4 * i + 2]),
                                __float_as_uint(o[4 * i + 3])));
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
        __stcg(p.line.ml + piece * 128 + row, make_float2(m, ok ? l : __int_as_float(0x7FC00000)));
      }
      tc_fence_before();
      turns[0] += (units + 1) / 2;
      turns[1] += units / 2;
      tile_no += tiles;
      at = seg_end;
    }
  } else if (warp < (C::kWeighers + C::kMovers) / 32) {
    // ---- movers: 128 threads for K, 128 for V: codes to f16 ----
    const bool v = warp >= (C::kWeighers + 128) / 32;
    const int t = (tid - C::kWeighers) & 127;
    const uint8_t* const codes = v ? p.v_codes : p.k_codes;
    const uint32_t ring = sm + (v ? C::kVOff : C::kKOff);
    const int32_t* const table = p.table + static_cast<int64_t>(owner) * p.max_blocks;
    const int64_t head_bytes = static_cast<int64_t>(kDim) << p.block_log2;
    constexpr int kCols = kDim / 16;
    // lane l looks up the page of the tile's tokens 16 (l mod 8): -1 past the share, -2 where there is none
    auto look_up = [&](int at) -> int {
      if (at >= end) return -1;
      const int token = (at % tiles_each) * C::kTile + 16 * (lane & (C::kGroups - 1));
      const int id = __ldg(table + (token >> p.block_log2));
      return id >= 0 && id < p.num_blocks ? id : -2;
    };
    // the page and head of a tile's group of 16 tokens, and where it begins there
    auto place_of = [&](int at, int id, int group16) -> const uint8_t* {
      const int token = (at % tiles_each) * C::kTile + 16 * group16, head = at / tiles_each / p.line.items;
      return codes + (static_cast<int64_t>(id) * p.kv_heads + head) * head_bytes +
             (token & ((1 << p.block_log2) - 1)) * kDim;
    };
    uint4 raw[C::kChunks];
    auto load = [&](int at, int ids) {
#pragma unroll
      for (int i = 0; i < C::kChunks; ++i) {
        const int chunk = t + 128 * i, r = chunk / kCols, c = chunk - r * kCols;
        const int id = __shfl_sync(0xFFFFFFFFu, ids, r >> 4);
        raw[i] = make_uint4(0, 0, 0, 0);
        if (id >= 0) raw[i] = __ldg(reinterpret_cast<const uint4*>(place_of(at, id, r >> 4) + (r & 15) * kDim) + c);
      }
    };
    auto prefetch = [&](int at, int ids) {  // 128 bytes for each thread, as far as the tile has them
      const int line = t, r = line * 128 / kDim;
      const int id = __shfl_sync(0xFFFFFFFFu, ids, (r >> 4) & 7);
      if (id >= 0 && r < C::kTile)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(place_of(at, id, r >> 4) + (r & 15) * kDim + line * 128 % kDim));
    };
    int ids[4] = {look_up(begin), look_up(begin + 1), look_up(begin + 2), look_up(begin + 3)};
    load(begin, ids[0]);
    prefetch(begin + 1, ids[1]);
    prefetch(begin + 2, ids[2]);
    for (int at = begin, tile = 0; at < end; ++at, ++tile) {
      const int stage = tile % C::kStages;
      const int far = look_up(at + 4);
      if (tile >= C::kStages) wait(v ? v_empty(stage) : k_empty(stage), (tile / C::kStages - 1) & 1);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      const uint32_t dst = ring + stage * C::kTileBytes;
#pragma unroll
      for (int i = 0; i < C::kChunks; ++i) {
        const int chunk = t + 128 * i, r = chunk / kCols, c = chunk - r * kCols;
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        uint4 h[2];
        h[0] = make_uint4(codes2_lo<kInt8>(w[0]), codes2_hi<kInt8>(w[0]), codes2_lo<kInt8>(w[1]), codes2_hi<kInt8>(w[1]));
        h[1] = make_uint4(codes2_lo<kInt8>(w[2]), codes2_hi<kInt8>(w[2]), codes2_lo<kInt8>(w[3]), codes2_hi<kInt8>(w[3]));
        // (neighbours whose chunks lie in different blocks of 64 dims store their halves in the other order: no two of
        // eight lanes meet a bank)
        const int swap = (c >> 2) & 1;
        const uint32_t row_at = dst + (c >> 2) * C::kBlockBytes + r * 128;
        const int pos = 2 * (c & 3);
        sts128(row_at + (((pos + swap) ^ (r & 7)) << 4), swap ? h[1] : h[0]);
        sts128(row_at + (((pos + 1 - swap) ^ (r & 7)) << 4), swap ? h[0] : h[1]);
      }
      if (v && t < C::kGroups) {
        const int id = ids[0], head = at / tiles_each / p.line.items;
        float ks = 0.0f, vs = 0.0f;
        if (id >= 0) {
          ks = __ldg(p.k_scale + static_cast<int64_t>(id) * p.kv_heads + head);
          vs = __ldg(p.v_scale + static_cast<int64_t>(id) * p.kv_heads + head);
        } else {
          raise_error(p.err, FP4_ERR_BADIDX);
        }
        const float lv = attn_lg2(fmaxf(vs, 7.888609052210118e-31f));
        float* const scales = reinterpret_cast<float*>(smem + C::kScaleOff) + stage * 24;
        scales[t] = ks;
        scales[8 + t] = lv;
        scales[16 + t] = attn_ex2(-lv);
      }
      fence_proxy_async_smem();
      mbar_arrive(v ? v_full(stage) : k_full(stage));
      ids[0] = ids[1], ids[1] = ids[2], ids[2] = ids[3], ids[3] = far;
      if (at + 1 < end) load(at + 1, ids[0]);
      prefetch(at + 3, ids[2]);
    }
  } else {
    // ---- MMA warp ----
    constexpr uint32_t id_s = idesc_f16_f32(128, C::kTile, false), id_o = idesc_f16_f32(128, kDim, true);
    int turns[2] = {0, 0}, tile_no = 0, segment = 0;
    for (int at = begin; at < end; ++segment) {
      const int item = at / tiles_each, seg_end = min(end, (item + 1) * tiles_each), tiles = seg_end - at;
      const bool pair = paired(item);
      const int units = pair ? 2 * tiles : tiles;
      wait(q_there, segment & 1);
      tc_fence_after();
      auto score = [&](int u) {
        const int b = u & 1, tile = tile_no + (pair ? u >> 1 : u), stage = tile % C::kStages;
        wait(k_full(stage), (tile / C::kStages) & 1);
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
        if (ok && elect_one()) {
          const uint64_t q_desc = sdesc_sw128(sm + (C::kSlots == 2 ? b : 0) * C::kQBytes);
          const uint64_t k_desc = sdesc_sw128(sm + C::kKOff + stage * C::kTileBytes);
#pragma unroll
          for (int k = 0; k < kDim / 16; ++k)
            mma_ss(tmem + b * 128, q_desc + (k >> 2) * (128 * 128 >> 4) + 2 * (k & 3),
                   k_desc + (k >> 2) * (C::kBlockBytes >> 4) + 2 * (k & 3), id_s, k > 0);
          mma_commit(scored(b));
          if (!pair || b == 1) mma_commit(k_empty(stage));
        }
        __syncwarp();
      };
      score(0);
      if (units > 1) score(1);
      for (int u = 0; u < units; ++u) {
        const int b = u & 1, tile = tile_no + (pair ? u >> 1 : u), stage = tile % C::kStages;
        wait(weighed(b), (turns[b] + (u >> 1)) & 1);
        wait(v_full(stage), (tile / C::kStages) & 1);
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
        if (ok && elect_one()) {
          const uint64_t v_desc = sdesc_n_major_f16(sm + C::kVOff + stage * C::kTileBytes, C::kBlockBytes);
          const uint32_t o = tmem + 256 + (C::kSlots == 2 ? b : 0) * 128;
#pragma unroll
          for (int k = 0; k < C::kTile / 16; ++k)  // 16 tokens each, 2048 bytes
            mma_ts(o, tmem + b * 128 + 8 * k, v_desc + 128 * k, id_o, (C::kSlots == 2 ? u > 1 : u > 0) || k > 0);
          mma_commit(added(b));
          if (!pair || b == 1) mma_commit(v_empty(stage));
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
}

}  // namespace fp4
