// k_kv_attention_tc.cuh -- the attention of fp4gemv_kv_attention on the
// 5th-generation tensor core, for E4M3 codes of head_dim 128 and 17 to 32 query
// rows per KV head.
//
// The mathematics of k_kv_attention.cuh, with both products on the codes as
// they lie in the cache: tcgen05.mma of kind f8f6f4 takes E4M3 from shared
// memory, so no code is converted.  What meets the codes is made 8 bits wide as
// well, as sums of such values:
//
// * a query row, scaled by a power of two to a largest magnitude in
//   [128, 256), is q1 + (q2 + q3) / 32 in E4M3 of 4 bits each.  Two parts hold
//   bf16's 8 bits and three f16's 11; values below 2^-14 of the row's largest
//   (f16: 2^-11) lose bits below 2^-22 of it.  S^T [128 tokens x 64] = K
//   [128 x 128] [q1 | q2 + q3]^T, the parts side by side on N, q3 added by an MMA
//   of its own (f16 only).
// * a weight w = 2^(s + log2 vs - m + kWScale), rounded to f16 as it is there, is
//   w1 + w2 / 16 + w3 / 256 in E5M2, of 3 bits each and f16's exponents: exactly,
//   for every f16 up to 2^15.  (What a part leaves is at most half the last place
//   of its 3 bits, 2^11 of 2^15, so 16 times it fits the next; with the parts'
//   signs that is 11 bits.)  The maximum's weight is 2^kWScale, so that a long tail
//   of small ones is not lost: f16 has 11 bits of them down to 2^-25 of the maximum
//   and loses what is below 2^-36.  (E4M3 parts of weights up to 1 end at 2^-24.)
//   out^T [128 dims x 96] = V^T [128 dims x 128 tokens] [w1 | w2 | w3]: V^T is
//   read from the V tile as it lies (M-major), the weights' tile has a token's
//   96 bytes in a row (N-major).
//
// A thread owns a token of the tile while it makes weights (TMEM lane = token),
// so a token's scales, its place among the masks and its own V row, which it
// clears where the token is of no sequence, are plain registers; and a
// dimension while it moves sums (TMEM lane = dim).
//
// The work: a CTA per SM, twelve warps.  A producer warp for K and one for V
// bring tiles of 128 tokens, whole pages by TMA, into rings of their own (K is
// free as soon as its scores are made); two groups of four warps take the tiles
// by turns, each with sums and running maxima of its own, and an MMA warp for
// each.  While a group makes weights the other's products run and its own next
// scores are made.  Shares, segments, partials and their joining are those of
// k_kv_attention.cuh; shares are cut at tiles, so that tiles hold whole pages.
//
// What bounds it.  32 sequences of 16384 tokens, 4 new ones each, 64 heads over
// 8: 174 us, 0.93 of the measured bandwidth (mma.sync with the codes converted
// in registers: 263, bound by issue: 447 instructions a strip of 16 tokens,
// where this kernel needs 342).  Steps to it: both rings as one, a V tile held
// as long as its K and 16 TMA boxes a tile from one warp 228; rings apart, boxes
// of a page 175.  Short calls pay for the set-up and the first tile's chain
// (13.4 us for one sequence of 1000 tokens; mma.sync 16), several items in a share
// for the drains between them (kAttnTcItemCost: 24 ragged sequences of up to
// 8191 tokens 68 us with 16, 58 with 32, 54 with 64; mma.sync 90).
//
// Every wait is bounded.  After a failed one (the error word holds
// FP4_ERR_TIMEOUT) the waits that follow are skipped, so that all roles come to
// their ends, named barriers included, and the outputs of the items concerned
// are NaN.
#pragma once

#include "k_kv_attention.cuh"

namespace fp4 {

struct AttnTc {
  static constexpr int kDim = 128;
  static constexpr int kTile = 128;          // tokens
  static constexpr int kRows = 32;
  static constexpr int kGroups = 2;          // of 128 threads
  static constexpr int kWeighers = kGroups * 128;
  static constexpr int kThreads = kWeighers + 64 + 32 * kGroups;  // + producers + MMA warps
  // tiles in the rings: K is free again as soon as its scores are made, V waits for the weights
  static constexpr int kKStages = 4, kVStages = 6;
  static constexpr int kTileBytes = kTile * kDim;
  static constexpr int kQBytes = 96 * kDim;           // three parts of 32 rows
  // rings | weights, a tile for each group | queries | pages' scales [V stage][K, V][8] | sequences
  static constexpr int kVOff = kKStages * kTileBytes;
  static constexpr int kWOff = kVOff + kVStages * kTileBytes;
  static constexpr int kQOff = kWOff + kGroups * kTileBytes;
  static constexpr int kScaleOff = kQOff + kQBytes;
  static constexpr int kSeqOff = kScaleOff + kVStages * 64;
  static constexpr int smem(int B) { return 1024 + kSeqOff + (B + 1) * 12; }
  static constexpr uint32_t kCols = 512;     // TMEM: S 64 for each group, then out 96 for each
  static constexpr int kSCols = 64, kOCols = 96;
  static constexpr float kWScale = 11.0f;    // log2 of the maximum's weight
  static constexpr float kWUnscale = 0x1p-11f;
  static constexpr float kSlack = 4.0f;      // ... and of how much larger one may be before m moves: 2^15 in all
};

// D[tmem] (+)= A[smem] B[smem], of the 8-bit types that the instruction descriptor names
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(
          d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// kind::f8f6f4, fp32 D: E4M3 A and B, both K-major; E4M3 A and E5M2 B, M- and N-major
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(uint32_t M, uint32_t N) {
  return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
__host__ __device__ constexpr uint32_t idesc_e4m3_e5m2_f32_mn(uint32_t M, uint32_t N) {
  return (1u << 4) | (1u << 10) | (1u << 15) | (1u << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
// Shared-memory matrix descriptor of an M- or N-major tile of up to 128 one-byte
// rows: 128-byte lines, one for each k, swizzled in atoms of 8.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr) {
  return (sdesc_sw128(saddr) & ~(static_cast<uint64_t>(0x3FFF) << 16)) | (static_cast<uint64_t>(1024 >> 4) << 16);
}
// Each thread of the warp reads 32 consecutive columns of its lane (and has
// them: the wait is part of the statement, so that nothing moves before it).
__device__ __forceinline__ void tmem_get32(uint32_t taddr, float (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
        "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
        "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(taddr)
      : "memory");
}
// Two values to two codes (too large: the largest), and back.
__device__ __forceinline__ uint16_t e4m3x2_of_f16x2(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
__device__ __forceinline__ uint16_t e5m2x2_of_f16x2(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_of_e5m2x2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
__device__ __forceinline__ uint32_t join16(uint16_t lo, uint16_t hi) {
  uint32_t r;
  asm("mov.b32 %0, {%1, %2};" : "=r"(r) : "h"(lo), "h"(hi));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_mul32(uint32_t a) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(0x50005000u));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_mul16(uint32_t a) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(0x4C004C00u));
  return r;
}
template <int kId>
__device__ __forceinline__ void named_sync(int threads) {
  asm volatile("barrier.cta.sync.aligned %0, %1;" ::"n"(kId), "r"(threads) : "memory");
}
__device__ __forceinline__ void group_sync(int group) {
  asm volatile("barrier.cta.sync.aligned %0, 128;" ::"r"(1 + group) : "memory");
}
// Barrier `id` of `threads` threads: whether v holds for any.
__device__ __forceinline__ bool named_any(int id, int threads, bool v) {
  uint32_t r;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 p, %3, 0; barrier.cta.red.or.pred.aligned q, %1, %2, p; selp.u32 %0, 1, 0, q; }"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(v))
      : "memory");
  return r != 0;
}
// v[0 .. 31] of every lane: returns the reduction of v[lane] over the warp.
template <class Op>
__device__ __forceinline__ float warp_columns(float (&v)[32], Op op) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float give = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
      v[i] = op(keep, __shfl_xor_sync(0xFFFFFFFFu, give, o));
    }
  }
  return v[0];
}

// NaN codes of tokens that some of an item's rows see and some do not (`part` of the warp's 32 tokens, their V rows from
// shared address v_rows on; the first of them is seen by queries from `since` on): a weight of 0 does not silence them, so
// they give way to zeros, and the rows that do see their token are noted in nan_dims for the segment's end.  The warp takes
// four tokens at a time, a lane for each 16 bytes (chunk k of a row lies at k ^ its number mod 8).  A function of its own,
// since the masks' path is short of instruction cache: 128 sequences of 500 tokens, 4 new ones, 64 heads on 8, 67.4 us,
// 68.2 where it stands.
__device__ __noinline__ void attn_tc_quiet(uint32_t part, uint32_t v_rows, int since, int window, int q_len, int group,
                                           int row0, int used, uint32_t (*nan_dims)[AttnTc::kDim / 32], int* nan_any) {
  const int lane = threadIdx.x & 31, k = lane & 7;
  while (part != 0u) {
    uint32_t mine = part;
    for (int i = lane >> 3; i > 0; --i) mine &= mine - 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) part &= part - 1;
    const int token = __ffs(mine) - 1;
    const uint32_t at = v_rows + token * 128 + ((k ^ (token & 7)) << 4);
    uint32_t u[4] = {0u, 0u, 0u, 0u};
    if (mine != 0u) {
      const uint4 chunk = lds128(at);
      u[0] = chunk.x, u[1] = chunk.y, u[2] = chunk.z, u[3] = chunk.w;
    }
    if ((nan_codes(u[0]) | nan_codes(u[1]) | nan_codes(u[2]) | nan_codes(u[3])) == 0u) continue;
    uint32_t dims = 0u;  // of the chunk's 16
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t nan = nan_codes(u[i]);
      u[i] &= ~((nan >> 7) * 0xFFu);
      dims |= nan_lanes(nan) << (4 * i);
    }
    sts128(at, make_uint4(u[0], u[1], u[2], u[3]));
    const int first = max(since + token, 0), last = window > 0 ? min(since + token + window, q_len) : q_len;  // its queries
    for (int r = max(first * group - row0, 0); r < min(last * group - row0, used); ++r) {
      atomicOr(&nan_dims[r][k >> 1], dims << (16 * (k & 1)));
      *nan_any = 1;
    }
  }
  __syncwarp();
}

__global__ void __launch_bounds__(AttnTc::kThreads, 1) kv_attention_tc_kernel(const __grid_constant__ KvAttnTcParams p) {
  using C = AttnTc;
  extern __shared__ __align__(128) uint8_t smem_tc[];
  __shared__ AttnPlace places[3];
  __shared__ int plan_words[6];
  __shared__ int last_flag;
  __shared__ uint32_t tmem_slot;
  __shared__ __align__(8) uint64_t bars[2 * (C::kKStages + C::kVStages) + 5 * C::kGroups];
  __shared__ __align__(16) float row_factor[C::kRows];             // of the scores
  __shared__ __align__(16) float row_m[C::kGroups][C::kRows];
  __shared__ __align__(16) float row_base[C::kGroups][C::kRows];   // kWScale - m; 0 while there is no m to go by
  __shared__ float row_tmp[C::kWeighers / 32][C::kRows];          // maxima, sums of the warps
  __shared__ __align__(16) float row_fall[C::kGroups][C::kRows];
  __shared__ float2 ml[C::kRows];
  __shared__ uint32_t nan_dims[C::kRows][C::kDim / 32];  // of the segment's rows: dims where a token that the row sees is NaN
  __shared__ int nan_any;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  uint8_t* const smem = smem_tc + (-smem_u32(smem_tc) & 1023u);  // (swizzle atoms of 1024 bytes)
  const uint32_t sm = smem_u32(smem), bar0 = smem_u32(bars);
  constexpr int kBars = 2 * (C::kKStages + C::kVStages);
  auto k_full = [&](int s) -> uint32_t { return bar0 + 8 * s; };
  auto k_empty = [&](int s) -> uint32_t { return bar0 + 8 * (C::kKStages + s); };
  auto v_full = [&](int s) -> uint32_t { return bar0 + 8 * (2 * C::kKStages + s); };
  auto v_empty = [&](int s) -> uint32_t { return bar0 + 8 * (2 * C::kKStages + C::kVStages + s); };
  auto scored = [&](int g) -> uint32_t { return bar0 + 8 * (kBars + g); };       // S is there
  auto taken = [&](int g) -> uint32_t { return bar0 + 8 * (kBars + 2 + g); };    // S has been read
  auto weighed = [&](int g) -> uint32_t { return bar0 + 8 * (kBars + 4 + g); };  // the weights are there
  auto added = [&](int g) -> uint32_t { return bar0 + 8 * (kBars + 6 + g); };    // the sums are
  auto idle = [&](int g) -> uint32_t { return bar0 + 8 * (kBars + 8 + g); };     // no MMA is in flight any more
  int* const strips_before = reinterpret_cast<int*>(smem + C::kSeqOff);
  int* const line_before = strips_before + p.B + 1;
  int* const tokens = line_before + p.B + 1;

  if (tid == 0) {
    pdl_launch_dependents();
    for (int s = 0; s < C::kKStages; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(k_empty(s), 1);
    }
    for (int s = 0; s < C::kVStages; ++s) {
      mbar_init(v_full(s), 33);
      mbar_init(v_empty(s), 1);
    }
    for (int g = 0; g < C::kGroups; ++g) {
      mbar_init(scored(g), 1);
      mbar_init(taken(g), 128);
      mbar_init(weighed(g), 128);
      mbar_init(added(g), 1);
      mbar_init(idle(g), 1);
    }
    mbar_fence_init();
    prefetch_tensormap(&p.k_map);
    prefetch_tensormap(&p.v_map);
  }
  if (tid < C::kRows * (C::kDim / 32)) (&nan_dims[0][0])[tid] = 0u;
  if (tid == 0) nan_any = 0;
  pdl_wait();
  if (warp == C::kWeighers / 32) {
    tmem_alloc(smem_u32(&tmem_slot), C::kCols);
    tc_fence_before();
  }
  attn_plan<C::kThreads>(p, strips_before, line_before, tokens, plan_words, places);  // (ends with a barrier)
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int begin = plan_words[0], end = plan_words[1];
  attn_empty<C::kDim, C::kThreads>(p, tokens);

  bool ok = true;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (ok) ok = mbar_wait(bar, parity, p.err);
    __syncwarp();
  };
  const uint32_t group_s[2] = {tmem, tmem + C::kSCols};
  const uint32_t group_o[2] = {tmem + 2 * C::kSCols, tmem + 2 * C::kSCols + C::kOCols};
  AttnPlace cur = places[0];
  int at = begin;

  if (warp >= C::kWeighers / 32 + C::kGroups) {
    // ---- producer of K or of V: lane l looks up page l % 8 of tile l / 8 of every four ----
    const bool v = warp > C::kWeighers / 32 + C::kGroups;
    struct Ref {
      int id, head, want;  // page; KV head; whether any query sees some of it
    };
    int seg_end = begin < end ? min(end, at + cur.strips - cur.strip) : begin;
    auto advance = [&](int tiles) {
      for (; tiles > 0 && at < end; --tiles) {
        const int count = min(8, seg_end - at);
        cur.strip += count;
        at += count;
        if (at == seg_end && at < end) {
          cur = attn_next(p, cur, strips_before, tokens);
          seg_end = min(end, at + cur.strips);
        }
      }
    };
    auto look_up = [&]() -> Ref {
      Ref r = {0, 0, -1};  // (-1: past the last tile)
      if (at < end) {
        const int n = tokens[cur.b], page = (((cur.first + cur.strip) << 4) >> p.block_log2) + (lane & 7);
        const int low = p.window > 0 ? n - p.q_len - p.window + 1 : 0;  // the first token that any query sees
        r.head = cur.head;
        r.want = (lane & 7) << p.block_log2 < C::kTile && page << p.block_log2 < n && (page + 1) << p.block_log2 > low;
        if (r.want) r.id = __ldg(p.table + static_cast<int64_t>(cur.b) * p.max_blocks + page);
      }
      advance(4);
      return r;
    };
    advance(lane >> 3);
    __syncwarp();
    Ref now = look_up(), ahead = look_up();
    const int stages = v ? C::kVStages : C::kKStages;
    const CUtensorMap* const map = v ? &p.v_map : &p.k_map;
    const uint32_t page_bytes = 128u << p.block_log2;
    int stage = 0, filled = 0;
    uint32_t parity = 1;
#pragma unroll 1
    for (int tile = 0;; ++tile) {
      if (tile > 0 && (tile & 3) == 0) {
        now = ahead;
        ahead = look_up();
      }
      const int from = (tile & 3) * 8 + (lane & 7);
      const int id = __shfl_sync(0xFFFFFFFFu, now.id, from), head = __shfl_sync(0xFFFFFFFFu, now.head, from);
      const int want = __shfl_sync(0xFFFFFFFFu, now.want, from);
      if (want < 0) break;  // (of all pages alike)
      wait(v ? v_empty(stage) : k_empty(stage), parity);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      const uint32_t bar = v ? v_full(stage) : k_full(stage);
      const uint32_t pages = __popc(__ballot_sync(0xFFFFFFFFu, want) & 0xFFu);
      const bool good = id >= 0 && id < p.num_blocks;
      const int page = good ? id * p.kv_heads + head : p.num_blocks * p.kv_heads;  // (past the map: zeros)
      const bool skip = v && tile == p.skip_tile;
      if (lane == 0 && !skip) mbar_arrive_expect_tx(bar, pages * page_bytes);
      __syncwarp();
      if (lane < 8 && want && !skip) {
        if (!good) raise_error(p.err, FP4_ERR_BADIDX);
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
            "[%5];" ::"r"(sm + (v ? C::kVOff : 0) + stage * C::kTileBytes + lane * page_bytes),
            "l"(map), "r"(0), "r"(0), "r"(page), "r"(bar)
            : "memory");
      }
      if (v) {
        if (lane < 16 && want) {  // the pages' scales, K's and V's
          const float* scale = (lane < 8 ? p.k_scale : p.v_scale) + (good ? page : 0);
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(sm + C::kScaleOff + stage * 64 + lane * 4),
                       "l"(scale), "r"(good ? 4u : 0u)
                       : "memory");
        }
        if (!skip) cp_async_arrive_noinc(bar);
      }
      filled = min(filled + 1, stages);
      if (++stage == stages) {
        stage = 0;
        parity ^= 1;
      }
    }
    if (!ok) {  // the copies in flight: the stages filled last
      ok = true;
      for (int k = 0; k < filled; ++k) {
        parity ^= stage == 0;
        stage = stage == 0 ? stages - 1 : stage - 1;
        wait(v ? v_full(stage) : k_full(stage), parity ^ 1);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= C::kWeighers / 32) {
    // ---- MMA warp of group g: the tiles of the CTA whose number is g mod 2 ----
    const int g = warp - C::kWeighers / 32;
    constexpr uint32_t id_s = idesc_e4m3_f32(128, 64), id_s3 = idesc_e4m3_f32(128, 32);
    constexpr uint32_t id_o = idesc_e4m3_e5m2_f32_mn(128, 96);
    const uint64_t q_desc = sdesc_sw128(sm + C::kQOff), w_desc = sdesc_mn_sw128(sm + C::kWOff + g * C::kTileBytes);
    int first_tile = 0, count = 0;  // tiles before the segment; the group's tiles
    while (at < end) {
      const int seg_end = min(end, at + cur.strips - cur.strip);
      const int tiles = (seg_end - at + 7) >> 3;
      named_sync<4>(C::kWeighers + 32 * C::kGroups);  // the queries are there
      tc_fence_after();
      auto score = [&](int tile, int number) {
        const int stage = tile % C::kKStages;
        wait(k_full(stage), (tile / C::kKStages) & 1);
        if (number > 0) wait(taken(g), (number - 1) & 1);
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
        if (ok && elect_one()) {
          const uint64_t k_desc = sdesc_sw128(sm + stage * C::kTileBytes);
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_f8(group_s[g], k_desc + 2 * k, q_desc + 2 * k, id_s, k > 0);
          if (p.f16) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_f8(group_s[g] + 32, k_desc + 2 * k, q_desc + (64 * C::kDim >> 4) + 2 * k, id_s3, 1u);
          }
          mma_commit(scored(g));
          mma_commit(k_empty(stage));
        }
        __syncwarp();
      };
      const int j0 = (g - first_tile) & 1;
      if (j0 < tiles) score(first_tile + j0, count);
      for (int j = j0; j < tiles; j += 2, ++count) {
        if (j + 2 < tiles) score(first_tile + j + 2, count + 1);
        const int tile = first_tile + j, stage = tile % C::kVStages;
        wait(v_full(stage), (tile / C::kVStages) & 1);
        wait(weighed(g), count & 1);
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
        if (ok && elect_one()) {
          const uint64_t v_desc = sdesc_mn_sw128(sm + C::kVOff + stage * C::kTileBytes);
#pragma unroll
          for (int k = 0; k < 4; ++k)  // 32 tokens each, 4096 bytes
            mma_f8(group_o[g], v_desc + 256 * k, w_desc + 256 * k, id_o, j > j0 || k > 0);
          mma_commit(added(g));
          mma_commit(v_empty(stage));
        }
        __syncwarp();
      }
      first_tile += tiles;
      at = seg_end;
      if (at < end) cur = attn_next(p, cur, strips_before, tokens);
    }
    if (elect_one()) mma_commit(idle(g));
    __syncwarp();
    mbar_wait(idle(g), 0, p.err);
  } else {
    // ---- weights and sums ----
    const int g = warp >> 2, who = tid & 127;  // token of the tile, dim of the sums
    const int rows = p.q_len * p.group;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // the warp's TMEM lanes
    const uint32_t s_cols = group_s[g] + lanes, o_cols = group_o[g] + lanes;
    const uint32_t w_row = sm + C::kWOff + g * C::kTileBytes + who * 128;  // the token's weights
    int first_tile = 0, count = 0;
    // queries: eight threads a row, 16 dims each
    const int q_row = tid >> 3, q_part = tid & 7;
    auto q_source = [&](const AttnPlace& x, int row) -> const uint4* {
      const int i = (row * p.group_magic) >> 16;
      return reinterpret_cast<const uint4*>(p.q + (static_cast<int64_t>(x.b) * p.q_len + i) * p.ldq +
                                            (x.head * p.group + row - i * p.group) * C::kDim + q_part * 16);
    };
    while (at < end) {
      const int seg_end = min(end, at + cur.strips - cur.strip);
      const int tiles = (seg_end - at + 7) >> 3;
      const int n = tokens[cur.b], row0 = cur.tile * C::kRows, tok0 = (cur.first + cur.strip) << 4;
      const int used = min(C::kRows, rows - row0);
      {
        uint32_t raw[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (q_row < used) {
          const uint4* src = q_source(cur, row0 + q_row);
          const uint4 a = __ldg(src), b = __ldg(src + 1);
          raw[0] = a.x, raw[1] = a.y, raw[2] = a.z, raw[3] = a.w, raw[4] = b.x, raw[5] = b.y, raw[6] = b.z, raw[7] = b.w;
        }
        float v[16];
        float top = 0.0f;
        bool finite = true;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (p.f16) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&raw[k]));
            v[2 * k] = f.x, v[2 * k + 1] = f.y;
          } else {
            v[2 * k] = __uint_as_float(raw[k] << 16), v[2 * k + 1] = __uint_as_float(raw[k] & 0xFFFF0000u);
          }
          top = fmaxf(top, fmaxf(fabsf(v[2 * k]), fabsf(v[2 * k + 1])));
          finite = finite && fabsf(v[2 * k]) <= 3.4e38f && fabsf(v[2 * k + 1]) <= 3.4e38f;
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        const int field = static_cast<int>(__float_as_uint(top) >> 23);
        const int e = field == 0 ? 0 : min(max(field - 127 - 7, -126), 126);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        uint32_t part[3][4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int u = 0; u < 3; ++u) part[u][k] = 0u;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          // (v down has at most 11 bits: f16 holds it, but for bits below 2^-24)
          const uint32_t h = pack_f16(v[2 * k] * down, v[2 * k + 1] * down);
          const uint16_t p1 = e4m3x2_of_f16x2(h);
          const uint32_t rest = f16x2_mul32(f16x2_sub(h, f16x2_of_e4m3x2(p1)));
          const uint16_t p2 = e4m3x2_of_f16x2(rest);
          const uint16_t p3 = e4m3x2_of_f16x2(f16x2_sub(rest, f16x2_of_e4m3x2(p2)));  // (of the second part's scale)
          part[0][k >> 1] |= static_cast<uint32_t>(finite ? p1 : 0x7F7Fu) << (16 * (k & 1));  // (else: NaN)
          part[1][k >> 1] |= static_cast<uint32_t>(p2) << (16 * (k & 1));
          part[2][k >> 1] |= static_cast<uint32_t>(p3) << (16 * (k & 1));
        }
        const uint32_t q_at = sm + C::kQOff + (q_row >> 3) * 1024 + (q_row & 7) * 128 + ((q_part ^ (q_row & 7)) << 4);
#pragma unroll
        for (int u = 0; u < 3; ++u)
          sts128(q_at + u * 32 * C::kDim, make_uint4(part[u][0], part[u][1], part[u][2], part[u][3]));
        if (q_part == 0)
          row_factor[q_row] = p.sm_scale * 1.4426950408889634f * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        if (q_part < C::kGroups) {
          row_base[q_part][q_row] = 0.0f;
          row_m[q_part][q_row] = kAttnFloor;
        }
        fence_proxy_async_smem();
      }
      named_sync<4>(C::kWeighers + 32 * C::kGroups);  // the queries and the rows' factors are there
      if (seg_end < end) {  // the next item's on their way to L2
        const AttnPlace x = attn_next(p, cur, strips_before, tokens);
        const int row = x.tile * C::kRows + q_row;
        if (row < rows) asm volatile("prefetch.global.L2 [%0];" ::"l"(q_source(x, row)));
      }
      const int tokens_all = n - p.q_len + 1;                          // every row sees those before this one
      const int tokens_low = p.window > 0 ? max(0, n - p.window) : 0;  // ... from this one on
      const int tok_end = min(n, tok0 + ((seg_end - at) << 4));
      const int tok_low = p.window > 0 ? n - p.q_len - p.window + 1 : 0;  // the first token that any query sees
      uint64_t sum[C::kRows / 2];  // of the thread's tokens: weights / vs
#pragma unroll
      for (int i = 0; i < C::kRows / 2; ++i) sum[i] = 0ull;
      bool fresh = true;  // the group has had no tile that every row sees some of: no maxima to go by
      const int j0 = (g - first_tile) & 1;
      for (int j = j0; j < tiles; j += 2, ++count) {
        const int tile = first_tile + j, stage = tile % C::kVStages;
        const int tile0 = tok0 + j * C::kTile, tok = tile0 + who;
        wait(scored(g), count & 1);
        wait(v_full(stage), (tile / C::kVStages) & 1);  // the scales and the V row
        tc_fence_after();
        uint64_t x[C::kRows / 2];  // rows 2 i and 2 i + 1
        {
          float high[32], low[32];
          tmem_get32(s_cols, high);
          tmem_get32(s_cols + 32, low);
          tc_fence_before();
          mbar_arrive(taken(g));
#pragma unroll
          for (int i = 0; i < 16; ++i)
            x[i] = fma2(pair(low[2 * i], low[2 * i + 1]), pair(0.03125f, 0.03125f), pair(high[2 * i], high[2 * i + 1]));
        }
        const uint32_t scales = sm + C::kScaleOff + stage * 64 + (who >> p.block_log2) * 4;
        const float ks = ldsf(scales), vs = ldsf(scales + 32);
        const float lv = attn_lg2(fmaxf(vs, 7.888609052210118e-31f)), inv_vs = attn_ex2(-lv);
        const bool live = tok < tok_end && tok >= tok_low;
        const bool masked = tile0 + C::kTile > min(tokens_all, tok_end) || tile0 < tokens_low;
        if (!live) {  // whatever lies there counts nothing
          const uint32_t v_row = sm + C::kVOff + stage * C::kTileBytes + who * 128;
#pragma unroll
          for (int k = 0; k < 8; ++k) sts128(v_row + ((k ^ (who & 7)) << 4), make_uint4(0, 0, 0, 0));
        }
        // the weights' exponents against the running maxima
        float top = 0.0f;
        {
          const uint64_t ks2 = pair(ks, ks), lv2 = pair(lv, lv);
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(&row_factor[2 * i]);
            const ulonglong2 m = *reinterpret_cast<const ulonglong2*>(&row_base[g][2 * i]);
            x[i] = fma2(x[i], mul2(f.x, ks2), add2(m.x, lv2));
            x[i + 1] = fma2(x[i + 1], mul2(f.y, ks2), add2(m.y, lv2));
            const float2 a = unpair(x[i]), b = unpair(x[i + 1]);
            top = fmaxf(fmaxf(top, fmaxf(a.x, a.y)), fmaxf(b.x, b.y));
          }
        }
        if (j > j0) wait(added(g), (count - 1) & 1);  // the sums so far; the weights' tile is free
        if (named_any(1 + g, 128, masked || fresh || top > C::kSlack + C::kWScale)) {
          // ---- masks; the running maxima move ----
          float v[32];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 a = unpair(x[i]);
            v[2 * i] = a.x - row_base[g][2 * i];
            v[2 * i + 1] = a.y - row_base[g][2 * i + 1];
          }
          if (masked) {
            // The rows [from, to) see the token: those of the queries from `since` on, and with a window of fewer than all.
            // (Rows that are no rows go with the last one, so that their maxima are not the floor.)
            const int since = tok - (n - p.q_len);
            const int from = max(since, 0) * p.group - row0;
            const int to = !live ? from
                           : p.window > 0 && since + p.window < p.q_len ? max(since + p.window, 0) * p.group - row0 : C::kRows;
#pragma unroll
            for (int r = 0; r < C::kRows; ++r)
              if (r < from || r >= to) v[r] = -__builtin_huge_valf();
            const uint32_t part = __ballot_sync(0xFFFFFFFFu, live && (tok >= tokens_all || tok < tokens_low));
            if (part != 0u)
              attn_tc_quiet(part, sm + C::kVOff + stage * C::kTileBytes + (who - lane) * 128, tok - lane - (n - p.q_len),
                            p.window, p.q_len, p.group, row0, used, nan_dims, &nan_any);
          }
          float w[32];
#pragma unroll
          for (int r = 0; r < 32; ++r) w[r] = v[r];
          row_tmp[warp][lane] = warp_columns(w, [](float a, float b) { return fmaxf(a, b); });
          group_sync(g);
          fresh = fresh && tile0 < tokens_low;
          if (who < C::kRows) {
            const float old = row_m[g][who];
            float now = old;
#pragma unroll
            for (int k = 0; k < 4; ++k) now = fmaxf(now, row_tmp[g * 4 + k][who]);
            row_m[g][who] = now;
            row_base[g][who] = fresh ? 0.0f : C::kWScale - now;
            row_fall[g][who] = attn_ex2(old - now);
          }
          group_sync(g);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            x[i] = pair(v[2 * i] - row_m[g][2 * i] + C::kWScale, v[2 * i + 1] - row_m[g][2 * i + 1] + C::kWScale);
            sum[i] = mul2(sum[i], *reinterpret_cast<const uint64_t*>(&row_fall[g][2 * i]));
          }
          if (j > j0) {
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < C::kOCols; c += 32) {
              float o[32];
              uint32_t u[16];
              tmem_get32(o_cols + c, o);
#pragma unroll
              for (int h = 0; h < 32; h += 16) {
#pragma unroll
                for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(o[h + k] * row_fall[g][h + k]);
                tmem_st16(o_cols + c + h, u);
              }
            }
            tmem_wait_st();
          }
        }
        // weights, their sums, their parts
        const uint64_t inv2 = pair(inv_vs * C::kWUnscale, inv_vs * C::kWUnscale);  // (sums are those of weights up to 1)
#pragma unroll
        for (int r0 = 0; r0 < C::kRows; r0 += 16) {
          uint32_t part[3][4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint16_t code[3][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int i = r0 / 2 + 2 * k + h;
              const float2 e = unpair(x[i]);
              const float a = attn_ex2(e.x), b = attn_ex2(e.y);
              sum[i] = fma2(pair(a, b), inv2, sum[i]);
              const uint32_t w = pack_f16(a, b);
              code[0][h] = e5m2x2_of_f16x2(w);
              const uint32_t rest = f16x2_mul16(f16x2_sub(w, f16x2_of_e5m2x2(code[0][h])));  // (exact)
              code[1][h] = e5m2x2_of_f16x2(rest);
              code[2][h] = e5m2x2_of_f16x2(f16x2_mul16(f16x2_sub(rest, f16x2_of_e5m2x2(code[1][h]))));
            }
#pragma unroll
            for (int u = 0; u < 3; ++u) part[u][k] = join16(code[u][0], code[u][1]);
          }
#pragma unroll
          for (int u = 0; u < 3; ++u)
            sts128(w_row + (((2 * u + (r0 >> 4)) ^ (who & 7)) << 4),
                   make_uint4(part[u][0], part[u][1], part[u][2], part[u][3]));
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(weighed(g));
      }

      // ---- the segment's end: sums of the two groups ----
      const bool any = j0 < tiles;
      if (any) wait(added(g), (count - 1) & 1);
      tc_fence_after();
      {
        float v[32];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 a = unpair(sum[i]);
          v[2 * i] = a.x, v[2 * i + 1] = a.y;
        }
        row_tmp[warp][lane] = warp_columns(v, [](float a, float b) { return a + b; });
      }
      {
        // the group's sums, dims by rows, in its weights' tile
        float o[32], low[32];
        tmem_get32(o_cols, o);
        tmem_get32(o_cols + 32, low);
#pragma unroll
        for (int r = 0; r < 32; ++r) o[r] = fmaf(low[r], 0.0625f, o[r]);
        tmem_get32(o_cols + 64, low);
        tc_fence_before();
        float* const mine = reinterpret_cast<float*>(smem + C::kWOff + g * C::kTileBytes);
#pragma unroll
        for (int r = 0; r < 32; ++r) mine[r * C::kDim + who] = any ? fmaf(low[r], 0.00390625f, o[r]) * C::kWUnscale : 0.0f;
      }
      const bool failed = named_any(3, C::kWeighers, !ok);  // (some wait ran out: NaN)
      if (nan_any != 0) {  // (written before that barrier, cleared behind the next: all threads alike)
        float* const sums = reinterpret_cast<float*>(smem + C::kWOff);
#pragma unroll 1
        for (int i = tid; i < C::kRows * C::kDim; i += C::kWeighers)
          if (nan_dims[i / C::kDim][i % C::kDim / 32] >> (i & 31) & 1u) sums[i] = __int_as_float(0x7FC00000);
        named_sync<3>(C::kWeighers);
        if (tid < C::kRows * (C::kDim / 32)) (&nan_dims[0][0])[tid] = 0u;
        if (tid == 0) nan_any = 0;
      }
      const bool starts = cur.strip == 0, whole = starts && seg_end - at == cur.strips;
      const AttnItemEnd<C::kDim, C::kWeighers> item_end = {p, cur, row0, used};
      float* const part = item_end.part_of(blockIdx.x, starts ? 1 : 0);
#pragma unroll
      for (int k = 0; k < C::kRows / (C::kWeighers / 32); ++k) {
        const int r = k * (C::kWeighers / 32) + warp, d = lane * 4;
        if (r >= used) break;
        const float m0 = row_m[0][r], m1 = row_m[1][r], top = fmaxf(m0, m1);
        const float f0 = attn_ex2(m0 - top), f1 = attn_ex2(m1 - top);
        const float l0 = (row_tmp[0][r] + row_tmp[1][r]) + (row_tmp[2][r] + row_tmp[3][r]);
        const float l1 = (row_tmp[4][r] + row_tmp[5][r]) + (row_tmp[6][r] + row_tmp[7][r]);
        const float* a = reinterpret_cast<const float*>(smem + C::kWOff) + r * C::kDim + d;
        const float4 u = *reinterpret_cast<const float4*>(a);
        const float4 w = *reinterpret_cast<const float4*>(a + C::kTileBytes / 4);
        const float4 v = make_float4(u.x * f0 + w.x * f1, u.y * f0 + w.y * f1, u.z * f0 + w.z * f1, u.w * f0 + w.w * f1);
        const float l = failed ? __int_as_float(0x7FC00000) : l0 * f0 + l1 * f1;
        if (whole) {
          item_end.store(r, d, v, top, l);
        } else {
          float* const o = part + r * (C::kDim + 4);
          __stcg(reinterpret_cast<float4*>(o + d), v);
          if (d == 0) __stcg(reinterpret_cast<float2*>(o + C::kDim), make_float2(top, l));
        }
      }
      if (!whole) item_end.share(plan_words, line_before, ml, &last_flag, [] { named_sync<3>(C::kWeighers); });
      named_sync<3>(C::kWeighers);  // (before the tables and tiles are written again)
      first_tile += tiles;
      at = seg_end;
      if (at < end) cur = attn_next(p, cur, strips_before, tokens);
    }
  }
  __syncthreads();
  if (warp == C::kWeighers / 32) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

}  // namespace fp4
