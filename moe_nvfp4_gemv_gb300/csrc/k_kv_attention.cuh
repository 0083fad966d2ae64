// k_kv_attention.cuh -- attention of a few newest tokens per sequence over
// the paged 8-bit cache (fp4gemv_kv_attention).
//
// The mathematics.  A page's scales leave the inner loops: with K = ks kc and
// V = vs vc (codes kc, vc) the score in base 2 is
//   s = (q . kc) ks sm_scale log2(e),
// and instead of p = 2^(s - max s) the kernel weighs codes directly with
//   w = 2^(s + log2 vs - m),   m + kAttnLift the running maximum of s + log2 vs,
// so that out = (sum w vc) / (sum w / vs) with w of one size whatever the
// scales: w is rounded to f16 for the product with vc, sums stay fp32.  The
// maximum's weight is 2^kAttnLift and not 1, so that f16 holds 11 bits of
// weights down to 2^-21 of it and loses only what is below 2^-32: with weights
// up to 1 the edge was 2^-25, and a long tail of tokens below it was missing
// from the output that its sum is counted in.  The codes are exact in f16.
// Queries are made exact f16 operands by a power of two for each row.
//
// Sums hold for scales of any sizes side by side: a page of zeros has scale
// 2^-100 and its tokens' w / vs count like others'.  Sums are brought to another
// maximum by factors that may be below binary32's range (attn_halves, attn_fall),
// and on pages of scales below 2^-60 w / vs is made as 2^(s - m) where the maxima
// move.  That costs 1 percent for 8 and 16 rows, 3 to 5 for 32, whose
// loop the registers are short of.
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
// m follows the maximum lazily: weights may grow to 2^(kAttnLift + kAttnSlack)
// before m moves (f16 holds them, fp32 sums do), so the usual strip costs one
// vote and no shuffles; a strip that would exceed it reduces its maxima over the warp
// and rescales.
//
// Every warp streams its own strips through its own ring of cp.async stages
// and keeps its own m, sums and accumulators: no barrier in the loop.
//
// The line.  The items (sequence, KV head, row tile) stand on one line, each
// as long as its strips and kAttnItemCost more, for what an item's end costs.
// The line is cut into equal shares, one per CTA, wherever the cuts fall; or,
// where each item can be cut into near equal pieces by itself with no more
// shares, at the items' ends too, so that no share holds two items.  At a
// segment's end (a share's part of one item) the warps' results are joined
// through the ring stage that happens to be free, while the other stages
// already fill for the next item.  An item that several shares cut is joined
// from fp32 partials in the workspace: the last of up to kAttnFan CTAs to
// arrive joins theirs; with more, the last of every kAttnFan2, and the last of
// those the joined ones (counters that are left at zero).  Nothing waits on another CTA.
//
// What bounds it (fractions of the measured copy bandwidth on the codes and
// scales read).  Long caches: HBM; 32 sequences of 16384 tokens, 8 KV heads of
// 128, us: E4M3 186 (0.86), INT8 187 (0.86), 16 rows 186 (0.87); heads of 64 98
// (0.82), of 96 143 (0.84), of 256 (16 sequences) 168 (0.96); pages of 16 tokens
// 188.  Fewer bytes: the launch, the plan, the first strips' latency and the
// joining, 8 us together: 24 ragged ones of up to 8191 tokens 45.0 us (0.70), one
// of 131071 (INT8) 51.3 (0.78), one of 777 7.5, one of 16 5.2.  32 rows: issue
// (INT8 295 us, 0.54; heads of 64 and 96, E4M3, 174 and 224, 0.46 and 0.54; E4M3 of 128 is k_kv_attention_tc.cuh's).  Measured and not
// taken: more shares than resident CTAs (24 ragged 46 to 51 .. 73 us: every CTA
// pays for its plan and first strips), two warps on one ring that part the rows
// or the dims of 32 rows between them (260 to 344 and 334 us).
//
// A window with first tokens that stay visible costs what the window alone does (kAttnSinks): 32 sequences of 32768,
// window 4096, 4 first tokens, 64 heads on 8, E4M3 53.5 us (52.7; 0.75 of the bandwidth on the tokens seen), one of 5000,
// window 1024, 8.4, 48 ragged ones of up to 3001, window 777, 130 first tokens, 4 new, INT8 heads of 96 29.4.  Many short
// windows go by warps (attn_items); more than 16 rows of E4M3 heads of 128 through k_kv_attention_tc.cuh.
#pragma once

#include <type_traits>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace fp4 {

struct KvAttnParams {
  static constexpr bool kByWarps = false;  // whether warps may take items of few strips by themselves (attn_items)
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
  float* partial;      // [CTAs][2][kAttnMaxRows][dim + 4]
  uint32_t* arrived;   // [CTAs][3], zero between calls
  int B, max_blocks, num_blocks, block_log2;
  int kv_heads, group, q_len, row_tiles;  // row tiles of 8 kN rows
  int window;
  int f16;             // element type of q and out
  int unit;            // strips (a power of two): items start and are cut at its multiples
  int item_cost;       // what an item's end costs, in strips
  int uncut;           // items of up to this many strips stay whole where there are CTAs for all
  int group_magic;     // ceil(2^16 / group): row / group = row group_magic >> 16 for the rows there are
  float inv_ctas;      // 1 / the grid's CTAs
  float sm_scale;
};

// What a kernel does beyond a window: first tokens that stay visible in it; or the rest of sequences whose beginning
// another kernel takes.
enum AttnMode { kAttnPlain, kAttnSinks, kAttnRest };
// A sequence's items hold `lead` strips of its beginning, then those of its window, with a gap between them that counts as
// no strips.
struct KvAttnSinksParams : KvAttnParams {
  static constexpr bool kByWarps = true;
  int sinks;  // the first tokens that stay visible
  int lead;   // their strips
};
// The beginning's strips count as none; a row's sums are left as they are for k_kv_prefix.cuh's join.
struct KvAttnRestParams : KvAttnParams {
  static constexpr bool kByWarps = true;
  const int32_t* prefix_len;
  float* sums;  // [kv_heads][B q_len group rows][dim]
  float2* ml;   // [kv_heads][rows]: m, the sum of weights
};
template <int kMode>
using AttnModeParams = std::conditional_t<kMode == kAttnSinks, KvAttnSinksParams,
                                          std::conditional_t<kMode == kAttnRest, KvAttnRestParams, KvAttnParams>>;
// How many tokens of a beginning of `said` tokens are taken together: a multiple of 128 before every sequence's first query.
// By a warp; *owner: the first sequence that is not empty.  kL2: past the first-level cache.
template <bool kL2>
__device__ __forceinline__ int attn_together(int said, const int32_t* lens, int B, int q_len, int64_t cap, int* owner) {
  int low = 0x7FFFFFFF, who = 0x7FFFFFFF;
  for (int b = threadIdx.x & 31; b < B; b += 32) {
    const int raw = kL2 ? __ldcg(lens + b) : __ldg(lens + b), n = raw < 0 ? 0 : raw > cap ? static_cast<int>(cap) : raw;
    if (n > 0) {
      low = min(low, n - q_len);  // (every row sees them, and some token is left)
      who = min(who, b);
    }
  }
  low = __reduce_min_sync(0xFFFFFFFFu, low);
  *owner = __reduce_min_sync(0xFFFFFFFFu, who);
  return *owner == 0x7FFFFFFF ? 0 : max(min(low, said), 0) & ~127;
}
// The same in shared memory, for the kernel's life.
__device__ __forceinline__ int& attn_taken() {
  __shared__ int taken;
  return taken;
}

// ... of the kernel on the 5th-generation tensor core
struct KvAttnTcParams : KvAttnParams {
  CUtensorMap k_map;  // [num_blocks kv_heads][block_size][128] bytes, boxes of a page, 128-byte swizzle
  CUtensorMap v_map;
  int skip_tile;      // test hook: V of this tile of every CTA is not brought (-1: of none)
};

constexpr int kAttnMaxRows = 32;  // rows of a row tile at most
constexpr int kAttnRound = 8;     // strips of a round, one for each warp: shares are whole rounds
// Partials that one CTA joins at once, and where the joined ones are joined again.  One sequence of 131072 tokens on one
// KV head, 8 rows: 16.3 us; all 152 partials at once 23.0.
constexpr int kAttnFan = 40;
constexpr int kAttnFan2 = 20;
// An item's end, in strips.  256 sequences of 500 tokens, 8 KV heads: 66 us with 8 or 16, 63 with 32.
constexpr int kAttnItemCost = 32;
constexpr int kAttnTcItemCost = 64;  // ... of the kernel on the 5th-generation tensor core (its figures there)
// The running maximum before any token: finite, so that no difference of two is a NaN, and below every finite score.
constexpr float kAttnFloor = -0x1.fffffep127f;
// Items of up to this many strips stay whole where there are CTAs for all: joining pieces costs 1.2 us, eight strips 0.15.
// Cut / whole, one sequence on 8 KV heads of 128, us: 130 tokens 7.2 / 5.5, 300 7.5 / 6.3, 500 7.5 / 7.4, 777 7.7 / 9.1;
// heads of 256: 300 9.0 / 8.3, 500 9.0 / 10.2; 32 rows, E4M3: 130 12.2 / 9.0, 500 12.5 / 10.3, 777 13.3 / 14.1.
constexpr int kAttnUncut = 40, kAttnUncut256 = 20;
// log2 of the weight of the running maximum; and of how much larger a weight may be before the running maximum moves: 256
// sequences of 500 tokens 66 us; with 0 68.8.  (2^15 in all: f16 holds 65504.)
constexpr float kAttnLift = 7.0f, kAttnSlack = 8.0f;
constexpr float kAttnUnlift = 0x1p-7f;  // 2^-kAttnLift

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
// Sums of weights / vs reach 2^100 beside a page of V that is zero, and the factors 2^d, d <= 0, to other pages' maxima
// 2^-130, which is no binary32 number; few tokens to a warp make that usual in the modes beyond the plain one.  There the
// root of 2^d is taken twice; the plain mode, whose loop a root costs more, takes 2^d as hi lo, lo 1 where 2^d is a number.
__device__ __forceinline__ float attn_halves(float l, float d) {
  const float half = attn_ex2(0.5f * d);
  return l * half * half;
}
struct AttnFall {
  float hi, lo;
};
__device__ __forceinline__ AttnFall attn_fall(float d) {
  const bool far = d < -126.0f;  // (not for a NaN)
  return {far ? 0x1p-126f : attn_ex2(d), far ? attn_ex2(d + 126.0f) : 1.0f};
}
__device__ __forceinline__ float attn_lower(float l, AttnFall f) { return l * f.lo * f.hi; }
// Pages of V of smaller scales, by log2: their tokens' weights can leave binary32's range beside others, so that in the
// sums of weights / vs they stand as 2^(s - m), made from the exponents without log2 vs.
constexpr float kAttnSmallScale = -60.0f;
// Whether l, joined from sums of up to `most` by their hi alone, lacks some that counts (at most `most` 2^-126 each).
__device__ __forceinline__ bool attn_lacks(float l, float most) { return most * 0x1p-90f > l; }
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

// Four E4M3 codes: the high bits of those that are NaN; and these as bits 0 to 3.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ uint32_t nan_lanes(uint32_t nan) {
  return (nan >> 7 & 1u) | (nan >> 14 & 2u) | (nan >> 21 & 4u) | (nan >> 28 & 8u);
}

// An item and a place in it.
struct AttnPlace {
  int b, head, tile;  // sequence, KV head, row tile
  int strip, strips;  // the place in strips; the item's number of strips
  int first;          // the sequence's first strip that any query sees (its token / 16); with leading strips, the gap
  int item;           // number of the item within the sequence
};

// ceil(x / y), x + y below 2^31
__device__ __forceinline__ int attn_div_up(int x, int y, float inv_y) {
  if (x >= 1 << 24) return (x + y - 1) / y;
  int q = static_cast<int>(static_cast<float>(x) * inv_y);  // (at most one off)
  q -= q * y > x;
  q += q * y + y <= x;
  return q + (q * y < x);
}
// The same for quotients below 2^20: no other path.
__device__ __forceinline__ int attn_div_up_small(int x, int y, float inv_y) {
  int q = static_cast<int>(static_cast<float>(x) * inv_y);  // (at most one off)
  q -= q * y > x;
  q += q * y + y <= x;
  return q + (q * y < x);
}
// Of a sequence of n tokens: the first strip that any query sees (or the unit that holds it), and the strips from there
// on; what strips take on the line.
__device__ __forceinline__ int attn_first_strip(const KvAttnParams& p, int n) {
  const int at = n - p.q_len;  // the first query's position
  return p.window > 0 && at >= p.window ? ((at - p.window + 1) >> 4) & -p.unit : 0;
}
// ... behind a beginning that is taken
__device__ __forceinline__ int attn_first_strip(const KvAttnRestParams& p, int n) { return attn_taken() >> 4; }
// ... with leading strips: the strips between them and the window
__device__ __forceinline__ int attn_first_strip(const KvAttnSinksParams& p, int n) {
  return max(attn_first_strip(static_cast<const KvAttnParams&>(p), n) - p.lead, 0);
}
template <class P>
__device__ __forceinline__ int attn_strips_of(const P& p, int n) {
  return ((n + 15) >> 4) - attn_first_strip(p, n);
}

__device__ __forceinline__ int attn_units(const KvAttnParams& p, int strips) { return (strips + p.unit - 1) & -p.unit; }

// Whether `items` of `strips` in all and `longest` at most are done sooner by a warp each than by CTAs one after another:
// a warp's strips follow on one another and its end is short; a CTA takes eight strips at a time, and an item's end and the
// chain to the next one's first sums take as long as 112 strips (kAttnItemCost is what the ends cost beside long items).
// us with 32 / 64 / 112 / 200: 512 items of 10 strips of 128 17.3 / 12.1 / 12.1 / 12.1, 1024 of 41 46.9 / 46.9 / 36.0 /
// 35.9, 400 of 33, 16 rows of 256, 53 / 53 / 37.3 / 37.3; 512 of 33 27.4 / 27.3 / 27.2 / 28.2.
inline __host__ __device__ bool attn_by_warps(float items, float strips, float longest, float warps) {
  return ceilf(items / warps) * (longest + 4.0f) * warps < strips + items * 112.0f;
}

// The plan, by the first warp (a lane per sequence, in rounds of 32; lens by
// all threads where there are many).  For every sequence: its tokens, and what
// the sequences before hold in strips and in length on the line.  The share:
// begin, end (strips), strips per share, an item's cost, and whether items are
// cut into pieces by themselves.  places[0] and [2]: the share's begin.
template <int kThreads, class P>
__device__ __forceinline__ void attn_plan(const P& p, int* strips_before, int* line_before, int* tokens,
                                          int* plan_words, AttnPlace* places) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int items = p.kv_heads * p.row_tiles;
  auto whole = [](int x) { return (x + kAttnRound - 1) / kAttnRound * kAttnRound; };  // whole rounds
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  const int64_t cap = static_cast<int64_t>(p.max_blocks) << p.block_log2;
  auto length = [&](int b) -> int {
    const int raw = __ldg(p.lens + b);
    const int n = raw < 0 ? 0 : raw > cap ? static_cast<int>(cap) : raw;
    if (n != raw && blockIdx.x == 0) raise_error(p.err, FP4_ERR_BADIDX);
    return n;
  };
  const bool few = p.B <= 32;
  if (!few) {
    for (int b = tid; b < p.B; b += kThreads) tokens[b] = length(b);
    __syncthreads();
  }
  const int ctas = static_cast<int>(gridDim.x);
  if (p.B == 1 && items <= ctas) {
    // one sequence: as many pieces of each item as there are CTAs for, without the sums over sequences below (a call of
    // 777 tokens 7.4 us, with them 8.6)
    if (warp == 0) {
      const int n = length(0), s = n > 0 ? attn_strips_of(p, n) : 0;
      const int most = attn_div_up(ctas + 1, items, __fdividef(1.0f, static_cast<float>(items))) - 1;
      const int even = attn_div_up(s, most, __fdividef(1.0f, static_cast<float>(most)));
      const int per = max(whole(s <= p.uncut ? s : even), kAttnRound);
      const int pieces = max(attn_div_up(s, per, __fdividef(1.0f, static_cast<float>(per))), 1);
      const int cta = static_cast<int>(blockIdx.x);
      const int item = attn_div_up(cta + 1, pieces, __fdividef(1.0f, static_cast<float>(pieces))) - 1;
      const int strip = (cta - item * pieces) * per;
      if (lane == 0) {
        AttnPlace place;
        place.b = 0;
        place.first = attn_first_strip(p, n);
        place.strips = s;
        place.item = item;
        place.strip = strip;
        place.head = p.row_tiles == 1 ? item : item / p.row_tiles;
        place.tile = item - place.head * p.row_tiles;
        places[0] = places[2] = place;
        tokens[0] = n;
        strips_before[0] = line_before[0] = 0;
        strips_before[1] = s * items;
        line_before[1] = per * pieces * items;
        plan_words[0] = item < items ? item * s + strip : s * items;
        plan_words[1] = item < items ? item * s + min(strip + per, s) : s * items;
        plan_words[2] = per;
        plan_words[3] = 0;
        plan_words[4] = 1;
        plan_words[5] = 0;
      }
    }
  } else if (warp == 0) {
    auto plan = [&](auto is_few) {
      constexpr bool kFew = decltype(is_few)::value;  // no more than a sequence for each lane: the loops run once
      auto again = [&](int b) -> bool { return kFew ? b == lane : b < p.B + lane; };  // (all lanes alike)
      int n0 = 0;
      if (kFew && lane < p.B) {
        n0 = length(lane);
        tokens[lane] = n0;
      }
      auto tokens_of = [&](int b) -> int { return kFew ? n0 : b < p.B ? tokens[b] : 0; };
      auto strips_at = [&](int b) -> int {
        const int n = tokens_of(b);
        return n > 0 ? attn_strips_of(p, n) : 0;
      };
      int total = 0, alive = 0, longest = 0;
      for (int b = lane; again(b); b += 32) {
        const int s = strips_at(b);
        total += __reduce_add_sync(kAll, attn_units(p, s));
        alive += __popc(__ballot_sync(kAll, s > 0));
        longest = max(longest, static_cast<int>(__reduce_max_sync(kAll, static_cast<unsigned>(s))));
      }
      total *= items;
      alive *= items;
      // pieces per item, if those of the shortest of three lengths are no more than the CTAs; one, where items are short
      int per = 0;
      if (alive <= ctas) {
        const int even = attn_div_up(total, ctas, p.inv_ctas);
        int len[3], sum[3] = {0, 0, 0};
        float inv[3];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          len[k] = max(kAttnRound, whole(even + (even * k >> 3)));
          inv[k] = __fdividef(1.0f, static_cast<float>(len[k]));
        }
        for (int b = lane; again(b); b += 32) {
          const int s = strips_at(b);
#pragma unroll
          for (int k = 0; k < 3; ++k) sum[k] += __reduce_add_sync(kAll, attn_div_up_small(s, len[k], inv[k]));
        }
#pragma unroll
        for (int k = 2; k >= 0; --k)
          if (sum[k] * items <= ctas) per = len[k];
        if (longest <= p.uncut) per = max(whole(longest), kAttnRound);
      }
      const bool pieces = per > 0;
      if (P::kByWarps && lane == 0) {
        const float slots = static_cast<float>(ctas * (kThreads / 32));
        plan_words[5] = !pieces && attn_by_warps(static_cast<float>(alive), static_cast<float>(total),
                                                 static_cast<float>(longest), slots);
      }
      const int lead = pieces ? 0 : p.item_cost;
      if (!pieces) per = max(whole(attn_div_up(total + alive * p.item_cost, ctas, p.inv_ctas)), kAttnRound);
      const float inv_per = __fdividef(1.0f, static_cast<float>(per));
      auto on_line = [&](int s) -> int {
        return pieces ? attn_div_up_small(s, per, inv_per) * per : s > 0 ? attn_units(p, s) + lead : 0;
      };
      // the sequences' places on both lines; and the share's begin and end in strips, where the cuts fall
      int strips_end = 0, line_end = 0, share[2] = {-1, -1};
      AttnPlace place = {};
      for (int b = lane; again(b); b += 32) {
        const int s = strips_at(b), len = on_line(s);
        int sum = s, line = len;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(kAll, sum, o), v = __shfl_up_sync(kAll, line, o);
          if (lane >= o) sum += u, line += v;
        }
        const float inv_len = __fdividef(1.0f, static_cast<float>(len));
        const int strips_here = strips_end + (sum - s) * items, line_here = line_end + (line - len) * items;
        if (b < p.B) {
          strips_before[b] = strips_here;
          line_before[b] = line_here;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int64_t at64 = static_cast<int64_t>(per) * (blockIdx.x + k);
          if (len > 0 && at64 >= line_here && at64 < line_here + static_cast<int64_t>(len) * items) {
            const int off = static_cast<int>(at64) - line_here;
            const int item = attn_div_up_small(off + 1, len, inv_len) - 1;
            // (a cut behind an item's last strip or in its cost: the strip that follows)
            const int strip = max(off - item * len - lead, 0);
            share[k] = strips_here + item * s + min(strip, s);
            if (k == 0) {
              place.b = b;
              place.first = attn_first_strip(p, tokens_of(b));
              place.strips = s;
              place.item = item;
              place.strip = strip;  // (below s wherever the share is not empty, or pieces end)
              place.head = p.row_tiles == 1 ? item : item / p.row_tiles;
              place.tile = item - place.head * p.row_tiles;
            }
          }
        }
        strips_end += __shfl_sync(kAll, sum, 31) * items;
        line_end += __shfl_sync(kAll, line, 31) * items;
      }
      // (the one lane that met a cut writes it; cuts past the line's end: no strip follows)
      if (share[0] >= 0) {
        plan_words[0] = share[0];
        places[0] = places[2] = place;
      }
      if (share[1] >= 0) plan_words[1] = share[1];
      const bool met0 = __any_sync(kAll, share[0] >= 0), met1 = __any_sync(kAll, share[1] >= 0);
      if (lane == 0) {
        strips_before[p.B] = strips_end;
        line_before[p.B] = line_end;
        if (!met0) plan_words[0] = strips_end;
        if (!met1) plan_words[1] = strips_end;
        plan_words[2] = per;
        plan_words[3] = lead;
        plan_words[4] = pieces;
      }
    };
    if (few) plan(std::true_type{});
    else plan(std::false_type{});
  }
  __syncthreads();
}

// Sequences nobody visits: zeros, lse -inf.
template <int kDim, int kThreads>
__device__ __forceinline__ void attn_empty(const KvAttnParams& p, const int* tokens) {
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (tokens[b] > 0) continue;
    const int heads = p.kv_heads * p.group;
    for (int i = threadIdx.x; i < p.q_len * heads * (kDim / 8); i += kThreads) {
      const int64_t row = i / (kDim / 8);
      const int64_t tok = static_cast<int64_t>(b) * p.q_len + row / heads;
      reinterpret_cast<uint4*>(p.out + tok * p.ldo + (row % heads) * kDim)[i % (kDim / 8)] = make_uint4(0, 0, 0, 0);
      if (p.lse && i % (kDim / 8) == 0) p.lse[tok * heads + row % heads] = -__builtin_huge_valf();
    }
  }
}

// The place after an item: the next item's begin (there is one).
template <class P>
__device__ __forceinline__ AttnPlace attn_next(const P& p, AttnPlace x, const int* strips_before,
                                               const int* tokens) {
  x.strip = 0;
  ++x.item;
  if (++x.tile == p.row_tiles) {
    x.tile = 0;
    if (++x.head == p.kv_heads) {
      x.head = x.item = 0;
      do ++x.b;
      while (strips_before[x.b + 1] == strips_before[x.b]);
      const int len = tokens[x.b];
      x.first = attn_first_strip(p, len);
      x.strips = attn_strips_of(p, len);
    }
  }
  return x;
}

// Four outputs of a row, and (lse not NULL) its log of the sums.
__device__ __forceinline__ void attn_put(float4 v, float top, float l, uint16_t* out, float* lse, int f16) {
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;
  v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
  uint2 w;
  if (f16) {
    w.x = pack_f16(v.x, v.y);
    w.y = pack_f16(v.z, v.w);
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    w.x = *reinterpret_cast<const uint32_t*>(&a);
    w.y = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint2*>(out) = w;
  if (lse) *lse = l > 0.0f ? 0.6931471805599453f * (top + log2f(l)) : l == l ? -__builtin_huge_valf() : l;
}

// The sum of `cnt` partials' sums of weights against the maximum `top`; the first lies `off` further.
inline __device__ __noinline__ float attn_sums(const float* at, int64_t step, int cnt, int off, float top) {
  float l = 0.0f;
#pragma unroll 1
  for (int k = 0; k < cnt; ++k) {
    const float2 o = __ldcg(reinterpret_cast<const float2*>(at + k * step + (k == 0 ? off : 0)));
    l += attn_lower(o.y, attn_fall(o.x - top));
  }
  return l;
}

// What follows an item's sums: row r's outputs, or its partials and their
// joining.  A partial row holds the sums, m and the sum of weights.
template <int kDim, int kThreads, class P = KvAttnParams>
struct AttnItemEnd {
  static constexpr int kRowFloats = kDim + 4;
  static constexpr int kMode = std::is_same_v<P, KvAttnSinksParams>  ? kAttnSinks
                               : std::is_same_v<P, KvAttnRestParams> ? kAttnRest
                                                                     : kAttnPlain;
  static constexpr bool kHalves = kMode != kAttnPlain;
  const P& p;
  const AttnPlace& cur;
  int row0, used;  // the item's first row, its rows

  __device__ __forceinline__ float* part_of(int cta, int slot) const {
    return p.partial + (static_cast<int64_t>(cta) * 2 + slot) * (kAttnMaxRows * kRowFloats);
  }
  // four outputs of local row r, dims d .. d + 3
  __device__ __forceinline__ void store(int r, int d, float4 v, float top, float l) const {
    if constexpr (kMode == kAttnRest) {
      const int rows = p.q_len * p.group;
      const int64_t at = static_cast<int64_t>(cur.head) * p.B * rows + cur.b * rows + row0 + r;
      *reinterpret_cast<float4*>(p.sums + at * kDim + d) = v;
      if (d == 0) p.ml[at] = make_float2(top, l);
      return;
    }
    const int row = row0 + r, i = (row * p.group_magic) >> 16;
    const int64_t tok_out = static_cast<int64_t>(cur.b) * p.q_len + i;
    const int head_out = cur.head * p.group + row - i * p.group;
    uint16_t* const out = p.out + tok_out * p.ldo + head_out * kDim + d;
    float* const lse = d == 0 && p.lse ? p.lse + tok_out * (p.kv_heads * p.group) + head_out : nullptr;
    attn_put(v, top, l, out, lse, p.f16);
  }
  // Behind the CTA's partial: the last CTA of those that share the item joins
  // them.  Called by kThreads threads, tid 0 on; sync() is their barrier; ml
  // holds a float2 for each row.
  template <class Sync>
  __device__ __forceinline__ void share(const int* plan_words, const int* line_before, float2* ml, int* last_flag,
                                        Sync sync) const {
    const int tid = threadIdx.x, per = plan_words[2], lead = plan_words[3];
    // the CTAs c0 .. c0 + n_parts - 1 share the item; a CTA's part is in its slot 1 if it starts the item, else 0
    const int len = plan_words[4] ? (cur.strips + per - 1) / per * per : attn_units(p, cur.strips) + lead;
    const int item0 = line_before[cur.b] + cur.item * len + lead;  // the item's first strip on the line
    const int c0 = item0 / per, n_parts = (item0 + cur.strips - 1) / per - c0 + 1;
    // true for the last of `of` CTAs to come here (all threads alike)
    auto last_of = [&](uint32_t* counter, int of) -> bool {
      sync();
      if (tid == 0) {
        __threadfence();  // (cumulative: what the barrier showed this thread goes before the count)
        *last_flag = of == 1 || atomicAdd(counter, 1u) == static_cast<uint32_t>(of - 1);
        if (*last_flag) {
          if (of > 1) *counter = 0u;
          __threadfence();
        }
      }
      sync();
      return *last_flag != 0;
    };
    // joins `cnt` partials, of every step-th CTA from `from` on, into the outputs or into the first of them
    auto join = [&](int from, int step, int cnt, bool final) {
      constexpr int kBatch = 8;  // partials in flight per thread
      const int cells = used * (kDim / 4);
      int ways = 1;  // neighbouring lanes that share a cell's partials out
      while (ways < 32 && 2 * ways * cells <= kThreads && ways * kBatch < cnt) ways *= 2;
      for (int x0 = 0; x0 < cells; x0 += kThreads / ways) {
        const int way = tid % ways, x = x0 + tid / ways;
        const bool live = x < cells;
        const int r = live ? x / (kDim / 4) : 0, d = live ? (x - r * (kDim / 4)) * 4 : 0;
        float top = kAttnFloor, l = 0.0f, most = 0.0f;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int k = way; live && k < cnt; k += kBatch * ways) {
          float2 cm[kBatch];
          float4 a[kBatch];
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const int kk = k + j * ways, c = from + kk * step;
            cm[j] = make_float2(kAttnFloor, 0.0f);
            a[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (kk < cnt) {
              const float* o = part_of(c, c == c0 ? 1 : 0) + r * kRowFloats;
              cm[j] = __ldcg(reinterpret_cast<const float2*>(o + kDim));
              a[j] = __ldcg(reinterpret_cast<const float4*>(o + d));
            }
          }
          float mn = top;
#pragma unroll
          for (int j = 0; j < kBatch; ++j) mn = fmaxf(mn, cm[j].x);
          const float fall = attn_ex2(top - mn);
          v.x *= fall, v.y *= fall, v.z *= fall, v.w *= fall;
          l = kHalves ? attn_halves(l, top - mn) : l * fall;
          top = mn;
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const float f = attn_ex2(cm[j].x - mn);
            v.x = fmaf(a[j].x, f, v.x), v.y = fmaf(a[j].y, f, v.y);
            v.z = fmaf(a[j].z, f, v.z), v.w = fmaf(a[j].w, f, v.w);
            l = kHalves ? l + attn_halves(cm[j].y, cm[j].x - mn) : fmaf(cm[j].y, f, l);
            if (!kHalves) most = fmaxf(most, cm[j].y);
          }
        }
        for (int o = 1; o < ways; o <<= 1) {
          const float to = __shfl_xor_sync(0xFFFFFFFFu, top, o), lo = __shfl_xor_sync(0xFFFFFFFFu, l, o);
          const float4 u = make_float4(__shfl_xor_sync(0xFFFFFFFFu, v.x, o), __shfl_xor_sync(0xFFFFFFFFu, v.y, o),
                                       __shfl_xor_sync(0xFFFFFFFFu, v.z, o), __shfl_xor_sync(0xFFFFFFFFu, v.w, o));
          const float mn = fmaxf(top, to);
          const float f = attn_ex2(top - mn), fo = attn_ex2(to - mn);
          v.x = v.x * f + u.x * fo, v.y = v.y * f + u.y * fo;
          v.z = v.z * f + u.z * fo, v.w = v.w * f + u.w * fo;
          l = kHalves ? attn_halves(l, top - mn) + attn_halves(lo, to - mn) : l * f + lo * fo;
          top = mn;
          if (!kHalves) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
        }
        if (!kHalves && live && way == 0 && attn_lacks(l, most))
          l = attn_sums(part_of(from, 0) + r * kRowFloats + kDim, step * 2 * kAttnMaxRows * kRowFloats, cnt,
                        from == c0 ? kAttnMaxRows * kRowFloats : 0, top);
        if (live && way == 0) {
          if (final) {
            store(r, d, v, top, l);
          } else {  // (m and the sum of weights once all threads have read the old ones)
            __stcg(reinterpret_cast<float4*>(part_of(from, from == c0 ? 1 : 0) + r * kRowFloats + d), v);
            if (d == 0) ml[r] = make_float2(top, l);
          }
        }
      }
      if (!final) {
        sync();
        if (tid < used)
          __stcg(reinterpret_cast<float2*>(part_of(from, from == c0 ? 1 : 0) + tid * kRowFloats + kDim), ml[tid]);
      }
    };
    const int fan = n_parts <= kAttnFan ? n_parts : kAttnFan2;
    const int mine = (static_cast<int>(blockIdx.x) - c0) / fan, from = c0 + mine * fan;
    const int members = min(fan, n_parts - mine * fan);
    if (last_of(p.arrived + from * 3 + (from == c0 ? 1 : 0), members)) {
      if (n_parts <= kAttnFan) {
        join(c0, 1, n_parts, true);
      } else {
        join(from, 1, members, false);
        if (last_of(p.arrived + c0 * 3 + 2, (n_parts + fan - 1) / fan)) join(c0, fan, (n_parts + fan - 1) / fan, true);
      }
    }
  }
};

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
  // Where the lane's i-th chunk of a strip goes, given that of its first: i 32
  // chunks further, 512 / kDim rows.
  static __device__ __forceinline__ int copy_to(int first, int i) {
    if (kDim == 128) return (first ^ ((i & 1) << 6)) + i * 512;
    if (kDim == 256) return (first ^ ((i & 3) << 5)) + i * 512;
    return first + i * 512;  // (64: eight rows further; 96: chunks in order)
  }
  // head_dim index of the first of the four values of K word i (block blk)
  static __device__ __forceinline__ int k_dim(int blk, int i, int t) {
    if (kBlk == 96) return 32 * (i >> 1) + 8 * t + 4 * (i & 1);
    return blk * kBlk + t * (kBlk / 4) + 4 * i;
  }
  // K words of token row g + 8 half, given the lane's place in row g
  static __device__ __forceinline__ int k_place(int g, int t) {
    return kBlk == 128 ? chunk(g, 2 * t) : kBlk == 64 ? chunk(g, t) : g * kDim + 8 * t;
  }
  static __device__ __forceinline__ void k_words(uint32_t strip, int place, int half, int blk, uint32_t (&w)[kWords]) {
    if constexpr (kBlk == 128) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 v = lds128(strip + (place ^ (16 * i)) + half * 8 * kDim + blk * 128);
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
    } else if constexpr (kBlk == 64) {
      const uint4 v = lds128(strip + place + half * 8 * kDim);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                     : "=r"(w[2 * i]), "=r"(w[2 * i + 1])
                     : "r"(strip + place + half * 8 * kDim + 32 * i));
    }
  }
  // head_dim index of the first byte of thread row g's V word i (block blk)
  static __device__ __forceinline__ int v_dim(int blk, int i, int g) {
    if (kBlk == 96) return 32 * i + 4 * g;
    return blk * kBlk + g * (kBlk / 8) + 4 * i;
  }
  // the V word (of all blocks) and the row g whose first byte is dim d (a multiple of 4)
  static __device__ __forceinline__ int2 v_place(int d) {
    if (kBlk == 96) return make_int2(d >> 5, (d & 31) >> 2);
    const int o = d % kBlk;
    return make_int2((d / kBlk) * kVWords + (o % (kBlk / 8)) / 4, o / (kBlk / 8));
  }
  // V words of token row 2 t + (c & 1) + 8 (c >> 1), given the lane's place in row 2 t
  static __device__ __forceinline__ int v_row_place(int g, int t) {
    return kBlk == 128 ? chunk(2 * t, g) : kBlk == 64 ? chunk(2 * t, g >> 1) + 8 * (g & 1) : 2 * t * kDim + 4 * g;
  }
  static __device__ __forceinline__ void v_words(uint32_t strip, int place, int c, int blk, uint32_t (&w)[kVWords]) {
    const int row = (c & 1) * kDim + (c >> 1) * 8 * kDim;
    if constexpr (kBlk == 128) {
      const uint4 v = lds128(strip + (place ^ (16 * (c & 1))) + row + blk * 128);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (kBlk == 64) {  // (rows 2 t and 2 t + 1 change places alike)
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(strip + place + row));
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i) w[i] = lds32(strip + place + row + 32 * i);
    }
  }
};

// NaN codes of tokens that some of an item's rows do not see, in a strip of V (`count` tokens, the first of them seen by
// queries from `since` on): a weight of 0 does not silence them, so they give way to zeros, and the rows that do see their
// token are noted in nan_dims for the segment's end.  By a warp, a lane for each 16 bytes.  kSinks: the strip's tokens
// before `sinks` are outside no window.
template <int kDim, bool kSinks>
__device__ __noinline__ void attn_quiet(uint32_t strip, int count, int since, int window, int q_len, int group, int row0,
                                        int used, uint32_t (*nan_dims)[kDim / 32], int* nan_any, int sinks) {
  using L = AttnLayout<kDim>;
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int i = lane; i < count * (kDim / 16); i += 32) {
    const int token = i / (kDim / 16), k = i - token * (kDim / 16), from = since + token;
    const bool stays = window == 0 || (kSinks && token < sinks);
    if (from <= 0 && (stays || from + window >= q_len)) continue;  // (all rows see it)
    const uint32_t at = strip + L::chunk(token, k);
    const uint4 chunk = lds128(at);
    uint32_t u[4] = {chunk.x, chunk.y, chunk.z, chunk.w};
    if ((nan_codes(u[0]) | nan_codes(u[1]) | nan_codes(u[2]) | nan_codes(u[3])) == 0u) continue;
    uint32_t dims = 0u;  // of the chunk's 16
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t nan = nan_codes(u[j]);
      u[j] &= ~((nan >> 7) * 0xFFu);
      dims |= nan_lanes(nan) << (4 * j);
    }
    sts128(at, make_uint4(u[0], u[1], u[2], u[3]));
    const int first = max(from, 0), last = stays ? q_len : min(from + window, q_len);  // its queries
    for (int r = max(first * group - row0, 0); r < min(last * group - row0, used); ++r) {
      atomicOr(&nan_dims[r][k >> 1], dims << (16 * (k & 1)));
      *nan_any = 1;
    }
  }
  __syncwarp();
}

// kN: tiles of 8 query rows that a warp serves; kRes: CTAs per SM (registers, shared memory).
template <int kDim, int kN, int kRes>
struct AttnCfg {
  using L = AttnLayout<kDim>;
  static constexpr int kWarps = kAttnRound;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kRows = 8 * kN;
  static constexpr bool kQInRegs = kN == 1;                         // a warp keeps its queries in registers
  // with 8 warps per SM a strip is scored while the one before is weighed: twice the independent work (32 rows leave
  // no registers for it)
  static constexpr bool kAhead = kRes == 1 && kN < 4;
  static constexpr int kStageBytes = 2 * L::kStripBytes + 16;       // K, V, the two scales
  static constexpr int kStages0 = (kRes == 2 ? 102400 : 204800) / (kWarps * kStageBytes);
  static constexpr int kStages = kStages0 > 8 ? 8 : kStages0;
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  static constexpr int kQBytes = kQInRegs ? 0 : kN * L::kSteps * 32 * 8;
  static constexpr int kSmem = kRingBytes + kQBytes + kWarps * kRows * 8 + kRows * 4;  // + the sequences
  // dynamic shared memory for B sequences
  static constexpr int smem(int B) { return kSmem + (B + 1) * 12; }
};

// What a thread takes of query `row` of a KV head's `rows`; zeros past the last one.
template <int kDim>
__device__ __forceinline__ void attn_q_load(const KvAttnParams& p, const AttnPlace& c, int row, int rows,
                                            uint4 (&raw)[kDim / 32]) {
  using L = AttnLayout<kDim>;
  const bool live = row < rows;
  const int i = live ? (row * p.group_magic) >> 16 : 0;
  const uint16_t* src = p.q + (static_cast<int64_t>(c.b) * p.q_len + i) * p.ldq +
                        (c.head * p.group + (live ? row - i * p.group : 0)) * kDim;
#pragma unroll
  for (int k = 0; k < L::kSteps / 2; ++k) {  // words 2 k and 2 k + 1: eight dims in a row
    const int d = L::k_dim(2 * k / L::kWords, 2 * k % L::kWords, threadIdx.x & 3);
    raw[k] = live ? __ldg(reinterpret_cast<const uint4*>(src + d)) : make_uint4(0, 0, 0, 0);
  }
}
// Operands in place; the row's factor of the scores.
template <int kDim>
__device__ __forceinline__ float attn_q_scale(const KvAttnParams& p, uint4 (&raw)[kDim / 32]) {
  const float factor = p.sm_scale * 1.4426950408889634f;
  if (p.f16) return factor;
  uint32_t top = 0;  // two magnitudes of bf16: ordered like their bits
#pragma unroll
  for (int k = 0; k < kDim / 32; ++k) {
    const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) top = __vmaxu2(top, w[j] & 0x7FFF7FFFu);
  }
  top = max(top & 0xFFFFu, top >> 16);
  top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
  // 2^-e brings the largest to [2^14, 2^15)
  const int field = static_cast<int>(top >> 7);
  const int e = field == 0 ? 0 : min(max(field - 127 - 14, -126), 126);
  const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
  for (int k = 0; k < kDim / 32; ++k) {
    uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = pack_f16(__uint_as_float(w[j] << 16) * down, __uint_as_float(w[j] & 0xFFFF0000u) * down);
    raw[k] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return factor * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

// Items of few strips, where there are many: a warp takes one from its queries to its outputs.  No barriers, nothing to
// join; the warps' waits fill one another's.  The warp's ring holds strips and, behind them, its queries.  By CTAs an item
// takes 3 us (16 rows of 256: 7), most of it between barriers.  By CTAs / by warps, us: first tokens and windows of up to 3
// strips, 784 items of 16 rows of 256 46 / 10.2, 848 of 16 rows of 64 19 / 8.7, 624 of one row of 256 17 / 6.6; 50 sequences
// of up to 27 tokens of their own, 1600 items of 16 rows of 256, with their beginning 69 / 54.7.
template <int kDim, bool kInt8, int kN, int kRes, int kMode>
__device__ __forceinline__ void attn_items(const AttnModeParams<kMode>& p, uint32_t ring, const int* tokens,
                                           uint32_t (*nan_dims)[kDim / 32], int* nan_any) {
  using C = AttnCfg<kDim, kN, kRes>;
  using L = AttnLayout<kDim>;
  constexpr int kRing = C::kStages - (kN == 1 ? 0 : (kN * L::kSteps * 256 + C::kStageBytes - 1) / C::kStageBytes);
  static_assert(kRing >= 2, "a strip in use and one on its way");
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);
  const uint32_t q_base = ring + kRing * C::kStageBytes;
  const int rows = p.q_len * p.group, items = p.kv_heads * p.row_tiles;
  const int k_place = L::k_place(g, t), v_place = L::v_row_place(g, t);
  const int copy_first = L::chunk(lane / (kDim / 16), lane % (kDim / 16));
  const int step = static_cast<int>(gridDim.x) * C::kWarps;
  if (!kInt8) {
    for (int i = lane; i < C::kRows * (kDim / 32); i += 32) (&nan_dims[0][0])[i] = 0u;
    if (lane == 0) *nan_any = 0;
  }
  for (int64_t id = blockIdx.x + gridDim.x * warp; id < static_cast<int64_t>(p.B) * items; id += step) {
    AttnPlace cur;
    cur.b = static_cast<int>(id) / items;
    cur.item = static_cast<int>(id) - cur.b * items;
    cur.head = cur.item / p.row_tiles;
    cur.tile = cur.item - cur.head * p.row_tiles;
    const int n = tokens[cur.b];
    if (n <= 0) continue;
    cur.first = attn_first_strip(p, n);
    cur.strip = 0;
    cur.strips = attn_strips_of(p, n);
    const int row0 = cur.tile * C::kRows, used = min(C::kRows, rows - row0);
    auto real = [&](int strip) -> int {
      if constexpr (kMode == kAttnSinks) return strip >= p.lead ? strip + cur.first : strip;
      else return strip + cur.first;
    };
    int batch = -1, filled = 0, fill_stage = 0;
    auto issue = [&]() {
      if ((filled & 31) == 0) {  // the next 32 strips' places: -1 past the last one, -2 on a bad page
        batch = -1;
        if (filled + lane < cur.strips) {
          const int strip = real(filled + lane), per_page = p.block_log2 - 4;
          const int page = __ldg(p.table + static_cast<int64_t>(cur.b) * p.max_blocks + (strip >> per_page));
          batch = page >= 0 && page < p.num_blocks
                      ? ((page * p.kv_heads + cur.head) << per_page) + (strip & ((1 << per_page) - 1))
                      : -2;
        }
      }
      int strip = __shfl_sync(0xFFFFFFFFu, batch, filled & 31);
      if (strip != -1) {
        const uint32_t dst = ring + fill_stage * C::kStageBytes;
        const uint32_t bytes = strip >= 0 ? 16u : 0u;
        if (strip < 0) {
          if (lane == 0) raise_error(p.err, FP4_ERR_BADIDX);
          strip = 0;
        }
        const int64_t at = static_cast<int64_t>(strip) * L::kStripBytes + lane * 16;
#pragma unroll
        for (int i = 0; i < kDim / 32; ++i) {
          cp_async16(dst + L::copy_to(copy_first, i), p.k_codes + at + i * 512, bytes);
          cp_async16(dst + L::kStripBytes + L::copy_to(copy_first, i), p.v_codes + at + i * 512, bytes);
        }
        if (lane < 2) {
          const float* scale = (lane ? p.v_scale : p.k_scale) + (strip >> (p.block_log2 - 4));
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + 2 * L::kStripBytes + 4 * lane),
                       "l"(scale), "r"(bytes >> 2)
                       : "memory");
        }
      }
      ++filled;
      if (++fill_stage == kRing) fill_stage = 0;
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    __syncwarp();  // (every lane is past the item before)
#pragma unroll
    for (int k = 0; k < kRing - 1; ++k) issue();
    uint4 qr[L::kSteps / 2];
    float rs[kN][2], m[kN][2], sum[kN][2], acc[kN][L::kTiles][4];
#pragma unroll
    for (int nt = 0; nt < kN; ++nt) {
      attn_q_load<kDim>(p, cur, row0 + nt * 8 + g, rows, qr);
      const float f = attn_q_scale<kDim>(p, qr);
      if (kN > 1) {  // (a lane reads what it wrote)
#pragma unroll
        for (int i = 0; i < L::kSteps / 2; ++i) sts128(q_base + ((nt * (L::kSteps / 2) + i) * 32 + lane) * 16, qr[i]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        rs[nt][h] = __shfl_sync(0xFFFFFFFFu, f, 8 * t + 4 * h);
        m[nt][h] = kAttnFloor;
        sum[nt][h] = 0.0f;
#pragma unroll
        for (int j = 0; j < L::kTiles; ++j) acc[nt][j][h] = acc[nt][j][2 + h] = 0.0f;
      }
    }
    const int tokens_all = n - p.q_len + 1;                          // every row sees those before this one
    const int tokens_low = p.window > 0 ? max(0, n - p.window) : 0;  // ... from this one on
    const bool parts = !kInt8 && (p.q_len > 1 || p.window > 0);
    bool fresh = true;
    int stage = 0;
#pragma unroll 1
    for (int k = 0; k < cur.strips; ++k) {
      const int here = real(k) << 4, left = n - here;
      const uint32_t kb = ring + stage * C::kStageBytes, vb = kb + L::kStripBytes;
      if (++stage == kRing) stage = 0;
      asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
      __syncwarp();  // the strip is there, and every lane is past the stage read last
      issue();
      if (parts && (here < tokens_low || here + 16 > tokens_all)) {
        int sinks = 0;
        if constexpr (kMode == kAttnSinks) sinks = p.sinks - here;
        attn_quiet<kDim, kMode == kAttnSinks>(vb, min(16, left), here - (n - p.q_len), p.window, p.q_len, p.group, row0, used,
                                              nan_dims, nan_any, sinks);
      }
      float sc[kN][4];  // tokens g (0, 1) and g + 8 (2, 3) by rows 2t and 2t + 1
#pragma unroll
      for (int nt = 0; nt < kN; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.0f;
#pragma unroll
      for (int blk = 0; blk < L::kBlocks; ++blk) {
        uint32_t w[2][L::kWords];
        L::k_words(kb, k_place, 0, blk, w[0]);
        L::k_words(kb, k_place, 1, blk, w[1]);
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
            const int pair = (blk * L::kWords + s) / 2;
            uint4 b;
            if constexpr (kN == 1) b = qr[pair];
            else b = lds128(q_base + ((nt * (L::kSteps / 2) + pair) * 32 + lane) * 16);
            mma_f16(sc[nt], a[0], b.x, b.y);
            mma_f16(sc[nt], a[1], b.z, b.w);
          }
        }
      }
      float ks, vs;
      asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(ks), "=f"(vs) : "r"(kb + 2 * L::kStripBytes));
      const float lv = attn_lg2(fmaxf(vs, 7.888609052210118e-31f));
      float inv_vs = attn_ex2(-lv) * kAttnUnlift;
      const bool small = lv < kAttnSmallScale;
      bool masked = here + 16 > tokens_all || here < tokens_low;
      bool some = here >= tokens_low;  // every row sees some of the strip
      if constexpr (kMode == kAttnSinks) {
        masked = here + 16 > tokens_all || (here < tokens_low && here + 16 > p.sinks);
        some = some || here < min(p.sinks, tokens_all);
      }
      // exponents; the running maxima move where they must (as in the kernel below)
      float high = -1.0f;
#pragma unroll
      for (int nt = 0; nt < kN; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float f = rs[nt][h] * ks, base = fresh ? lv : lv - m[nt][h];
          sc[nt][h] = fmaf(sc[nt][h], f, base);
          sc[nt][2 + h] = fmaf(sc[nt][2 + h], f, base);
          high = fmaxf(high, fmaxf(sc[nt][h], sc[nt][2 + h]));
        }
      if (masked || small || fresh || __any_sync(0xFFFFFFFFu, high > kAttnLift + kAttnSlack)) {
#pragma unroll
        for (int nt = 0; nt < kN; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float base = fresh ? 0.0f : m[nt][h];
            float r0 = sc[nt][h] + base, r1 = sc[nt][2 + h] + base;
            if (masked) {
              const int row = min(row0 + nt * 8 + 2 * t + h, rows - 1);
              const int see_to = n - p.q_len + ((row * p.group_magic) >> 16) + 1;
              const int see_from = p.window > 0 ? see_to - p.window : 0;
              bool out0 = here + g < see_from, out1 = here + 8 + g < see_from;
              if constexpr (kMode == kAttnSinks) {
                out0 = out0 && here + g >= p.sinks;
                out1 = out1 && here + 8 + g >= p.sinks;
              }
              if (here + g >= see_to || out0) r0 = -__builtin_huge_valf();
              if (here + 8 + g >= see_to || out1) r1 = -__builtin_huge_valf();
            }
            float top = fmaxf(r0, r1);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            const float mn = fmaxf(m[nt][h], top - kAttnLift);
            const float fall = attn_ex2(m[nt][h] - mn);
            sum[nt][h] = attn_halves(sum[nt][h], m[nt][h] - mn);
            m[nt][h] = mn;
#pragma unroll
            for (int j = 0; j < L::kTiles; ++j) {
              acc[nt][j][h] *= fall;
              acc[nt][j][2 + h] *= fall;
            }
            sc[nt][h] = r0 - mn;
            sc[nt][2 + h] = r1 - mn;
          }
        fresh = fresh && !some;
        if (small) {
#pragma unroll
          for (int nt = 0; nt < kN; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              sum[nt][h] = fmaf(attn_ex2(sc[nt][h] - lv) + attn_ex2(sc[nt][2 + h] - lv), kAttnUnlift, sum[nt][h]);
          inv_vs = 0.0f;
        }
      }
      uint32_t pb[kN][2];
#pragma unroll
      for (int nt = 0; nt < kN; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[nt][e] = attn_ex2(sc[nt][e]);
        sum[nt][0] = fmaf(sc[nt][0] + sc[nt][2], inv_vs, sum[nt][0]);
        sum[nt][1] = fmaf(sc[nt][1] + sc[nt][3], inv_vs, sum[nt][1]);
        pb[nt][0] = transpose8x8(pack_f16(sc[nt][0], sc[nt][1]));
        pb[nt][1] = transpose8x8(pack_f16(sc[nt][2], sc[nt][3]));
      }
#pragma unroll
      for (int blk = 0; blk < L::kBlocks; ++blk) {
        uint32_t w[4][L::kVWords];
#pragma unroll
        for (int c = 0; c < 4; ++c) L::v_words(vb, v_place, c, blk, w[c]);
        if (left < 16) {  // past the end: whatever lies there counts nothing
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (2 * t + (c & 1) + (c >> 1) * 8 >= left) {
#pragma unroll
              for (int i = 0; i < L::kVWords; ++i) w[c][i] = 0u;
            }
        }
#pragma unroll
        for (int i = 0; i < L::kVWords; ++i) {
          const uint32_t lo[2] = {__byte_perm(w[0][i], w[1][i], 0x5140), __byte_perm(w[0][i], w[1][i], 0x7362)};
          const uint32_t hi[2] = {__byte_perm(w[2][i], w[3][i], 0x5140), __byte_perm(w[2][i], w[3][i], 0x7362)};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t a[4] = {codes2_lo<kInt8>(lo[j]), codes2_hi<kInt8>(lo[j]), codes2_lo<kInt8>(hi[j]),
                                   codes2_hi<kInt8>(hi[j])};
#pragma unroll
            for (int nt = 0; nt < kN; ++nt) mma_f16(acc[nt][(blk * L::kVWords + i) * 2 + j], a, pb[nt][0], pb[nt][1]);
          }
        }
      }
    }
    // ---- outputs, from the registers ----
    const AttnItemEnd<kDim, C::kThreads, AttnModeParams<kMode>> item_end = {p, cur, row0, used};
    const bool nans = !kInt8 && *nan_any != 0;  // (every lane's marks are in: attn_quiet ends with a barrier)
#pragma unroll
    for (int nt = 0; nt < kN; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) sum[nt][h] += __shfl_xor_sync(0xFFFFFFFFu, sum[nt][h], o);
        const int r = nt * 8 + 2 * t + h;
        if (r >= used) continue;
#pragma unroll
        for (int k = 0; k < L::kTiles / 2; ++k) {
          const int d = L::v_dim(k / L::kVWords, k % L::kVWords, g);
          float v[4] = {acc[nt][2 * k][h] * kAttnUnlift, acc[nt][2 * k][2 + h] * kAttnUnlift,
                        acc[nt][2 * k + 1][h] * kAttnUnlift, acc[nt][2 * k + 1][2 + h] * kAttnUnlift};
          if (nans) {
            const uint32_t which = nan_dims[r][d >> 5] >> (d & 31);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (which >> i & 1u) v[i] = __int_as_float(0x7FC00000);
          }
          item_end.store(r, d, make_float4(v[0], v[1], v[2], v[3]), m[nt][h] + kAttnLift, sum[nt][h]);
        }
      }
    if (nans) {
      __syncwarp();
      for (int i = lane; i < C::kRows * (kDim / 32); i += 32) (&nan_dims[0][0])[i] = 0u;
      if (lane == 0) *nan_any = 0;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int kDim, bool kInt8, int kN, int kRes, int kMode = kAttnPlain>
__global__ void __launch_bounds__(AttnCfg<kDim, kN, kRes>::kThreads, kRes)
    kv_attention_kernel(const AttnModeParams<kMode> p) {
  using C = AttnCfg<kDim, kN, kRes>;
  using L = AttnLayout<kDim>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ AttnPlace places[3];  // the item being read and the next one by turns; the share's begin
  __shared__ int plan_words[6];
  __shared__ int free_stage[C::kWarps];  // byte offset of the warp's idle ring stage
  __shared__ uint32_t nan_dims[C::kRows][kDim / 32];  // of the segment's rows: dims where a token that the row sees is NaN
  __shared__ int nan_any;
  __shared__ int last_flag;
  const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);  // (uniform, and known to be)
  // ring | queries (where not in registers) | (m, sum) [warp][row] | row scales | sequences
  const uint32_t sm = smem_u32(smem);
  const uint32_t q_base = sm + C::kRingBytes;
  float2* const ml = reinterpret_cast<float2*>(smem + C::kRingBytes + C::kQBytes);
  float* const row_scale = reinterpret_cast<float*>(ml + C::kWarps * C::kRows);
  // of the sequences before: strips, length on the line; then each one's tokens
  int* const strips_before = reinterpret_cast<int*>(row_scale + C::kRows);
  int* const line_before = strips_before + p.B + 1;
  int* const tokens = line_before + p.B + 1;
  if (kMode != kAttnRest && tid == 0) pdl_launch_dependents();
  if (!kInt8) {
    for (int i = tid; i < C::kRows * (kDim / 32); i += C::kThreads) (&nan_dims[0][0])[i] = 0u;
    if (tid == 0) nan_any = 0;
  }
  pdl_wait();

  const int rows = p.q_len * p.group;  // query rows of a KV head
  // Queries and block table on their way to L2 while the first warp plans, each CTA a part.
  if (warp > 0) {
    const int per_row = (p.kv_heads * p.group * kDim * 2 + 127) >> 7, q_lines = p.B * p.q_len * per_row;
    const int t_lines = static_cast<int>((static_cast<int64_t>(p.B) * p.max_blocks * 4 + 127) >> 7);
    const int lines = q_lines + min(t_lines, 1 << 20), step = gridDim.x * (C::kThreads - 32);
    for (int i = blockIdx.x * (C::kThreads - 32) + tid - 32, k = 0; i < lines && k < 2; i += step, ++k) {
      const int row = i < q_lines ? i / per_row : 0;
      const char* at = i < q_lines ? reinterpret_cast<const char*>(p.q + row * p.ldq) + (i - row * per_row) * 128
                                   : reinterpret_cast<const char*>(p.table) + static_cast<int64_t>(i - q_lines) * 128;
      asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
    }
  }
  if constexpr (kMode == kAttnRest) {
    // (the kernel that takes the beginning may start now: what this one waited for is there)
    if (tid == 0) pdl_launch_dependents();
    if (warp == 0) {  // (the plan is the first warp's, and ends with a barrier)
      int owner;
      const int taken = attn_together<false>(__ldg(p.prefix_len), p.lens, p.B, p.q_len,
                                      static_cast<int64_t>(p.max_blocks) << p.block_log2, &owner);
      if (lane == 0) attn_taken() = taken;
      __syncwarp();
    }
  }
  auto first_strip = [&](int n) -> int { return attn_first_strip(p, n); };
  auto strips_of = [&](int n) -> int { return attn_strips_of(p, n); };
  attn_plan<C::kThreads>(p, strips_before, line_before, tokens, plan_words, places);
  const int begin = plan_words[0], end = plan_words[1];

  if (kMode != kAttnRest) attn_empty<kDim, C::kThreads>(p, tokens);  // (the join sees to them)
  // (The rest of sequences, up to 8 rows, or 16 with two CTAs to an SM: the code beside it costs the other path more than
  // it spares where items are short.  Heads of 256, 7 sequences on 65536, 49.8 us, with it 56.3; 16 rows of 64, 24 on
  // 8191, 34.4, 35.3; 8 rows of 128, 64 on 16384, up to 20 own tokens, 62.3, 58.5.)
  if constexpr (kMode == kAttnSinks || (kMode == kAttnRest && kN > 1 && kRes == 1)) {
    if (plan_words[5] != 0) {
      __shared__ uint32_t nan_words[kInt8 ? 1 : C::kWarps][C::kRows][kDim / 32];
      __shared__ int nan_flags[C::kWarps];
      attn_items<kDim, kInt8, kN, kRes, kMode>(p, sm + warp * C::kStages * C::kStageBytes, tokens,
                                               nan_words[kInt8 ? 0 : warp], &nan_flags[warp]);
      return;
    }
  }
  if (begin >= end) return;

  // ---- queries: f16 operands; bf16 ones scaled by a power of two for each row ----
  auto q_load = [&](const AttnPlace& c, int tile8, uint4 (&raw)[L::kSteps / 2]) {  // row g of the item's tile of 8
    attn_q_load<kDim>(p, c, c.tile * C::kRows + tile8 * 8 + g, rows, raw);
  };
  auto q_scale = [&](uint4 (&raw)[L::kSteps / 2]) -> float { return attn_q_scale<kDim>(p, raw); };
  uint4 qr[L::kSteps / 2];
  if (C::kQInRegs) q_load(places[0], 0, qr);

  // ---- the warp's ring: strips warp, warp + kWarps, ... of the share ----
  const uint32_t ring = sm + warp * C::kStages * C::kStageBytes;
  // Lane l looks up every 32nd strip of the warp, from its l-th on: one batch to copy from, one ahead.  What it
  // keeps is the strip's number in the cache, -1 past the share, -2 for a bad page.
  int looked = begin + warp + lane * C::kWarps;  // the strip that the lane looks up next
  auto look_up = [&]() -> int {
    int found = -1;
    if (looked < end) {
      int b = places[2].b, head = places[2].head, strip = places[2].strip + (looked - begin);
      if (strip >= places[2].strips) {  // (not the share's first item)
        int lo = b, hi = p.B - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (strips_before[mid] <= looked) lo = mid;
          else hi = mid - 1;
        }
        b = lo;
        const int s = strips_of(tokens[b]), off = looked - strips_before[b], item = off / s;
        strip = off - item * s;
        head = item / p.row_tiles;
      }
      if constexpr (kMode == kAttnSinks) strip += strip >= p.lead ? first_strip(tokens[b]) : 0;
      else strip += first_strip(tokens[b]);
      const int per_page = p.block_log2 - 4;
      const int id = __ldg(p.table + static_cast<int64_t>(b) * p.max_blocks + (strip >> per_page));
      found = id >= 0 && id < p.num_blocks
                  ? ((id * p.kv_heads + head) << per_page) + (strip & ((1 << per_page) - 1))
                  : -2;
    }
    looked += 32 * C::kWarps;
    return found;
  };
  int batch = look_up(), batch_next = -1, copied = 0;
  const int copy_first = L::chunk(lane / (kDim / 16), lane % (kDim / 16));
  auto issue = [&](int stage) {
    const int source = copied & 31;
    if (source == 0 && copied > 0) batch = batch_next;
    if (source == 16) batch_next = look_up();  // (halfway: there in time for the next batch)
    ++copied;
    int strip = __shfl_sync(0xFFFFFFFFu, batch, source);
    if (strip != -1) {
      const uint32_t dst = ring + stage * C::kStageBytes;
      const uint32_t bytes = strip >= 0 ? 16u : 0u;
      if (strip < 0) {
        if (lane == 0) raise_error(p.err, FP4_ERR_BADIDX);
        strip = 0;
      }
      const int64_t at = static_cast<int64_t>(strip) * L::kStripBytes + lane * 16;
      const uint8_t* ksrc = p.k_codes + at;
      const uint8_t* vsrc = p.v_codes + at;
#pragma unroll
      for (int i = 0; i < kDim / 32; ++i) {
        cp_async16(dst + L::copy_to(copy_first, i), ksrc + i * 512, bytes);
        cp_async16(dst + L::kStripBytes + L::copy_to(copy_first, i), vsrc + i * 512, bytes);
      }
      if (lane < 2) {
        const float* s = (lane ? p.v_scale : p.k_scale) + (strip >> (p.block_log2 - 4));
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + 2 * L::kStripBytes + 4 * lane), "l"(s),
                     "r"(bytes >> 2)
                     : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < C::kStages - 1; ++s) issue(s);
  const int k_place = L::k_place(g, t), v_place = L::v_row_place(g, t);

  // ---- segments: the parts of items in this CTA's share ----
  int at = begin;
  int stage = 0;
  int which = 0;                // of places
  float acc[kN][L::kTiles][4];  // dims by rows: thread's rows 2t, 2t + 1 of every tile of 8
  float m[kN][2], sum[kN][2];
  while (at < end) {
    int seg_end, n, row0, tok0;  // tok0: the token at strip `at`; with sinks: as if there were no gap,
    int gap = 0;                 // ... which is that many tokens long
    {
      const AttnPlace c = places[which];
      seg_end = min(end, at + c.strips - c.strip);
      n = tokens[c.b];
      row0 = c.tile * C::kRows;
      if constexpr (kMode == kAttnSinks) {
        tok0 = c.strip << 4;
        gap = c.first << 4;
      } else {
        tok0 = (c.first + c.strip) << 4;
      }
      if (tid == 0 && seg_end < end) {  // the next item (read behind the barriers of the joining)
        places[which ^ 1] = attn_next(p, c, strips_before, tokens);
      }
    }
    float rs[2];  // (queries in shared memory: so are the rows' factors)
    if constexpr (C::kQInRegs) {
      const float f = q_scale(qr);
      rs[0] = __shfl_sync(0xFFFFFFFFu, f, 8 * t);
      rs[1] = __shfl_sync(0xFFFFFFFFu, f, 8 * t + 4);
    } else {
      if (warp < kN) {
        q_load(places[which], warp, qr);
        const float f = q_scale(qr);
        if (t == 0) row_scale[warp * 8 + g] = f;
#pragma unroll
        for (int i = 0; i < L::kSteps / 2; ++i)
          sts128(q_base + ((warp * (L::kSteps / 2) + i) * 32 + lane) * 16, qr[i]);
      }
      __syncthreads();
    }
#pragma unroll
    for (int nt = 0; nt < kN; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        m[nt][h] = kAttnFloor;
        sum[nt][h] = 0.0f;
#pragma unroll
        for (int j = 0; j < L::kTiles; ++j) acc[nt][j][h] = acc[nt][j][2 + h] = 0.0f;
      }
    const int tokens_all = n - p.q_len + 1;                          // every row sees those before this one
    const int tokens_low = p.window > 0 ? max(0, n - p.window) : 0;  // ... from this one on

    // the token at place `tok` of the strips that there are
    auto real = [&](int tok) -> int {
      if constexpr (kMode == kAttnSinks) return tok >= p.lead << 4 ? tok + gap : tok;
      else return tok;
    };
    auto after = [](int stage) { return stage + 1 == C::kStages ? 0 : stage + 1; };
    auto before = [](int stage) { return stage == 0 ? C::kStages - 1 : stage - 1; };
    // S^T += K Q^T of two k-steps of a strip; w: its K words of a block, of rows g and g + 8
    auto score = [&](const uint32_t (&w)[2][L::kWords], int blk, int s, float (&sc)[kN][4]) {
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
        const int pair = (blk * L::kWords + s) / 2;
        uint4 b;
        if constexpr (C::kQInRegs) b = qr[pair];
        else b = lds128(q_base + ((nt * (L::kSteps / 2) + pair) * 32 + lane) * 16);
        mma_f16(sc[nt], a[0], b.x, b.y);
        mma_f16(sc[nt], a[1], b.z, b.w);
      }
    };
    auto k_load = [&](uint32_t kb, int blk, uint32_t (&w)[2][L::kWords]) {
      L::k_words(kb, k_place, 0, blk, w[0]);
      L::k_words(kb, k_place, 1, blk, w[1]);
    };
    // out^T += V^T w^T of one V word's dims
    auto weigh = [&](const uint32_t (&w)[4][L::kVWords], int blk, int k, const uint32_t (&pb)[kN][2]) {
      const uint32_t lo[2] = {__byte_perm(w[0][k], w[1][k], 0x5140), __byte_perm(w[0][k], w[1][k], 0x7362)};
      const uint32_t hi[2] = {__byte_perm(w[2][k], w[3][k], 0x5140), __byte_perm(w[2][k], w[3][k], 0x7362)};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t a[4] = {codes2_lo<kInt8>(lo[j]), codes2_hi<kInt8>(lo[j]), codes2_lo<kInt8>(hi[j]),
                               codes2_hi<kInt8>(hi[j])};
#pragma unroll
        for (int nt = 0; nt < kN; ++nt) mma_f16(acc[nt][(blk * L::kVWords + k) * 2 + j], a, pb[nt][0], pb[nt][1]);
      }
    };
    auto v_load = [&](uint32_t vb, int blk, int left, uint32_t (&w)[4][L::kVWords]) {
#pragma unroll
      for (int c = 0; c < 4; ++c) L::v_words(vb, v_place, c, blk, w[c]);
      if (left < 16) {  // past the end: whatever lies there counts nothing
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (2 * t + (c & 1) + (c >> 1) * 8 >= left) {
#pragma unroll
            for (int k = 0; k < L::kVWords; ++k) w[c][k] = 0u;
          }
      }
    };
    // this warp's strips of the segment: begin + warp + k kWarps
    int tok = tok0 + (((begin + warp - at) & (C::kWarps - 1)) << 4);
    const int tok_end = tok0 + ((seg_end - at) << 4);
    bool fresh = true;
    float sc[kN][4];  // tokens g (0, 1) and g + 8 (2, 3) by rows 2t and 2t + 1
    if (C::kAhead && tok < tok_end) {
      asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 2) : "memory");
      __syncwarp();
#pragma unroll
      for (int nt = 0; nt < kN; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.0f;
#pragma unroll
      for (int blk = 0; blk < L::kBlocks; ++blk) {
        uint32_t w[2][L::kWords];
        k_load(ring + stage * C::kStageBytes, blk, w);
#pragma unroll
        for (int s = 0; s < L::kWords; s += 2) score(w, blk, s, sc);
      }
    }
    // Strips that some row sees in part are gone through one by one, quieted first: outside the loop over the others, where
    // even a call costs registers.  32 rows, heads of 64, 32 sequences of 16384: 169 us, with the call inside 182.
    const bool parts = !kInt8 && (p.q_len > 1 || p.window > 0);
    for (int stop = tok_end; tok < tok_end;) {
      if (parts) {
        stop = min(tok_end, tokens_all - gap - 15);  // (a gap ends before the first query's position)
        if (real(tok) < tokens_low || tok >= stop) {
          if (!C::kAhead) {
            asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 2) : "memory");
            __syncwarp();
          }
          int sinks = 0;
          if constexpr (kMode == kAttnSinks) sinks = p.sinks - real(tok);
          attn_quiet<kDim, kMode == kAttnSinks>(ring + stage * C::kStageBytes + L::kStripBytes, min(16, n - real(tok)),
                                  real(tok) - (n - p.q_len), p.window, p.q_len, p.group, row0,
                                  min(C::kRows, rows - row0), nan_dims, &nan_any, sinks);
          stop = tok + 1;
        }
      }
      for (; tok < stop; tok += C::kWarps * 16) {
        const int here = real(tok);
        const uint32_t kb = ring + stage * C::kStageBytes, vb = kb + L::kStripBytes;
        if (!C::kAhead) {
          asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 2) : "memory");
          __syncwarp();  // the strip is there, and every lane is past the stage read last
          issue(before(stage));
#pragma unroll
          for (int nt = 0; nt < kN; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.0f;
#pragma unroll
          for (int blk = 0; blk < L::kBlocks; ++blk) {
            uint32_t w[2][L::kWords];
            k_load(kb, blk, w);
#pragma unroll
            for (int s = 0; s < L::kWords; s += 2) score(w, blk, s, sc);
          }
        }
        float ks, vs;
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(ks), "=f"(vs) : "r"(kb + 2 * L::kStripBytes));
        const float lv = attn_lg2(fmaxf(vs, 7.888609052210118e-31f));
        float inv_vs = attn_ex2(-lv) * kAttnUnlift;  // (sums stay those of weights up to 1)
        const bool small = lv < kAttnSmallScale;
        bool masked = here + 16 > tokens_all || here < tokens_low;
        bool some = here >= tokens_low;  // every row sees some of the strip
        if constexpr (kMode == kAttnSinks) {
          masked = here + 16 > tokens_all || (here < tokens_low && here + 16 > p.sinks);
          some = some || here < min(p.sinks, tokens_all);
        }
        // Exponents against the running maxima, in the scores' place; against 0 while the warp has seen no strip that
        // every row sees some of (`fresh`: a row's first maximum is only known then).  Where they are masked, too high
        // or fresh, or the page's scale is small, the maxima are taken and the exponents made again.
        float high = -1.0f;
#pragma unroll
        for (int nt = 0; nt < kN; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float f = (C::kQInRegs ? rs[h] : row_scale[nt * 8 + 2 * t + h]) * ks;
            const float base = fresh ? lv : lv - m[nt][h];
            sc[nt][h] = fmaf(sc[nt][h], f, base);
            sc[nt][2 + h] = fmaf(sc[nt][2 + h], f, base);
            high = fmaxf(high, fmaxf(sc[nt][h], sc[nt][2 + h]));
          }
        if (masked || small || fresh || __any_sync(0xFFFFFFFFu, high > kAttnLift + kAttnSlack)) {
#pragma unroll
          for (int nt = 0; nt < kN; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float base = fresh ? 0.0f : m[nt][h];
              float r0 = sc[nt][h] + base, r1 = sc[nt][2 + h] + base;
              if (masked) {
                const int row = min(row0 + nt * 8 + 2 * t + h, rows - 1);
                const int see_to = n - p.q_len + ((row * p.group_magic) >> 16) + 1;
                const int see_from = p.window > 0 ? see_to - p.window : 0;
                bool out0 = here + g < see_from, out1 = here + 8 + g < see_from;
                if constexpr (kMode == kAttnSinks) {
                  out0 = out0 && here + g >= p.sinks;
                  out1 = out1 && here + 8 + g >= p.sinks;
                }
                if (here + g >= see_to || out0) r0 = -__builtin_huge_valf();
                if (here + 8 + g >= see_to || out1) r1 = -__builtin_huge_valf();
              }
              float top = fmaxf(r0, r1);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
              const float mn = fmaxf(m[nt][h], top - kAttnLift);
              const AttnFall fall = attn_fall(m[nt][h] - mn);
              sum[nt][h] = kMode != kAttnPlain ? attn_halves(sum[nt][h], m[nt][h] - mn) : attn_lower(sum[nt][h], fall);
              m[nt][h] = mn;
#pragma unroll
              for (int j = 0; j < L::kTiles; ++j) {
                acc[nt][j][h] *= fall.hi;
                acc[nt][j][2 + h] *= fall.hi;
              }
              sc[nt][h] = r0 - mn;
              sc[nt][2 + h] = r1 - mn;
            }
          fresh = fresh && !some;
          if (small) {
#pragma unroll
            for (int nt = 0; nt < kN; ++nt)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                sum[nt][h] = fmaf(attn_ex2(sc[nt][h] - lv) + attn_ex2(sc[nt][2 + h] - lv), kAttnUnlift, sum[nt][h]);
            inv_vs = 0.0f;
          }
        }
        uint32_t pb[kN][2];
#pragma unroll
        for (int nt = 0; nt < kN; ++nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[nt][e] = attn_ex2(sc[nt][e]);
          sum[nt][0] = fmaf(sc[nt][0] + sc[nt][2], inv_vs, sum[nt][0]);
          sum[nt][1] = fmaf(sc[nt][1] + sc[nt][3], inv_vs, sum[nt][1]);
          pb[nt][0] = transpose8x8(pack_f16(sc[nt][0], sc[nt][1]));
          pb[nt][1] = transpose8x8(pack_f16(sc[nt][2], sc[nt][3]));
        }
        if constexpr (C::kAhead) {
          // the next strip's scores along with this one's sums (past the last strip: of no use, and none is made)
          asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 3) : "memory");
          __syncwarp();  // the next strip is there, and every lane is past the stage read last
          issue(before(stage));
          const uint32_t next_kb = ring + after(stage) * C::kStageBytes;
#pragma unroll
          for (int nt = 0; nt < kN; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.0f;
          static_assert(L::kWords == 2 * L::kVWords, "a V word for every two K words");
#pragma unroll
          for (int blk = 0; blk < L::kBlocks; ++blk) {
            uint32_t wk[2][L::kWords], wv[4][L::kVWords];
            k_load(next_kb, blk, wk);
            v_load(vb, blk, n - here, wv);
#pragma unroll
            for (int k = 0; k < L::kVWords; ++k) {
              score(wk, blk, 2 * k, sc);
              weigh(wv, blk, k, pb);
            }
          }
        } else {
#pragma unroll
          for (int blk = 0; blk < L::kBlocks; ++blk) {
            uint32_t w[4][L::kVWords];
            v_load(vb, blk, n - here, w);
#pragma unroll
            for (int k = 0; k < L::kVWords; ++k) weigh(w, blk, k, pb);
          }
        }
        stage = after(stage);
      }
    }

    // ---- the segment's end: join the warps ----
#pragma unroll
    for (int nt = 0; nt < kN; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) sum[nt][h] += __shfl_xor_sync(0xFFFFFFFFu, sum[nt][h], o);
        if (g == 0) ml[warp * C::kRows + nt * 8 + 2 * t + h] = make_float2(m[nt][h] + kAttnLift, sum[nt][h]);
      }
    // the stage that is neither being read nor being filled, the one before the next: 8 rows of dims, fp32
    const int idle = (warp * C::kStages + before(stage)) * C::kStageBytes;
    if (lane == 0) free_stage[warp] = idle;
    // 16-byte cell of word k, thread row g2 and query row r: places change by row, against bank conflicts
    auto cell = [](int r, int k, int g2) -> int { return ((r * (L::kTiles / 2) + k) * 8 + (g2 ^ (r & 6))) * 4; };
    const AttnPlace cur = places[which];
    const int used = min(C::kRows, rows - row0);
    const bool starts = cur.strip == 0, whole = starts && seg_end - at == cur.strips;
    const AttnItemEnd<kDim, C::kThreads, AttnModeParams<kMode>> item_end = {p, cur, row0, used};
    float* const part = item_end.part_of(blockIdx.x, starts ? 1 : 0);
    bool nans = false;
#pragma unroll
    for (int nt = 0; nt < kN; ++nt) {  // eight rows at a time
      if (nt * 8 >= used) break;
      float* const mine = reinterpret_cast<float*>(smem + idle);
#pragma unroll
      for (int k = 0; k < L::kTiles / 2; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float4*>(mine + cell(2 * t + h, k, g)) = make_float4(
              acc[nt][2 * k][h], acc[nt][2 * k][2 + h], acc[nt][2 * k + 1][h], acc[nt][2 * k + 1][2 + h]);
      __syncthreads();
      if (!kInt8 && nan_any != 0) {  // (set before that barrier, cleared behind the last: all threads alike)
        nans = true;
#pragma unroll 1
        for (int i = tid; i < 8 * kDim; i += C::kThreads) {
          const int r8 = i / kDim, d = i - r8 * kDim;
          if (nan_dims[nt * 8 + r8][d >> 5] >> (d & 31) & 1u) {
            const int2 place = L::v_place(d & ~3);
            reinterpret_cast<float*>(smem + free_stage[0])[cell(r8, place.x, place.y) + (d & 3)] =
                __int_as_float(0x7FC00000);
          }
        }
        __syncthreads();
      }
      if (C::kQInRegs && seg_end < end) q_load(places[which ^ 1], 0, qr);  // (arrives during the joining)
      for (int x = tid; x < 8 * (kDim / 4); x += C::kThreads) {
        const int r8 = x / (kDim / 4), d = (x - r8 * (kDim / 4)) * 4, r = nt * 8 + r8;
        if (r >= used) break;
        float top = kAttnFloor, l = 0.0f, most = 0.0f;
#pragma unroll
        for (int w = 0; w < C::kWarps; ++w) top = fmaxf(top, ml[w * C::kRows + r].x);
        const int2 place = L::v_place(d);
        const int from_cell = cell(r8, place.x, place.y);
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < C::kWarps; ++w) {
          const float2 o = ml[w * C::kRows + r];
          const float f = attn_ex2(o.x - top), fv = f * kAttnUnlift;  // (sums of weights up to 1, as those of weights are)
          const float* const cells = reinterpret_cast<const float*>(smem + free_stage[w]);
          const float4 a = *reinterpret_cast<const float4*>(cells + from_cell);
          v.x = fmaf(a.x, fv, v.x), v.y = fmaf(a.y, fv, v.y), v.z = fmaf(a.z, fv, v.z), v.w = fmaf(a.w, fv, v.w);
          l = kMode != kAttnPlain ? l + attn_halves(o.y, o.x - top) : fmaf(o.y, f, l);
          most = fmaxf(most, o.y);
        }
        if (kMode == kAttnPlain && attn_lacks(l, most)) {
          l = 0.0f;
#pragma unroll 1
          for (int w = 0; w < C::kWarps; ++w) {
            const float2 o = ml[w * C::kRows + r];
            l += attn_lower(o.y, attn_fall(o.x - top));
          }
        }
        if (whole) {
          item_end.store(r, d, v, top, l);
        } else {
          float* const o = part + r * (kDim + 4);
          __stcg(reinterpret_cast<float4*>(o + d), v);
          if (d == 0) __stcg(reinterpret_cast<float2*>(o + kDim), make_float2(top, l));
        }
      }
      __syncthreads();
    }
    if (nans) {
      for (int i = tid; i < C::kRows * (kDim / 32); i += C::kThreads) (&nan_dims[0][0])[i] = 0u;
      if (tid == 0) nan_any = 0;
      __syncthreads();
    }
    if (!whole)
      item_end.share(plan_words, line_before, ml, &last_flag, [] { __syncthreads(); });
    // on to the next item
    at = seg_end;
    which ^= 1;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

}  // namespace fp4
