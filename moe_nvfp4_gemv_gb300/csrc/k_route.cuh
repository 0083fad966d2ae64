// k_route.cuh -- routing of tokens to experts (fp4gemv_moe_route).
//
// score = softmax(x) or sigmoid(x); key = score + bias, or the logit itself
// when neither a bias nor a sum of two keys needs the score; the topk largest
// keys within the topk_group strongest groups; weights = scores of those,
// renormalised on request.
//
// kL lanes per token (a warp, or a part of one where there are many tokens),
// expert e on lane e / S of the token's, slot e % S: a lane's experts are
// neighbours, so of equal keys the lowest lane's lowest slot is the lower
// index.  Expert groups of any size begin at lanes of their own, a power of two
// of lanes each (group_lanes), unless that takes more than 16 slots.  Keys are
// compared as unsigned integers that order like the floats (0: taken or
// absent).  A round of the selection is a maximum over the lanes' best keys and
// a vote for the lane.
//
// Keys have to come out the same for every order of summation, or experts
// whose keys nearly tie would change places: exp and the division are the
// library's and the IEEE-rounded one, and the softmax's sum is carried as an
// unevaluated sum of two floats (Knuth's two-sum), ~48 bits.
//
// What bounds it.  Few tokens: the launch (one token of 128 experts, top 8:
// 1.9 us; 96 tokens of 256 with 8 groups 3.5).  Many: the selection's
// instructions, issue slots 64 % taken (20011 tokens of 60 experts, top 4, fp32:
// 7.2 us, where reading and writing would take 0.8; one warp per token 12.4).
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace fp4 {

struct RouteParams {
  const void* logits;
  int64_t ldl;
  const float* bias;
  int32_t* ids;
  float* weights;
  int M, E, topk;
  int n_group, topk_group, group_top;
  int group_lanes, lane_experts;  // lanes of a group and experts on each; 0: groups lie across lanes
  int sigmoid, renormalize;
  float scale;
};

constexpr int kRouteThreads = 128;

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_float<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

constexpr float kNegInf = -__builtin_huge_valf();

// Unsigned keys that order like the floats; NaN like -inf, -0 like +0.  The
// key of -inf is 0x007FFFFF, so 0 is free for "not here".
__device__ __forceinline__ uint32_t order_key(float x) {
  x = x == x ? x + 0.0f : kNegInf;
  const uint32_t b = __float_as_uint(x);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// (hi, lo) += (b, c) with the rounding error of hi + b kept in lo.
__device__ __forceinline__ void two_sum(float& hi, float& lo, float b, float c) {
  const float s = __fadd_rn(hi, b);
  const float bb = __fsub_rn(s, hi);
  const float err = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, bb)), __fsub_rn(b, bb));
  lo = __fadd_rn(lo, __fadd_rn(err, c));
  hi = s;
}

// a / b from r = 1 / b rounded to nearest: the quotient a r, its remainder by
// a fused operation and one correction give the correctly rounded quotient as
// long as nothing leaves the normal range (P. Markstein, IBM J. Res. Dev. 34,
// 1990); b in [1, 512] here, so a from 2^-100 on (0 is exact too).
__device__ __forceinline__ float divide_by(float a, float b, float r) {
  const float q = __fmul_rn(a, r);
  return __fmaf_rn(__fmaf_rn(-q, b, a), r, q);
}

// The largest of the token's lanes' values.
template <int kL>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  if constexpr (kL == 32) {
    return __reduce_max_sync(0xFFFFFFFFu, v);
  } else {
#pragma unroll
    for (int o = kL / 2; o; o >>= 1) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
  }
}
// The first of the token's lanes for which `is` holds (one does).
template <int kL>
__device__ __forceinline__ int first_lane(bool is, int lane) {
  const uint32_t vote = __ballot_sync(0xFFFFFFFFu, is);
  if constexpr (kL == 32) return __ffs(vote) - 1;
  else return __ffs((vote >> (lane & ~(kL - 1))) & ((1u << kL) - 1u)) - 1;
}

template <typename T, int kL, int S>
__global__ void __launch_bounds__(kRouteThreads) moe_route_kernel(const RouteParams p) {
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  const int lane = threadIdx.x & 31, sub = lane & (kL - 1);
  const int64_t t = (static_cast<int64_t>(blockIdx.x) * kRouteThreads + threadIdx.x) / kL;
  if (threadIdx.x == 0) pdl_launch_dependents();
  pdl_wait();
  const bool live = t < p.M;  // (the lanes of no token go along)
  const T* row = static_cast<const T*>(p.logits) + (live ? t : 0) * p.ldl;
  // the lane's experts: e0, e0 + 1, ... (cnt of them)
  int e0 = sub * S, cnt = min(max(p.E - e0, 0), S), group = 0;
  if (kL < 32) {  // (groups, if any, are whole lanes of S)
    if (p.n_group > 1) group = sub / p.group_lanes;
  } else if (p.group_lanes > 0) {
    const int size = p.E / p.n_group, within = (sub & (p.group_lanes - 1)) * p.lane_experts;
    group = sub / p.group_lanes;
    e0 = group * size + within;
    cnt = group < p.n_group ? min(max(size - within, 0), p.lane_experts) : 0;
  }
  float x[S];
  if (S * sizeof(T) >= 16 && cnt == S && (reinterpret_cast<uintptr_t>(row + e0) & 15u) == 0) {
    constexpr int kPer = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < S / kPer; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + e0) + i);
      const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
      for (int j = 0; j < kPer; ++j) x[i * kPer + j] = to_float(e[j]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < S; ++i) x[i] = i < cnt ? to_float(row[e0 + i]) : kNegInf;
  }
#pragma unroll
  for (int i = 0; i < S; ++i) x[i] = x[i] == x[i] ? x[i] : kNegInf;
  // scores where the keys or an unnormalised softmax need all of them
  const bool by_logit = p.bias == nullptr && p.group_top == 1;
  float top = 0.0f, sum = 1.0f;
  if (!p.sigmoid) {
    float m = x[0];
#pragma unroll
    for (int i = 1; i < S; ++i) m = fmaxf(m, x[i]);
#pragma unroll
    for (int o = kL / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
    top = m;
  }
  auto raw_score = [&](float v) -> float {  // softmax: before the division by the sum
    if (p.sigmoid) return __frcp_rn(__fadd_rn(1.0f, expf(-v)));
    return v == kNegInf ? 0.0f : v == top ? 1.0f : expf(__fsub_rn(v, top));
  };
  uint32_t key[S];
  if (by_logit) {
#pragma unroll
    for (int i = 0; i < S; ++i) key[i] = i < cnt ? order_key(x[i]) : 0u;
  }
  if (!by_logit || !(p.sigmoid || p.renormalize)) {
    float score[S];
#pragma unroll
    for (int i = 0; i < S; ++i) score[i] = raw_score(x[i]);  // (past E: x = -inf, score 0)
    if (!p.sigmoid) {
      float hi = score[0], lo = 0.0f;
#pragma unroll
      for (int i = 1; i < S; ++i) two_sum(hi, lo, score[i], 0.0f);
#pragma unroll
      for (int o = kL / 2; o; o >>= 1) {
        const float h2 = __shfl_xor_sync(kAll, hi, o), l2 = __shfl_xor_sync(kAll, lo, o);
        two_sum(hi, lo, h2, l2);
      }
      sum = __fadd_rn(hi, lo);
    }
    if (!by_logit) {
      if (!p.sigmoid && sum > 0.0f) {  // (no sum: every score is 0)
        const float inv = __fdiv_rn(1.0f, sum);
        float least = 1.0f;
#pragma unroll
        for (int i = 0; i < S; ++i) least = fminf(least, score[i] > 0.0f ? score[i] : 1.0f);
        if (least >= 0x1p-100f) {
#pragma unroll
          for (int i = 0; i < S; ++i) score[i] = divide_by(score[i], sum, inv);
        } else {
#pragma unroll 1
          for (int i = 0; i < S; ++i) {  // (registers are not indexed: the first moves to the end)
            const float q = __fdiv_rn(score[0], sum);
#pragma unroll
            for (int j = 0; j + 1 < S; ++j) score[j] = score[j + 1];
            score[S - 1] = q;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < S; ++i) {
        float s = score[i];
        if (p.bias && i < cnt) s = __fadd_rn(s, __ldg(p.bias + e0 + i));
        key[i] = i < cnt ? order_key(s) : 0u;
      }
    }
  }
  if (p.n_group > 1) {
    const int size = p.E / p.n_group, width = p.group_lanes;
    uint32_t chosen = 0;  // the groups that take part
    if (kL < 32 || width > 0) {
      // a group's two best keys by exchange within its lanes
      uint32_t a = 0, b = 0;
#pragma unroll
      for (int i = 0; i < S; ++i) {
        b = max(b, min(a, key[i]));
        a = max(a, key[i]);
      }
      for (int o = 1; o < width; o <<= 1) {
        const uint32_t a2 = __shfl_xor_sync(kAll, a, o), b2 = __shfl_xor_sync(kAll, b, o);
        b = max(min(a, a2), max(b, b2));
        a = max(a, a2);
      }
      const uint32_t strength =
          group >= p.n_group ? 0u : p.group_top == 2 ? order_key(__fadd_rn(key_value(a), key_value(b))) : a;
      // its place among the groups: those that are stronger, or as strong and earlier
      int before = 0;
      for (int g = 0; g < p.n_group; ++g) {
        const uint32_t other = __shfl_sync(kAll, strength, (lane & ~(kL - 1)) + g * width);
        before += other > strength || (other == strength && g < group);
      }
      if (before >= p.topk_group) {
#pragma unroll
        for (int i = 0; i < S; ++i) key[i] = 0;
      }
    } else {
      uint32_t strength[32 / kL];  // group g: lane g % kL's entry g / kL
#pragma unroll
      for (int i = 0; i < 32 / kL; ++i) strength[i] = 0;
      for (int g = 0; g < p.n_group; ++g) {
        uint32_t a = 0, b = 0;  // this lane's two best of the group
#pragma unroll
        for (int i = 0; i < S; ++i) {
          const uint32_t k = e0 + i >= g * size && e0 + i < (g + 1) * size ? key[i] : 0u;
          b = max(b, min(a, k));
          a = max(a, k);
        }
        uint32_t s = lanes_max<kL>(a);
        if (p.group_top == 2) {
          const int who = first_lane<kL>(a == s, lane);
          const uint32_t second = lanes_max<kL>(sub == who ? b : a);
          s = order_key(__fadd_rn(key_value(s), key_value(second)));
        }
#pragma unroll
        for (int i = 0; i < 32 / kL; ++i)
          if (g == i * kL + sub) strength[i] = s;
      }
      for (int j = 0; j < p.topk_group; ++j) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < 32 / kL; ++i) best = max(best, strength[i]);
        best = lanes_max<kL>(best);
        int g = 32;  // the lowest group that has it: the lowest entry's lowest lane
#pragma unroll
        for (int i = 0; i < 32 / kL; ++i) {
          const uint32_t vote = __ballot_sync(kAll, strength[i] == best) >> (lane & ~(kL - 1));
          const uint32_t here = kL == 32 ? vote : vote & ((1u << (kL & 31)) - 1u);
          if (g == 32 && here != 0) g = i * kL + __ffs(here) - 1;
        }
        chosen |= 1u << g;
#pragma unroll
        for (int i = 0; i < 32 / kL; ++i)
          if (g == i * kL + sub) strength[i] = 0;
      }
#pragma unroll
      for (int i = 0; i < S; ++i)
        if (e0 + i < p.E && !((chosen >> ((e0 + i) / size)) & 1u)) key[i] = 0;
    }
  }
  // the selection: the token's lane j keeps the j-th (and lane j % kL the later ones)
  constexpr int kKeep = 32 / kL;
  int mine[kKeep];
  float logit[kKeep];
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    mine[i] = 0;
    logit[i] = kNegInf;
  }
  for (int j = 0; j < p.topk; ++j) {
    uint32_t best = key[0], best_x = __float_as_uint(x[0]);
    int slot = 0;
#pragma unroll
    for (int i = 1; i < S; ++i)
      if (key[i] > best) {
        best = key[i];
        best_x = __float_as_uint(x[i]);
        slot = i;
      }
    const uint32_t most = lanes_max<kL>(best);
    const int who = first_lane<kL>(best == most, lane);
    // (the winner, and its logit where that is not the key itself)
    const int e = __shfl_sync(kAll, e0 + slot, (lane & ~(kL - 1)) + who);
    const float v = by_logit ? key_value(most)
                             : __uint_as_float(__shfl_sync(kAll, best_x, (lane & ~(kL - 1)) + who));
#pragma unroll
    for (int i = 0; i < S; ++i)
      if (kL < 32 ? e0 + i == e : sub == who && slot == i) key[i] = 0;
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
      if (j == i * kL + sub) {
        mine[i] = e;
        logit[i] = v;
      }
  }
  float w[kKeep], total = 0.0f;
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    w[i] = i * kL + sub < p.topk ? raw_score(logit[i]) : 0.0f;
    total += w[i];
  }
  if (p.renormalize) {
#pragma unroll
    for (int o = kL / 2; o; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
  } else {
    total = p.sigmoid ? 1.0f : sum;
  }
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    const int j = i * kL + sub;
    if (live && j < p.topk) {
      p.ids[t * p.topk + j] = mine[i];
      p.weights[t * p.topk + j] = (total > 0.0f ? __fdiv_rn(w[i], total) : 0.0f) * p.scale;
    }
  }
}

}  // namespace fp4
