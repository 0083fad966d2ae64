// k_route.cuh -- routing of tokens to experts (fp4gemv_moe_route).
//
// score = softmax(x) or sigmoid(x); key = score + bias, or the logit itself
// when neither a bias nor a sum of two keys needs the score; the topk largest
// keys within the topk_group strongest groups; weights = scores of those,
// renormalised on request.
//
// One warp per token, element e on lane e % 32, slot e / 32, so each slot is
// one contiguous load.  Keys are compared as unsigned integers that order
// like the floats (0: taken or absent), so a round of the selection is one
// redux.sync over each lane's best plus a vote; the lower index wins because
// a lane's slots are scanned upwards and equal lanes compare their indices.
//
// Keys have to come out the same for every order of summation, or experts
// whose keys nearly tie would change places: exp and the division are the
// IEEE-rounded or library ones, and the softmax's sum is carried as an
// unevaluated sum of two floats (Knuth's two-sum), ~48 bits.
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
  int sigmoid, renormalize;
  float scale;
};

constexpr int kRouteWarps = 4;  // tokens per CTA

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

// Warp-wide: the lane and slot of the largest key (ties: the lowest index).
template <int S>
__device__ __forceinline__ uint32_t warp_best(const uint32_t (&key)[S], uint32_t lane, uint32_t* index) {
  uint32_t best = key[0], slot = 0;
#pragma unroll
  for (int i = 1; i < S; ++i)
    if (key[i] > best) {
      best = key[i];
      slot = i;
    }
  const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
  *index = __reduce_min_sync(0xFFFFFFFFu, best == top ? slot * 32 + lane : 0xFFFFFFFFu);
  return top;
}

template <typename T, int S>
__global__ void __launch_bounds__(kRouteWarps * 32) moe_route_kernel(const RouteParams p) {
  const uint32_t lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5);
  if (threadIdx.x == 0) pdl_launch_dependents();
  pdl_wait();
  if (t >= p.M) return;
  const T* row = static_cast<const T*>(p.logits) + t * p.ldl;
  float x[S];
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const int e = i * 32 + lane;
    x[i] = e < p.E ? to_float(row[e]) : kNegInf;
    if (x[i] != x[i]) x[i] = kNegInf;
  }
  // scores where the keys or an unnormalised softmax need all of them
  const bool by_logit = p.bias == nullptr && p.group_top == 1;
  float top = 0.0f, sum = 1.0f;
  if (!p.sigmoid) {
    float m = x[0];
#pragma unroll
    for (int i = 1; i < S; ++i) m = fmaxf(m, x[i]);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    top = m;
  }
  auto raw_score = [&](float v) -> float {  // softmax: before the division by the sum
    if (p.sigmoid) return __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-v)));
    return v == kNegInf ? 0.0f : v == top ? 1.0f : expf(__fsub_rn(v, top));
  };
  uint32_t key[S];
  if (by_logit && (p.sigmoid || p.renormalize)) {
#pragma unroll
    for (int i = 0; i < S; ++i) key[i] = i * 32 + lane < p.E ? order_key(x[i]) : 0u;
  } else {
    float score[S];
#pragma unroll
    for (int i = 0; i < S; ++i) score[i] = raw_score(x[i]);  // (past E: x = -inf, sigmoid 0)
    if (!p.sigmoid) {
      float hi = 0.0f, lo = 0.0f;
#pragma unroll
      for (int i = 0; i < S; ++i) two_sum(hi, lo, score[i], 0.0f);
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const float h2 = __shfl_xor_sync(0xFFFFFFFFu, hi, o), l2 = __shfl_xor_sync(0xFFFFFFFFu, lo, o);
        two_sum(hi, lo, h2, l2);
      }
      sum = __fadd_rn(hi, lo);
    }
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int e = i * 32 + lane;
      if (by_logit) {
        key[i] = e < p.E ? order_key(x[i]) : 0u;
      } else {
        float s = p.sigmoid ? score[i] : sum > 0.0f ? __fdiv_rn(score[i], sum) : 0.0f;
        if (p.bias && e < p.E) s = __fadd_rn(s, __ldg(p.bias + e));
        key[i] = e < p.E ? order_key(s) : 0u;
      }
    }
  }
  if (p.n_group > 1) {
    // strengths: lane g ends with group g's
    const int size = p.E / p.n_group;
    uint32_t strength = 0;
    for (int g = 0; g < p.n_group; ++g) {
      uint32_t a = 0, b = 0;  // this lane's two best of the group
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const int e = i * 32 + lane;
        const uint32_t k = e >= g * size && e < (g + 1) * size ? key[i] : 0u;
        b = max(b, min(a, k));
        a = max(a, k);
      }
      const uint32_t first = __reduce_max_sync(0xFFFFFFFFu, a);
      uint32_t s = first;
      if (p.group_top == 2) {
        const uint32_t who = __ballot_sync(0xFFFFFFFFu, a == first);
        const uint32_t rest = lane == __ffs(who) - 1 ? b : a;
        const uint32_t second = __reduce_max_sync(0xFFFFFFFFu, rest);
        s = order_key(__fadd_rn(key_value(first), key_value(second)));
      }
      if (lane == g) strength = s;
    }
    uint32_t chosen = 0;
    for (int j = 0; j < p.topk_group; ++j) {
      const uint32_t best = __reduce_max_sync(0xFFFFFFFFu, strength);
      const uint32_t g = __ffs(__ballot_sync(0xFFFFFFFFu, strength == best)) - 1;
      chosen |= 1u << g;
      if (lane == g) strength = 0;
    }
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int e = i * 32 + lane;
      if (e < p.E && !((chosen >> (e / size)) & 1u)) key[i] = 0;
    }
  }
  // the selection: lane j keeps the j-th
  uint32_t mine = 0;
  float logit = kNegInf;
  for (int j = 0; j < p.topk; ++j) {
    uint32_t e;
    warp_best<S>(key, lane, &e);
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < S; ++i)
      if (static_cast<uint32_t>(i) == e >> 5) {
        v = x[i];
        if (lane == (e & 31)) key[i] = 0;
      }
    v = __shfl_sync(0xFFFFFFFFu, v, e & 31);
    if (lane == static_cast<uint32_t>(j)) {
      mine = e;
      logit = v;
    }
  }
  const bool live = lane < static_cast<uint32_t>(p.topk);
  float w = live ? raw_score(logit) : 0.0f;
  if (p.renormalize) {
    float total = w;
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
    w = total > 0.0f ? __fdiv_rn(w, total) : 0.0f;
  } else if (!p.sigmoid) {
    w = sum > 0.0f ? __fdiv_rn(w, sum) : 0.0f;
  }
  if (live) {
    p.ids[t * p.topk + lane] = static_cast<int32_t>(mine);
    p.weights[t * p.topk + lane] = w * p.scale;
  }
}

}  // namespace fp4
