// k_logprobs.cuh -- log probabilities of given tokens, their rank, the
// entropy and the top alternatives (fp4gemv_token_logprobs).
//
// One pass over the row with running statistics (m, s, u): the maximum so
// far, s = sum 2^(c (x - m)) and u = sum 2^(c (x - m)) (x - m), c =
// inv_temperature log2(e); a new maximum rescales them, u to
// f u + (f s) (m - m'), f = 2^(c (m - m')).  u is in the logits' units, and f s
// comes before its product: differences of logits are finite, c times them or s
// times them need not be, and a weight or f of 0 has to leave 0.  At the end
//   log Z = ln s,  H = log Z - inv_temperature u / s,
//   logprob = (x - m) inv_temperature - log Z.
//
// Top n without sorting the row: the threads form 64 groups, each with the
// maximum of its elements (the running maximum, which the softmax needs
// anyway); the n-th largest group maximum is a lower bound of the n-th largest
// logit, so only threads whose own maximum reaches it look at their elements
// again, and the elements that reach it, some n to 2 n of them, are ranked by
// counting.  Where more reach it than the buffer holds (ties: a row of masked
// or equal logits), the n-th largest of some that were collected is a better
// bound, indices included, and the collection is repeated.
//
// A row is split over the CTAs of a cluster when there are few rows; they
// meet in the shared memory of the cluster's first CTA.
//
// What bounds it.  Many rows: HBM (2048 rows of 131072 bf16: 92.6 us, 0.87 of the
// measured copy bandwidth), with the exponentials close behind (issue slots 60 %
// taken; one scalar chain per element 114 us, paired fp32 sums 101, loads of a
// slot ahead 92; the difference to the maximum as an operation of its own 92.6).
// Few: latency; one row of 128003 6.2 us (2.1 of it the top
// alternatives), 64 rows of 100001 fp32 9.8.  Measured and not taken: 512 or 1024
// threads (fewer CTAs to fill the phases without loads), double-buffered loads
// (104 us for the 2048 rows).
#pragma once

#include "k_route.cuh"

namespace fp4 {

struct LogprobParams {
  const void* logits;
  int64_t ldl;
  const int32_t* tokens;
  float* logprob;
  int32_t* rank;
  float* entropy;
  int32_t* top_ids;
  float* top_logprobs;
  uint32_t* err;
  int V, n;
  float inv_t;
};

constexpr int kLpThreads = 256;
constexpr int kLpResident = 5;  // CTAs per SM
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpGroups = 64;
constexpr int kMaxCand = 512;
constexpr int kRaiseFrom = 256;  // collected elements that a better bound is taken from
constexpr int kLpMaxCluster = 8;
// Logits at or below this are masked: probability 0.  The statistics see them
// as this value, so that no difference of two finite ones is a NaN or overflows.
constexpr float kMasked = -0x1p100f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

struct LpStat {
  float m, s, u;
};
// The warp's statistics as one, in every lane: the maximum first, then sums
// of what each lane has against it (a shorter chain than joining pairs).
__device__ __forceinline__ void lp_join_warp(LpStat& a, float c) {
  float m = a.m;
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  const float d = a.m - m, f = ex2(d * c);
  a.s *= f;
  a.u = fmaf(a.s, d, f * a.u);
  a.m = m;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    a.s += __shfl_xor_sync(0xFFFFFFFFu, a.s, o);
    a.u += __shfl_xor_sync(0xFFFFFFFFu, a.u, o);
  }
}

// What a thread gathers: the statistics with s and u in two halves, and the
// number of logits above the given token's.
struct LpThread {
  float m;
  uint64_t s, u;
  int above;
};

// A new running maximum, if bm is one.
__device__ __forceinline__ void lp_raise(LpThread& st, float bm, float c) {
  if (bm > st.m) {
    const float d = st.m - bm, e = ex2(d * c);
    const uint64_t f = pair(e, e), d2 = pair(d, d);
    st.s = mul2(f, st.s);
    st.u = fma2(st.s, d2, mul2(f, st.u));
    st.m = bm;
  }
}
// Two logits (masked ones already at kMasked) into the sums; c2 = (c, c), m2 = (-m, -m).  The difference comes first: it is
// 0 for the maximum itself and rounds to its own size, where x c - RN(m c) would carry the rounding of m c, which grows
// with |m| / temperature, into every term and into log Z.
__device__ __forceinline__ void lp_sum(LpThread& st, uint64_t x, uint64_t c2, uint64_t m2) {
  const uint64_t d = add2(x, m2);
  const float2 df = unpair(mul2(d, c2));
  const uint64_t e = pair(ex2(df.x), ex2(df.y));
  st.s = add2(st.s, e);
  st.u = fma2(e, d, st.u);
}

template <typename T>
struct LpVec {
  static constexpr int kN = 16 / sizeof(T);
};

template <typename T>
__device__ __forceinline__ void lp_unpack(const uint4& v, float (&x)[LpVec<T>::kN]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      x[i] = __uint_as_float(w[i]);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

// Adds kW words of logits (each one fp32 or two 16-bit ones).  Rows' given
// tokens are mostly likely ones, so a batch none of whose logits is above
// the token's is the usual case and is not counted through.
template <typename T, int kW>
__device__ __forceinline__ void lp_add(LpThread& st, const uint32_t (&w)[kW], float xr, float c) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    auto two = [](uint32_t v) { return *reinterpret_cast<const __nv_bfloat162*>(&v); };
    __nv_bfloat162 top = two(w[0]);
#pragma unroll
    for (int i = 1; i < kW; ++i) top = __hmax2(top, two(w[i]));
    const float bm = fmaxf(__low2float(top), __high2float(top));
    lp_raise(st, bm, c);
    if (bm > xr) {
      const __nv_bfloat162 limit = __float2bfloat162_rn(xr);  // (a logit of the row: exact)
      __nv_bfloat162 n = __float2bfloat162_rn(0.0f);
#pragma unroll
      for (int i = 0; i < kW; ++i) n = __hadd2(n, __hgt2(two(w[i]), limit));  // (at most kW: exact)
      st.above += static_cast<int>(__low2float(n) + __high2float(n));
    }
    const uint64_t c2 = pair(c, c), m2 = pair(-st.m, -st.m);
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      const __nv_bfloat162 x = __hmax2_nan(two(w[i]), __float2bfloat162_rn(kMasked));
      const uint32_t b = *reinterpret_cast<const uint32_t*>(&x);
      lp_sum(st, pair(__uint_as_float(b << 16), __uint_as_float(b & 0xFFFF0000u)), c2, m2);
    }
  } else {
    constexpr int kX = std::is_same<T, float>::value ? kW : 2 * kW;
    float x[kX];
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      if constexpr (std::is_same<T, float>::value) {
        x[i] = __uint_as_float(w[i]);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[2 * i] = f.x, x[2 * i + 1] = f.y;
      }
    }
    float bm = x[0];
#pragma unroll
    for (int i = 1; i < kX; ++i) bm = fmaxf(bm, x[i]);
    lp_raise(st, bm, c);
    if (bm > xr) {
#pragma unroll
      for (int i = 0; i < kX; ++i) st.above += x[i] > xr;
    }
    const uint64_t c2 = pair(c, c), m2 = pair(-st.m, -st.m);
#pragma unroll
    for (int i = 0; i < kX; i += 2)
      lp_sum(st, pair(max_nan(x[i], kMasked), max_nan(x[i + 1], kMasked)), c2, m2);
  }
}

__device__ __forceinline__ uint64_t lp_key(float x, uint32_t i) {
  return (static_cast<uint64_t>(order_key(x)) << 32) | (0xFFFFFFFFu - i);
}

// How many of the keys are above k: the list is followed by zeros up to a
// multiple of 8 keys (two per load, eight in flight).
__device__ __forceinline__ int count_above(const uint64_t* list, int n, uint64_t k) {
  int r = 0;
#pragma unroll 1
  for (int j = 0; j < n; j += 8) {
    ulonglong2 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = reinterpret_cast<const ulonglong2*>(list + j)[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) r += (v[i].x > k) + (v[i].y > k);
  }
  return r;
}

struct LpShared {
  LpStat stat[kLpMaxCluster][kLpWarps];
  int count[kLpMaxCluster][kLpWarps];
  uint32_t group[kLpGroups];
  unsigned long long bound;
  int n_flag, n_cand;
  uint16_t flagged[kLpThreads];
  alignas(16) uint64_t cand[kMaxCand];
  alignas(16) uint64_t top[kLpMaxCluster * 32];
};

template <typename T>
__global__ void __launch_bounds__(kLpThreads, kLpResident) token_logprobs_kernel(const LogprobParams p) {
  __shared__ LpShared sh;
  constexpr int kN = LpVec<T>::kN;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t C = cluster_nctarank(), rank = cluster_ctarank();
  const int64_t t = blockIdx.x / C;
  if (tid == 0) pdl_launch_dependents();
  if (tid < kLpGroups) sh.group[tid] = 0;
  if (tid == 0) {
    sh.n_flag = 0;
    sh.n_cand = 0;
  }
  if (p.n > 0) {
    for (int i = tid; i < kMaxCand; i += kLpThreads) sh.cand[i] = 0;
    for (int i = tid; i < kLpMaxCluster * 32; i += kLpThreads) sh.top[i] = 0;
  }
  // (what was cleared, before any thread adds to it: the first store into another CTA waits for all of the cluster)
  if (C > 1) cluster_arrive();
  else __syncthreads();
  pdl_wait();
  const T* row = static_cast<const T*>(p.logits) + t * p.ldl;
  const int token = __ldg(p.tokens + t);
  const bool valid = token >= 0 && token < p.V;
  const float xt = valid ? to_float(row[token]) : 0.0f;
  const float xr = xt == xt ? xt : kNegInf;  // what ranks compare with
  const float c = p.inv_t * 1.4426950408889634f;

  // the row as single elements up to a 16-byte boundary, whole vectors, and
  // single elements again; this CTA's vectors are [v0, v1), and every thread
  // takes every kLpThreads-th of them
  const int lead = static_cast<int>(
      min(static_cast<uint64_t>(p.V), ((16u - (reinterpret_cast<uintptr_t>(row) & 15u)) & 15u) / sizeof(T)));
  const int nvec = (p.V - lead) / kN;
  const int v0 = static_cast<int>(static_cast<int64_t>(nvec) * rank / C);
  const int v1 = static_cast<int>(static_cast<int64_t>(nvec) * (rank + 1) / C);
  const uint4* vec = reinterpret_cast<const uint4*>(row + lead);
  // (the single elements, at most 2 (kN - 1), belong to the first CTA)
  const int singles = rank == 0 ? p.V - nvec * kN : 0;
  auto single_index = [&](int i) { return i < lead ? i : nvec * kN + i; };

  LpThread mine = {kMasked, 0ull, 0ull, 0};
  if (tid < singles) {
    const float x = to_float(row[single_index(tid)]);
    lp_raise(mine, x, c);
    mine.above += x > xr;
    const float d = max_nan(x, kMasked) - mine.m, e = ex2(d * c);
    mine.s = add2(mine.s, pair(e, 0.0f));
    mine.u = add2(mine.u, pair(e * d, 0.0f));
  }
  constexpr int kU = 4;  // vectors in flight per thread
  int v = v0 + tid;
  for (; v + (kU - 1) * kLpThreads < v1; v += kU * kLpThreads) {
    uint32_t w[4 * kU];
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      const uint4 raw = __ldg(vec + v + j * kLpThreads);
      w[4 * j] = raw.x, w[4 * j + 1] = raw.y, w[4 * j + 2] = raw.z, w[4 * j + 3] = raw.w;
    }
    lp_add<T, 4 * kU>(mine, w, xr, c);
  }
  {
    uint32_t w[kU - 1][4];  // the last few, loaded together
#pragma unroll
    for (int j = 0; j < kU - 1; ++j)
      if (v + j * kLpThreads < v1) {
        const uint4 raw = __ldg(vec + v + j * kLpThreads);
        w[j][0] = raw.x, w[j][1] = raw.y, w[j][2] = raw.z, w[j][3] = raw.w;
      }
#pragma unroll
    for (int j = 0; j < kU - 1; ++j)
      if (v + j * kLpThreads < v1) lp_add<T, 4>(mine, w[j], xr, c);
  }
  const float2 s2 = unpair(mine.s), u2 = unpair(mine.u);
  LpStat st = {mine.m, s2.x + s2.y, u2.x + u2.y};
  int above = mine.above;

  const float own_max = st.m;
  const bool any = tid < singles || v0 + tid < v1;
  lp_join_warp(st, c);
  above = __reduce_add_sync(0xFFFFFFFFu, above);
  // statistics, counts and winners meet in the first CTA's shared memory
  if (C > 1) cluster_wait();
  if (lane == 0) {
    const uint32_t a = mapa(smem_u32(&sh.stat[rank][warp]), 0), b = mapa(smem_u32(&sh.count[rank][warp]), 0);
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(st.m) : "memory");
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a + 4), "f"(st.s) : "memory");
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a + 8), "f"(st.u) : "memory");
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(b), "r"(above) : "memory");
  }
  const int n = p.n;
  if (n > 0) {
    // (a thread with masked elements only counts with the least key: bounds
    // then lie above all masked values or below everything)
    const uint32_t own = any ? order_key(own_max > kMasked ? own_max : kNegInf) : 0u;
    if (own) atomicMax(&sh.group[tid & (kLpGroups - 1)], own);
    __syncthreads();
    {  // four threads rank a group among the others
      static_assert(kLpThreads == 4 * kLpGroups, "");
      const int mine_at = tid >> 2;
      const uint32_t group_max = sh.group[mine_at];
      int r = 0;
#pragma unroll 4
      for (int k = 0; k < kLpGroups / 4; ++k) {
        const int j = 4 * k + (tid & 3);
        const uint32_t o = sh.group[j];
        r += o > group_max || (o == group_max && j < mine_at);
      }
      r += __shfl_xor_sync(0xFFFFFFFFu, r, 1);
      r += __shfl_xor_sync(0xFFFFFFFFu, r, 2);
      if (r == n - 1 && (tid & 3) == 0) sh.bound = static_cast<unsigned long long>(group_max) << 32;
    }
    __syncthreads();
    uint64_t bound = sh.bound;
    if (own && own >= static_cast<uint32_t>(bound >> 32))
      sh.flagged[atomicAdd(&sh.n_flag, 1)] = static_cast<uint16_t>(tid);
    __syncthreads();
    const int nf = sh.n_flag;
    const int steps = (v1 - v0 + kLpThreads - 1) / kLpThreads;
    float bound_value = key_value(static_cast<uint32_t>(bound >> 32));
    auto offer = [&](float x, int i) {
      const uint64_t k = lp_key(x, i);
      if (k >= bound) {
        const int at = atomicAdd(&sh.n_cand, 1);
        if (at < kMaxCand) sh.cand[at] = k;
      }
    };
    const int flag_bits = nf > 1 ? 32 - __clz(nf - 1) : 0;  // their number rounded up to a power of two
    int nc;
    for (;;) {
      for (int w = tid; w < steps << flag_bits; w += kLpThreads) {
        const int f = w & ((1 << flag_bits) - 1);
        const int j = f < nf ? v0 + sh.flagged[f] + (w >> flag_bits) * kLpThreads : v1;
        if (j < v1) {
          float x[kN];
          lp_unpack<T>(__ldg(vec + j), x);
          uint32_t hits = 0;  // (a NaN goes on to its key)
#pragma unroll
          for (int i = 0; i < kN; ++i) hits |= x[i] < bound_value ? 0u : 1u << i;
          for (; hits; hits &= hits - 1) {
            const int i = lead + j * kN + __ffs(hits) - 1;
            offer(to_float(row[i]), i);
          }
        }
      }
      if (tid < singles) offer(to_float(row[single_index(tid)]), single_index(tid));
      __syncthreads();
      nc = sh.n_cand;
      if (nc <= kMaxCand) break;
      // at least n elements reach the n-th largest of kRaiseFrom of them
      if (tid < kRaiseFrom) {
        const uint64_t k = sh.cand[tid];
        int r = 0;
        for (int j = 0; j < kRaiseFrom; ++j) r += sh.cand[j] > k;
        if (r == n - 1) sh.bound = k;
      }
      __syncthreads();
      bound = sh.bound;
      bound_value = key_value(static_cast<uint32_t>(bound >> 32));
      if (tid == 0) sh.n_cand = 0;
      for (int i = tid; i < kMaxCand; i += kLpThreads) sh.cand[i] = 0;
      __syncthreads();
    }
    for (int i = tid; i < nc; i += kLpThreads) {
      const uint64_t k = sh.cand[i];
      const int r = count_above(sh.cand, nc, k);
      if (r < n) {
        const uint32_t a = mapa(smem_u32(&sh.top[rank * n + r]), 0);
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(k) : "memory");
      }
    }
    // (a slice of fewer than n elements leaves zeros)
  }

  if (C == 1) __syncthreads();
  else cluster_sync();
  if (rank != 0) return;
  // one warp-wide join of all partial statistics, by every warp alike
  LpStat all = {kMasked, 0.0f, 0.0f};
  int total = 0;
  static_assert(kLpMaxCluster * kLpWarps <= 64, "");
  if (lane < static_cast<int>(C) * kLpWarps) {
    all = (&sh.stat[0][0])[lane];
    total = (&sh.count[0][0])[lane];
    if (lane + 32 < static_cast<int>(C) * kLpWarps) {
      const LpStat b = (&sh.stat[0][0])[lane + 32];
      total += (&sh.count[0][0])[lane + 32];
      const float m = fmaxf(all.m, b.m), da = all.m - m, db = b.m - m, fa = ex2(da * c), fb = ex2(db * c);
      const float sa = fa * all.s, sb = fb * b.s;
      all.u = fmaf(sa, da, fa * all.u) + fmaf(sb, db, fb * b.u);
      all.s = sa + sb;
      all.m = m;
    }
  }
  lp_join_warp(all, c);
  total = __reduce_add_sync(0xFFFFFFFFu, total);
  const bool empty = all.m <= kMasked && all.s == all.s;  // (a NaN keeps the statistics' NaN)
  const float log_z = logf(all.s);
  auto logprob_of = [&](float x) {
    return empty || (x <= kMasked && log_z == log_z) ? kNegInf : fmaf(x - all.m, p.inv_t, -log_z);
  };
  if (tid == 0) {
    p.entropy[t] = empty ? 0.0f : log_z - p.inv_t * (all.u / all.s);
    if (valid) {
      p.logprob[t] = logprob_of(xt);
      p.rank[t] = 1 + total;
    } else {
      raise_error(p.err, FP4_ERR_BADIDX);
    }
  }
  if (n > 0) {
    // The CTAs' winners, each ranked among all (one CTA's are in order already): by counting, or, where they are many, by
    // its place in its own CTA's list and a binary search in the others'.  Counting / searching, us: top 20 of a row of
    // 128003 6.6 / 6.1, top 5 of 64 rows of 100001 9.5 / 9.9.
    const int have = static_cast<int>(C) * n;
    for (int i = tid; i < have; i += kLpThreads) {
      const uint64_t k = sh.top[i];
      int r = i;
      if (have <= 64) {
        if (C > 1) r = count_above(sh.top, have, k);
      } else {
        const int own_list = i / n;
        int above[kLpMaxCluster];
#pragma unroll
        for (int l = 0; l < kLpMaxCluster; ++l) above[l] = 0;
#pragma unroll
        for (int step = 32; step > 0; step >>= 1)
#pragma unroll
          for (int l = 0; l < kLpMaxCluster; ++l) {
            const int at = above[l] + step;
            const uint64_t o = sh.top[l * n + min(at, n) - 1];  // (lists past the cluster's: zeros)
            above[l] += at <= n && o > k ? step : 0;
          }
        r -= own_list * n;
#pragma unroll
        for (int l = 0; l < kLpMaxCluster; ++l) r += l == own_list ? 0 : above[l];
      }
      if (r < n && k != 0) {
        const int64_t o = t * n + r;
        p.top_ids[o] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(k));
        p.top_logprobs[o] = logprob_of(key_value(static_cast<uint32_t>(k >> 32)));
      }
    }
  }
}

}  // namespace fp4
