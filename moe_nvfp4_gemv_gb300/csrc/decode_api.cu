// decode_api.cu -- the C ABI of the decode step's operators (see
// include/fp4gemv_decode.h).  Host side only: argument validation before any
// launch, the choice of row tiles, and the launches.
#include <cmath>
#include <cstdint>

#include "decode_launch.h"
#include "fp4gemv_decode.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

fp4gemv_status from_cuda(cudaError_t e) { return e == cudaSuccess ? FP4GEMV_OK : FP4GEMV_ERR_CUDA; }

// The least x with 2^x = n for the block sizes, -1 for others.
int block_log2(int n) { return n == 16 ? 4 : n == 32 ? 5 : n == 64 ? 6 : n == 128 ? 7 : -1; }

bool dim_ok(int d) { return d == 64 || d == 96 || d == 128 || d == 256; }

// Sizes and flags of a cache; *nulls and *crooked for the later checks.
fp4gemv_status check_cache(const fp4gemv_kv_cache* c, bool* nulls, bool* crooked) {
  if (!c) return FP4GEMV_ERR_INVALID_ARG;
  if (c->num_blocks < 1 || c->kv_heads < 1 || c->block_size < 1 || c->head_dim < 1) return FP4GEMV_ERR_INVALID_ARG;
  if (c->format != FP4GEMV_KV_E4M3 && c->format != FP4GEMV_KV_INT8) return FP4GEMV_ERR_INVALID_ARG;
  if (block_log2(c->block_size) < 0 || !dim_ok(c->head_dim) || c->kv_heads > 65535) return FP4GEMV_ERR_UNSUPPORTED_SHAPE;
  *nulls = !c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale;
  *crooked = !aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4);
  return FP4GEMV_OK;
}

}  // namespace

fp4gemv_status fp4gemv_kv_append(const fp4gemv_kv_cache* cache, const void* k, int64_t ldk, const void* v, int64_t ldv,
                                 int dtype, int T, const int32_t* cu_new, const int32_t* block_table, int max_blocks,
                                 const int32_t* seq_lens, int B, int pdl, cudaStream_t stream) {
  bool nulls, crooked;
  fp4gemv_status st = check_cache(cache, &nulls, &crooked);
  if (st != FP4GEMV_OK) return st;
  if (pdl != 0 && pdl != 1) return FP4GEMV_ERR_INVALID_ARG;
  if (dtype != FP4GEMV_BF16 && dtype != FP4GEMV_F16) return FP4GEMV_ERR_INVALID_ARG;
  const int64_t width = static_cast<int64_t>(cache->kv_heads) * cache->head_dim;
  if (T < 0 || B < 1 || max_blocks < 1 || ldk < width || ldv < width) return FP4GEMV_ERR_INVALID_ARG;
  if (!cu_new && T % B != 0) return FP4GEMV_ERR_INVALID_ARG;
  if (B > FP4GEMV_KV_MAX_BATCH || static_cast<int64_t>(max_blocks) * cache->block_size > (1ll << 30) || T > (1 << 30))
    return FP4GEMV_ERR_UNSUPPORTED_SHAPE;
  if (crooked || !aligned(k, 16) || !aligned(v, 16) || ldk % 8 != 0 || ldv % 8 != 0 || !aligned(cu_new, 4) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4))
    return FP4GEMV_ERR_MISALIGNED;
  if (nulls || !block_table || !seq_lens) return FP4GEMV_ERR_INVALID_ARG;
  if (T == 0) return FP4GEMV_OK;
  if (!k || !v) return FP4GEMV_ERR_INVALID_ARG;
  uint32_t* err = nullptr;
  st = fp4::current_device_state(&err, nullptr);
  if (st != FP4GEMV_OK) return st;
  fp4::KvAppendParams p = {};
  p.src[0] = static_cast<const uint16_t*>(k);
  p.src[1] = static_cast<const uint16_t*>(v);
  p.ld[0] = ldk;
  p.ld[1] = ldv;
  p.codes[0] = cache->k_codes;
  p.codes[1] = cache->v_codes;
  p.scale[0] = cache->k_scale;
  p.scale[1] = cache->v_scale;
  p.cu = cu_new;
  p.table = block_table;
  p.lens = seq_lens;
  p.err = err;
  p.uniform = T / B;
  p.B = B;
  p.T = T;
  p.max_blocks = max_blocks;
  p.num_blocks = cache->num_blocks;
  p.heads = cache->kv_heads;
  p.block_log2 = block_log2(cache->block_size);
  p.dim = cache->head_dim;
  fp4::count_launch();
  return from_cuda(fp4::launch_kv_append(p, cache->format == FP4GEMV_KV_INT8, dtype == FP4GEMV_F16, pdl, stream));
}

// [arrival counters, three for each CTA | partials, two for each CTA]
static size_t attn_counter_bytes(int ctas) { return (static_cast<size_t>(ctas) * 12 + 15) / 16 * 16; }

size_t fp4gemv_kv_attention_workspace_bytes(int head_dim) {
  if (!dim_ok(head_dim)) return 0;
  int sms = 0;
  if (fp4::current_device_state(nullptr, &sms) != FP4GEMV_OK) return 0;
  const int ctas = fp4::kv_attention_max_ctas(sms);
  return attn_counter_bytes(ctas) + static_cast<size_t>(ctas) * 2 * fp4::kAttnMaxRows * (head_dim + 4) * 4;
}

uint64_t fp4gemv_stream_capture_id(cudaStream_t stream) {
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  unsigned long long id = 0;
  if (cudaStreamGetCaptureInfo(stream, &status, &id) != cudaSuccess) {
    cudaGetLastError();  // (the legacy stream beside a capture: it takes no part)
    return 0;
  }
  return status == cudaStreamCaptureStatusActive ? id : 0;
}

fp4gemv_status fp4gemv_kv_attention(const fp4gemv_kv_cache* cache, const void* q, int64_t ldq, int dtype, int heads,
                                    int q_len, const int32_t* block_table, int max_blocks, const int32_t* seq_lens,
                                    int B, float sm_scale, int window, void* out, int64_t ldo, float* lse,
                                    void* workspace, size_t workspace_bytes, int pdl, cudaStream_t stream) {
  bool nulls, crooked;
  fp4gemv_status st = check_cache(cache, &nulls, &crooked);
  if (st != FP4GEMV_OK) return st;
  if (pdl != 0 && pdl != 1) return FP4GEMV_ERR_INVALID_ARG;
  if (dtype != FP4GEMV_BF16 && dtype != FP4GEMV_F16) return FP4GEMV_ERR_INVALID_ARG;
  if (heads < 1 || q_len < 1 || B < 1 || max_blocks < 1 || window < 0 || !std::isfinite(sm_scale))
    return FP4GEMV_ERR_INVALID_ARG;
  const int64_t width = static_cast<int64_t>(heads) * cache->head_dim;
  if (ldq < width || ldo < width) return FP4GEMV_ERR_INVALID_ARG;
  const int group = heads / cache->kv_heads;
  if (heads % cache->kv_heads != 0 || group > FP4GEMV_KV_MAX_GROUP || q_len > FP4GEMV_KV_MAX_QLEN ||
      B > FP4GEMV_KV_MAX_BATCH)
    return FP4GEMV_ERR_UNSUPPORTED_SHAPE;
  // row tiles: the 8, 16 or 32 rows that a pass over the codes serves
  // (head_dim 256 has registers for 16).  One pass of 16 rows or two of 8, 32
  // sequences of 16384 tokens, 8 KV heads: 185 us against 350.
  const int rows = q_len * group;
  const int row_units = rows <= 8 ? 1 : rows <= 16 || cache->head_dim > 128 ? 2 : 4;
  const int row_tiles = (rows + 8 * row_units - 1) / (8 * row_units);
  const int64_t tokens = static_cast<int64_t>(max_blocks) * cache->block_size;
  // (32-bit: places on the line of strips, a quarter more with padding, and strips of the cache)
  if (tokens > (1ll << 30) || static_cast<int64_t>(cache->kv_heads) * row_tiles >= (1 << 20) ||
      (static_cast<double>(tokens) / 16 + fp4::kAttnTcItemCost + 8) * B * cache->kv_heads * row_tiles >= 1.2e9 ||
      static_cast<double>(cache->num_blocks) * cache->kv_heads * (cache->block_size / 16) >= 2147483647.0)
    return FP4GEMV_ERR_UNSUPPORTED_SHAPE;
  if (crooked || !aligned(q, 16) || !aligned(out, 16) || ldq % 8 != 0 || ldo % 8 != 0 || !aligned(lse, 4) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(workspace, 16))
    return FP4GEMV_ERR_MISALIGNED;
  if (nulls || !q || !out || !block_table || !seq_lens || !workspace) return FP4GEMV_ERR_INVALID_ARG;
  uint32_t* err = nullptr;
  int sms = 0;
  st = fp4::current_device_state(&err, &sms);
  if (st != FP4GEMV_OK) return st;
  if (workspace_bytes < fp4gemv_kv_attention_workspace_bytes(cache->head_dim)) return FP4GEMV_ERR_INVALID_ARG;
  fp4::KvAttnTcParams p = {};
  p.k_codes = cache->k_codes;
  p.v_codes = cache->v_codes;
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.q = static_cast<const uint16_t*>(q);
  p.ldq = ldq;
  p.out = static_cast<uint16_t*>(out);
  p.ldo = ldo;
  p.lse = lse;
  p.table = block_table;
  p.lens = seq_lens;
  p.err = err;
  p.arrived = static_cast<uint32_t*>(workspace);
  p.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                       attn_counter_bytes(fp4::kv_attention_max_ctas(sms)));
  p.B = B;
  p.max_blocks = max_blocks;
  p.num_blocks = cache->num_blocks;
  p.block_log2 = block_log2(cache->block_size);
  p.kv_heads = cache->kv_heads;
  p.group = group;
  p.group_magic = (65536 + group - 1) / group;
  p.q_len = q_len;
  p.row_tiles = row_tiles;
  // (a window that no sequence is longer than is none: on the device differences of it and a position fit 32 bits)
  p.window = window >= tokens ? 0 : window;
  p.unit = 1;
  p.item_cost = fp4::kAttnItemCost;
  p.uncut = cache->head_dim > 128 ? fp4::kAttnUncut256 : fp4::kAttnUncut;
  p.f16 = dtype == FP4GEMV_F16;
  p.sm_scale = sm_scale;
  if (row_units == 4 && cache->head_dim == 128 && cache->format == FP4GEMV_KV_E4M3) {
    const int64_t pages = static_cast<int64_t>(cache->num_blocks) * cache->kv_heads;
    if (!fp4::encode_pages_128(&p.k_map, cache->k_codes, cache->block_size, pages) ||
        !fp4::encode_pages_128(&p.v_map, cache->v_codes, cache->block_size, pages))
      return FP4GEMV_ERR_CUDA;
    p.unit = 8;  // tiles of 128 tokens are of whole pages
    p.item_cost = fp4::kAttnTcItemCost;
    p.skip_tile = fp4::skipped_stage();
    fp4::count_launch();
    return from_cuda(fp4::launch_kv_attention_tc(p, sms, pdl, stream));
  }
  fp4::count_launch();
  return from_cuda(fp4::launch_kv_attention(p, cache->head_dim, cache->format == FP4GEMV_KV_INT8, row_units, sms, pdl,
                                            stream));
}

fp4gemv_status fp4gemv_moe_route(const void* logits, int64_t ldl, int dtype, int M, int E, int topk, int scores,
                                 const float* bias, int n_group, int topk_group, int group_top, int renormalize,
                                 float scale, int32_t* ids, float* weights, int pdl, cudaStream_t stream) {
  if (pdl != 0 && pdl != 1) return FP4GEMV_ERR_INVALID_ARG;
  if (dtype < FP4GEMV_BF16 || dtype > FP4GEMV_F32) return FP4GEMV_ERR_INVALID_ARG;
  if (scores != FP4GEMV_ROUTE_SOFTMAX && scores != FP4GEMV_ROUTE_SIGMOID) return FP4GEMV_ERR_INVALID_ARG;
  if (renormalize != 0 && renormalize != 1) return FP4GEMV_ERR_INVALID_ARG;
  if (M < 1 || E < 1 || topk < 1 || n_group < 1 || topk_group < 1 || topk_group > n_group || ldl < E ||
      !std::isfinite(scale))
    return FP4GEMV_ERR_INVALID_ARG;
  if (group_top != 1 && group_top != 2) return FP4GEMV_ERR_INVALID_ARG;
  if (E > 512 || topk > 32 || n_group > 32 || E % n_group != 0 || topk > topk_group * (E / n_group) ||
      group_top > E / n_group)
    return FP4GEMV_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(logits, dtype == FP4GEMV_F32 ? 4 : 2) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
    return FP4GEMV_ERR_MISALIGNED;
  if (!logits || !ids || !weights) return FP4GEMV_ERR_INVALID_ARG;
  int sms = 0;
  fp4gemv_status st = fp4::current_device_state(nullptr, &sms);
  if (st != FP4GEMV_OK) return st;
  fp4::RouteParams p = {};
  p.logits = logits;
  p.ldl = ldl;
  p.bias = bias;
  p.ids = ids;
  p.weights = weights;
  p.M = M;
  p.E = E;
  p.topk = topk;
  p.n_group = n_group;
  p.topk_group = topk_group;
  p.group_top = n_group > 1 ? group_top : 1;
  p.sigmoid = scores == FP4GEMV_ROUTE_SIGMOID;
  p.renormalize = renormalize;
  p.scale = scale;
  fp4::count_launch();
  return from_cuda(fp4::launch_moe_route(p, dtype, sms, pdl, stream));
}

fp4gemv_status fp4gemv_token_logprobs(const void* logits, int64_t ldl, int dtype, int T, int V, const int32_t* tokens,
                                      float inv_temperature, int top_n, float* logprob, int32_t* rank, float* entropy,
                                      int32_t* top_ids, float* top_logprobs, int pdl, cudaStream_t stream) {
  if (pdl != 0 && pdl != 1) return FP4GEMV_ERR_INVALID_ARG;
  if (dtype < FP4GEMV_BF16 || dtype > FP4GEMV_F32) return FP4GEMV_ERR_INVALID_ARG;
  if (T < 1 || V < 1 || top_n < 0 || top_n > V || ldl < V) return FP4GEMV_ERR_INVALID_ARG;
  // (below: a masked logit, 2^100 away from the others, would come to weigh something)
  if (!(inv_temperature >= 1e-20f) || inv_temperature > 1e6f) return FP4GEMV_ERR_INVALID_ARG;
  if (top_n > FP4GEMV_MAX_TOP_N || T > (1 << 28)) return FP4GEMV_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(logits, dtype == FP4GEMV_F32 ? 4 : 2) || !aligned(tokens, 4) || !aligned(logprob, 4) ||
      !aligned(rank, 4) || !aligned(entropy, 4) || !aligned(top_ids, 4) || !aligned(top_logprobs, 4))
    return FP4GEMV_ERR_MISALIGNED;
  if (!logits || !tokens || !logprob || !rank || !entropy || (top_n > 0 && (!top_ids || !top_logprobs)))
    return FP4GEMV_ERR_INVALID_ARG;
  uint32_t* err = nullptr;
  int sms = 0;
  fp4gemv_status st = fp4::current_device_state(&err, &sms);
  if (st != FP4GEMV_OK) return st;
  fp4::LogprobParams p = {};
  p.logits = logits;
  p.ldl = ldl;
  p.tokens = tokens;
  p.logprob = logprob;
  p.rank = rank;
  p.entropy = entropy;
  p.top_ids = top_ids;
  p.top_logprobs = top_logprobs;
  p.err = err;
  p.V = V;
  p.n = top_n;
  p.inv_t = inv_temperature;
  fp4::count_launch();
  return from_cuda(fp4::launch_token_logprobs(p, dtype, T, sms, pdl, stream));
}
