// decode_api.cu -- the C ABI of the decode step's operators (see
// include/fp4gemv_decode.h).  Host side only: argument validation before any
// launch, the choice of row tiles, and the launches.
#include <cmath>
#include <cstdint>

#include "decode_launch.h"
#include "fp4gemv_decode.h"
#include "k_kv_prefix.cuh"

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

fp4gemv_status fp4gemv_kv_read(const fp4gemv_kv_cache* cache, void* k, int64_t ldk, void* v, int64_t ldv, int dtype,
                               int T, const int32_t* cu, const int32_t* block_table, int max_blocks,
                               const int32_t* seq_lens, int B, int pdl, cudaStream_t stream) {
  bool nulls, crooked;
  fp4gemv_status st = check_cache(cache, &nulls, &crooked);
  if (st != FP4GEMV_OK) return st;
  if (pdl != 0 && pdl != 1) return FP4GEMV_ERR_INVALID_ARG;
  if (dtype < FP4GEMV_BF16 || dtype > FP4GEMV_F32) return FP4GEMV_ERR_INVALID_ARG;
  const int64_t width = static_cast<int64_t>(cache->kv_heads) * cache->head_dim;
  if (T < 0 || B < 1 || max_blocks < 1 || ldk < width || ldv < width) return FP4GEMV_ERR_INVALID_ARG;
  if (!cu && T % B != 0) return FP4GEMV_ERR_INVALID_ARG;
  if (B > FP4GEMV_KV_MAX_BATCH || static_cast<int64_t>(max_blocks) * cache->block_size > (1ll << 30) || T > (1 << 30))
    return FP4GEMV_ERR_UNSUPPORTED_SHAPE;
  const int unit = dtype == FP4GEMV_F32 ? 4 : 8;  // elements of 16 bytes
  if (crooked || !aligned(k, 16) || !aligned(v, 16) || ldk % unit != 0 || ldv % unit != 0 || !aligned(cu, 4) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4))
    return FP4GEMV_ERR_MISALIGNED;
  if (nulls || !block_table || !seq_lens) return FP4GEMV_ERR_INVALID_ARG;
  if (T == 0) return FP4GEMV_OK;
  if (!k || !v) return FP4GEMV_ERR_INVALID_ARG;
  uint32_t* err = nullptr;
  int sms = 0;
  st = fp4::current_device_state(&err, &sms);
  if (st != FP4GEMV_OK) return st;
  fp4::KvReadParams p = {};
  p.codes[0] = cache->k_codes;
  p.codes[1] = cache->v_codes;
  p.scale[0] = cache->k_scale;
  p.scale[1] = cache->v_scale;
  p.dst[0] = k;
  p.dst[1] = v;
  p.ld[0] = ldk;
  p.ld[1] = ldv;
  p.cu = cu;
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
  return from_cuda(fp4::launch_kv_read(p, cache->format == FP4GEMV_KV_INT8, dtype, sms, pdl, stream));
}

fp4gemv_status fp4gemv_add_norm(const void* x, int64_t ldx, int x_dtype, const void* y, int64_t ldy, int dtype,
                                const void* weight, const void* post_weight, int weight_dtype, const void* gate,
                                int64_t ldg, int gate_dtype, int gate_kind, int gate_sigmoid, float scale, float eps,
                                float weight_offset, void* residual, int64_t ldr, void* out, int64_t ldo, int M, int H,
                                int pdl, cudaStream_t stream) {
  if (pdl != 0 && pdl != 1) return FP4GEMV_ERR_INVALID_ARG;
  if (dtype != FP4GEMV_BF16 && dtype != FP4GEMV_F16) return FP4GEMV_ERR_INVALID_ARG;
  auto kind = [&](int t) { return t == dtype || t == FP4GEMV_F32; };
  if (!kind(x_dtype) || !kind(weight_dtype) || (gate && !kind(gate_dtype))) return FP4GEMV_ERR_INVALID_ARG;
  if (gate && gate_kind != FP4GEMV_GATE_CHANNEL && gate_kind != FP4GEMV_GATE_TOKEN) return FP4GEMV_ERR_INVALID_ARG;
  if (gate_sigmoid != 0 && gate_sigmoid != 1) return FP4GEMV_ERR_INVALID_ARG;
  if (M < 1 || H < 1 || ldx < H || ldo < H || (y && (ldy < H || ldr < H))) return FP4GEMV_ERR_INVALID_ARG;
  const bool channel = gate && gate_kind == FP4GEMV_GATE_CHANNEL;
  if (gate && (channel ? ldg != 0 && ldg < H : ldg < 0)) return FP4GEMV_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !std::isfinite(weight_offset) || !std::isfinite(eps) || eps < 0.0f)
    return FP4GEMV_ERR_INVALID_ARG;
  if (!y && (post_weight || gate)) return FP4GEMV_ERR_INVALID_ARG;
  if (H > FP4GEMV_NORM_MAX_WIDTH) return FP4GEMV_ERR_UNSUPPORTED_SHAPE;
  auto size = [](int t) -> uintptr_t { return t == FP4GEMV_F32 ? 4 : 2; };
  if (!aligned(x, size(x_dtype)) || !aligned(residual, size(x_dtype)) || !aligned(y, 2) || !aligned(out, 2) ||
      !aligned(weight, size(weight_dtype)) || !aligned(post_weight, size(weight_dtype)) ||
      (gate && !aligned(gate, size(gate_dtype))))
    return FP4GEMV_ERR_MISALIGNED;
  if (!x || !weight || !out || (y && !residual)) return FP4GEMV_ERR_INVALID_ARG;
  int sms = 0;
  fp4gemv_status st = fp4::current_device_state(nullptr, &sms);
  if (st != FP4GEMV_OK) return st;
  fp4::AddNormParams p = {};
  p.x = x;
  p.y = y;
  p.weight = weight;
  p.post = post_weight;
  p.gate = gate;
  p.residual = residual;
  p.out = out;
  p.ldx = ldx;
  p.ldy = ldy;
  p.ldg = ldg;
  p.ldr = ldr;
  p.ldo = ldo;
  p.M = M;
  p.H = H;
  p.x_type = x_dtype;
  p.w_type = weight_dtype;
  p.g_type = gate_dtype;
  p.gate_scalar = gate && !channel;
  p.sigmoid = gate_sigmoid;
  p.scale = scale;
  p.eps = eps;
  p.offset = weight_offset;
  // whole chunks of 8 values on 16-byte boundaries (an f32 chunk is two of them); pairs on their own
  auto parts = [&](int n) {
    auto at = [&](const void* q, int t) { return aligned(q, std::min<uintptr_t>(n * size(t), 16)); };
    auto rows = [&](const void* q, int64_t ld, int t) { return at(q, t) && ld % n == 0; };
    return H % n == 0 && rows(x, ldx, x_dtype) && rows(out, ldo, dtype) && at(weight, weight_dtype) &&
           at(post_weight, weight_dtype) && (!y || (rows(y, ldy, dtype) && rows(residual, ldr, x_dtype))) &&
           (!channel || rows(gate, ldg, gate_dtype));
  };
  fp4::count_launch();
  return from_cuda(fp4::launch_add_norm(p, dtype == FP4GEMV_F16, parts(8) ? 8 : parts(2) ? 2 : 1, sms, pdl, stream));
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

// What the attention calls share: every check, and the kernels' parameters.
struct AttentionCall {
  const fp4gemv_kv_cache* cache;
  const void* q;
  int64_t ldq;
  int dtype, heads, q_len;
  const int32_t* block_table;
  int max_blocks;
  const int32_t* seq_lens;
  int B;
  float sm_scale;
  int window;
  void* out;
  int64_t ldo;
  float* lse;
  void* workspace;
  size_t workspace_bytes;
  int pdl;
  // of sequences that share a beginning
  bool shared;
  const int32_t* prefix_len;
  void* scratch;
  size_t scratch_bytes;
};

// Blocks of 128 rows of a KV head, items of the beginning's line of a KV head, and the pieces that they come to at most.
static int64_t shared_blocks(int64_t rows) { return (rows + 127) / 128; }
static int64_t shared_items(int64_t rows, int dim) {
  const int slots = fp4::kv_prefix_slots(dim);
  return (shared_blocks(rows) + slots - 1) / slots;
}
// [tokens taken together | (m, sum of weights) of the pieces' rows | their sums | those of the rows' own tokens | sums]
static size_t shared_ml_bytes(int64_t pieces, int dim) {
  return static_cast<size_t>(pieces) * fp4::kv_prefix_slots(dim) * 128 * 8;
}
static size_t shared_scratch_bytes(int kv_heads, int dim, int64_t rows, int sms) {
  const int64_t pieces = sms + kv_heads * shared_items(rows, dim);
  return 16 + shared_ml_bytes(pieces, dim) * (1 + dim / 2) + static_cast<size_t>(kv_heads) * ((rows + 1) / 2 * 2) * (8 + 4 * dim);
}

// Fills p, *row_units and *sms.
static fp4gemv_status attention_params(const AttentionCall& a, fp4::KvAttnParams* out_p, int* out_row_units, int* out_sms) {
  const fp4gemv_kv_cache* const cache = a.cache;
  bool nulls, crooked;
  fp4gemv_status st = check_cache(cache, &nulls, &crooked);
  if (st != FP4GEMV_OK) return st;
  if (a.pdl != 0 && a.pdl != 1) return FP4GEMV_ERR_INVALID_ARG;
  if (a.dtype != FP4GEMV_BF16 && a.dtype != FP4GEMV_F16) return FP4GEMV_ERR_INVALID_ARG;
  if (a.heads < 1 || a.q_len < 1 || a.B < 1 || a.max_blocks < 1 || a.window < 0 || !std::isfinite(a.sm_scale))
    return FP4GEMV_ERR_INVALID_ARG;
  const int64_t width = static_cast<int64_t>(a.heads) * cache->head_dim;
  if (a.ldq < width || a.ldo < width) return FP4GEMV_ERR_INVALID_ARG;
  const int group = a.heads / cache->kv_heads;
  if (a.heads % cache->kv_heads != 0 || group > FP4GEMV_KV_MAX_GROUP || a.q_len > FP4GEMV_KV_MAX_QLEN ||
      a.B > FP4GEMV_KV_MAX_BATCH)
    return FP4GEMV_ERR_UNSUPPORTED_SHAPE;
  // row tiles: the 8, 16 or 32 rows that a pass over the codes serves
  // (head_dim 256 has registers for 16).  One pass of 16 rows or two of 8, 32
  // sequences of 16384 tokens, 8 KV heads: 185 us against 350.
  const int rows = a.q_len * group;
  const int row_units = rows <= 8 ? 1 : rows <= 16 || cache->head_dim > 128 ? 2 : 4;
  const int row_tiles = (rows + 8 * row_units - 1) / (8 * row_units);
  const int64_t tokens = static_cast<int64_t>(a.max_blocks) * cache->block_size;
  // (32-bit: places on the line of strips, a quarter more with padding, and strips of the cache)
  if (tokens > (1ll << 30) || static_cast<int64_t>(cache->kv_heads) * row_tiles >= (1 << 20) ||
      (static_cast<double>(tokens) / 16 + fp4::kAttnTcItemCost + 8) * a.B * cache->kv_heads * row_tiles >= 1.2e9 ||
      static_cast<double>(cache->num_blocks) * cache->kv_heads * (cache->block_size / 16) >= 2147483647.0)
    return FP4GEMV_ERR_UNSUPPORTED_SHAPE;
  const int64_t all_rows = static_cast<int64_t>(a.B) * rows;
  if (a.shared && static_cast<double>(cache->kv_heads) * shared_blocks(all_rows) * (tokens / 64 + 1) > (1 << 30))
    return FP4GEMV_ERR_UNSUPPORTED_SHAPE;
  if (crooked || !aligned(a.q, 16) || !aligned(a.out, 16) || a.ldq % 8 != 0 || a.ldo % 8 != 0 || !aligned(a.lse, 4) ||
      !aligned(a.block_table, 4) || !aligned(a.seq_lens, 4) || !aligned(a.workspace, 16) || !aligned(a.prefix_len, 4) ||
      !aligned(a.scratch, 16))
    return FP4GEMV_ERR_MISALIGNED;
  if (nulls || !a.q || !a.out || !a.block_table || !a.seq_lens || !a.workspace) return FP4GEMV_ERR_INVALID_ARG;
  if (a.shared && (!a.prefix_len || !a.scratch)) return FP4GEMV_ERR_INVALID_ARG;
  uint32_t* err = nullptr;
  int sms = 0;
  st = fp4::current_device_state(&err, &sms);
  if (st != FP4GEMV_OK) return st;
  if (a.workspace_bytes < fp4gemv_kv_attention_workspace_bytes(cache->head_dim)) return FP4GEMV_ERR_INVALID_ARG;
  if (a.shared && a.scratch_bytes < shared_scratch_bytes(cache->kv_heads, cache->head_dim, all_rows, sms))
    return FP4GEMV_ERR_INVALID_ARG;
  fp4::KvAttnParams& p = *out_p;
  p.k_codes = cache->k_codes;
  p.v_codes = cache->v_codes;
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.q = static_cast<const uint16_t*>(a.q);
  p.ldq = a.ldq;
  p.out = static_cast<uint16_t*>(a.out);
  p.ldo = a.ldo;
  p.lse = a.lse;
  p.table = a.block_table;
  p.lens = a.seq_lens;
  p.err = err;
  p.arrived = static_cast<uint32_t*>(a.workspace);
  p.partial = reinterpret_cast<float*>(static_cast<char*>(a.workspace) +
                                       attn_counter_bytes(fp4::kv_attention_max_ctas(sms)));
  p.B = a.B;
  p.max_blocks = a.max_blocks;
  p.num_blocks = cache->num_blocks;
  p.block_log2 = block_log2(cache->block_size);
  p.kv_heads = cache->kv_heads;
  p.group = group;
  p.group_magic = (65536 + group - 1) / group;
  p.q_len = a.q_len;
  p.row_tiles = row_tiles;
  // (a window that no sequence is longer than is none: on the device differences of it and a position fit 32 bits)
  p.window = a.window >= tokens ? 0 : a.window;
  p.unit = 1;
  p.item_cost = fp4::kAttnItemCost;
  p.uncut = cache->head_dim > 128 ? fp4::kAttnUncut256 : fp4::kAttnUncut;
  p.f16 = a.dtype == FP4GEMV_F16;
  p.sm_scale = a.sm_scale;
  *out_row_units = row_units;
  *out_sms = sms;
  return FP4GEMV_OK;
}

// Whether the kernel on the 5th-generation tensor core takes the call.
static bool wide_e4m3(const fp4gemv_kv_cache* cache, int row_units) {
  return row_units == 4 && cache->head_dim == 128 && cache->format == FP4GEMV_KV_E4M3;
}

// (the checks are done)
static fp4gemv_status plain_attention(const AttentionCall& a, const fp4::KvAttnParams& base, int row_units, int sms,
                                      cudaStream_t stream) {
  const fp4gemv_kv_cache* const cache = a.cache;
  if (wide_e4m3(cache, row_units)) {
    fp4::KvAttnTcParams p = {};
    static_cast<fp4::KvAttnParams&>(p) = base;
    const int64_t pages = static_cast<int64_t>(cache->num_blocks) * cache->kv_heads;
    if (!fp4::encode_pages_128(&p.k_map, cache->k_codes, cache->block_size, pages) ||
        !fp4::encode_pages_128(&p.v_map, cache->v_codes, cache->block_size, pages))
      return FP4GEMV_ERR_CUDA;
    p.unit = 8;  // tiles of 128 tokens are of whole pages
    p.item_cost = fp4::kAttnTcItemCost;
    p.skip_tile = fp4::skipped_stage();
    fp4::count_launch();
    return from_cuda(fp4::launch_kv_attention_tc(p, sms, a.pdl, stream));
  }
  fp4::count_launch();
  return from_cuda(fp4::launch_kv_attention(base, cache->head_dim, cache->format == FP4GEMV_KV_INT8, row_units, sms,
                                            a.pdl, stream));
}

fp4gemv_status fp4gemv_kv_attention(const fp4gemv_kv_cache* cache, const void* q, int64_t ldq, int dtype, int heads,
                                    int q_len, const int32_t* block_table, int max_blocks, const int32_t* seq_lens,
                                    int B, float sm_scale, int window, void* out, int64_t ldo, float* lse,
                                    void* workspace, size_t workspace_bytes, int pdl, cudaStream_t stream) {
  const AttentionCall a = {cache, q, ldq, dtype, heads, q_len, block_table, max_blocks, seq_lens, B, sm_scale, window,
                           out, ldo, lse, workspace, workspace_bytes, pdl, false, nullptr, nullptr, 0};
  fp4::KvAttnParams p = {};
  int row_units, sms;
  const fp4gemv_status st = attention_params(a, &p, &row_units, &sms);
  return st != FP4GEMV_OK ? st : plain_attention(a, p, row_units, sms, stream);
}

fp4gemv_status fp4gemv_kv_attention_sinks(const fp4gemv_kv_cache* cache, const void* q, int64_t ldq, int dtype,
                                          int heads, int q_len, const int32_t* block_table, int max_blocks,
                                          const int32_t* seq_lens, int B, float sm_scale, int window, int sinks,
                                          void* out, int64_t ldo, float* lse, void* workspace, size_t workspace_bytes,
                                          int pdl, cudaStream_t stream) {
  if (sinks < 0) return FP4GEMV_ERR_INVALID_ARG;
  if (sinks > (1 << 30)) return FP4GEMV_ERR_UNSUPPORTED_SHAPE;
  const AttentionCall a = {cache, q, ldq, dtype, heads, q_len, block_table, max_blocks, seq_lens, B, sm_scale, window,
                           out, ldo, lse, workspace, workspace_bytes, pdl, false, nullptr, nullptr, 0};
  fp4::KvAttnSinksParams p = {};
  int row_units, sms;
  const fp4gemv_status st = attention_params(a, &p, &row_units, &sms);
  if (st != FP4GEMV_OK) return st;
  if (sinks == 0 || p.window == 0) return plain_attention(a, p, row_units, sms, stream);
  p.sinks = sinks;
  p.lead = (sinks + 15) / 16;
  if (wide_e4m3(cache, row_units)) {
    CUtensorMap k_map, v_map;
    const int64_t pages = static_cast<int64_t>(cache->num_blocks) * cache->kv_heads;
    if (!fp4::encode_pages_128(&k_map, cache->k_codes, cache->block_size, pages) ||
        !fp4::encode_pages_128(&v_map, cache->v_codes, cache->block_size, pages))
      return FP4GEMV_ERR_CUDA;
    p.unit = 8;  // tiles of 128 tokens are of whole pages
    p.item_cost = fp4::kAttnTcItemCost;
    p.lead = (p.lead + 7) / 8 * 8;
    fp4::count_launch();
    return from_cuda(fp4::launch_kv_attention_tc_sinks(p, k_map, v_map, fp4::skipped_stage(), sms, pdl, stream));
  }
  fp4::count_launch();
  return from_cuda(fp4::launch_kv_attention_sinks(p, cache->head_dim, cache->format == FP4GEMV_KV_INT8, row_units, sms,
                                                 pdl, stream));
}

size_t fp4gemv_kv_attention_shared_scratch_bytes(int kv_heads, int head_dim, int heads, int q_len, int B) {
  if (!dim_ok(head_dim) || kv_heads < 1 || kv_heads > 65535 || heads < 1 || heads % kv_heads != 0 ||
      heads / kv_heads > FP4GEMV_KV_MAX_GROUP || q_len < 1 || q_len > FP4GEMV_KV_MAX_QLEN || B < 1 ||
      B > FP4GEMV_KV_MAX_BATCH)
    return 0;
  int sms = 0;
  if (fp4::current_device_state(nullptr, &sms) != FP4GEMV_OK) return 0;
  return shared_scratch_bytes(kv_heads, head_dim, static_cast<int64_t>(B) * q_len * (heads / kv_heads), sms);
}

fp4gemv_status fp4gemv_kv_attention_shared(const fp4gemv_kv_cache* cache, const void* q, int64_t ldq, int dtype,
                                           int heads, int q_len, const int32_t* block_table, int max_blocks,
                                           const int32_t* seq_lens, int B, const int32_t* prefix_len, float sm_scale,
                                           void* out, int64_t ldo, float* lse, void* workspace,
                                           size_t workspace_bytes, void* scratch, size_t scratch_bytes, int always,
                                           int pdl, cudaStream_t stream) {
  if (always != 0 && always != 1) return FP4GEMV_ERR_INVALID_ARG;
  const AttentionCall a = {cache, q, ldq, dtype, heads, q_len, block_table, max_blocks, seq_lens, B, sm_scale, 0, out, ldo,
                           lse, workspace, workspace_bytes, pdl, true, prefix_len, scratch, scratch_bytes};
  fp4::KvAttnRestParams p = {};
  int row_units, sms;
  const fp4gemv_status st = attention_params(a, &p, &row_units, &sms);
  if (st != FP4GEMV_OK) return st;
  const int dim = cache->head_dim, int8 = cache->format == FP4GEMV_KV_INT8;
  // Where reading a common beginning again and again, out of L2, costs less than two more launches and a beginning cut over
  // all SMs.  What sharing can spare is that of all sequences but one, and reading apart goes over it (or converts it) for
  // every 16 rows.  Apart / together, us (MB by this measure): 8 rows of 128, E4M3, 16 sequences of 2112 tokens (65) 17 /
  // 26, 2 of 65375 (134) 48 / 64, 16 of 8256 (254) 46 / 31; 3 rows of 96, INT8, 7 of 37905 (87) 26 / 34; 14 rows of 96,
  // E4M3, 15 of 6033 (130) 30 / 35; 6 of 64, INT8, 38 of 2071 (157) 39 / 33; more rows: 112 of 128, INT8, 45 of 620 (98) 47 /
  // 46, 24 of 96, 5 of 11297 (278) 62 / 44, 56 of 256, E4M3, 7 of 14800 (364) 79 / 45.
  const int64_t all_rows = static_cast<int64_t>(B) * q_len * p.group, items = shared_items(all_rows, dim);
  const double spared = static_cast<double>(max_blocks) * cache->block_size * (B - 1) * cache->kv_heads * dim * 2;
  if (!always && spared * ((q_len * p.group + 15) / 16) <= FP4GEMV_KV_SHARE_FROM) {
    // Many items that cannot be long: the kernel whose warps take them by themselves (no window, no first tokens).
    // us, fp4gemv_kv_attention's kernel / this one: 50 sequences of 58 tokens, 64 rows of 256 on 8 KV heads, INT8, 86 / 25; 64
    // of 128, 8 rows of 128, E4M3, on 8 14 / 11, 16 rows on 16 32 / 16; 64 of 500, 8 rows, INT8, on 16 39 / 28.
    const int ctas = sms * (dim == 256 || row_units == 4 ? 1 : 2);
    const double items = static_cast<double>(B) * p.kv_heads * p.row_tiles;
    const double strips = (static_cast<double>(max_blocks) * cache->block_size + 15) / 16;
    if (items > ctas && !wide_e4m3(cache, row_units) &&
        fp4::attn_by_warps(static_cast<float>(items), static_cast<float>(items * strips), static_cast<float>(strips),
                           static_cast<float>(8 * ctas))) {
      fp4::KvAttnSinksParams x = {};
      static_cast<fp4::KvAttnParams&>(x) = p;
      fp4::count_launch();
      return from_cuda(fp4::launch_kv_attention_sinks(x, dim, int8, row_units, sms, pdl, stream));
    }
    return plain_attention(a, p, row_units, sms, stream);
  }
  const int64_t piece_ml = shared_ml_bytes(sms + cache->kv_heads * items, dim);
  const int64_t own_ml = static_cast<int64_t>(cache->kv_heads) * ((all_rows + 1) / 2 * 2) * 8;  // (16-byte places)
  char* at = static_cast<char*>(scratch);
  fp4::KvPrefixParams x = {};
  x.line.tokens = reinterpret_cast<int32_t*>(at);
  x.line.ml = reinterpret_cast<float2*>(at += 16);
  x.line.sums = reinterpret_cast<float*>(at += piece_ml);
  p.ml = reinterpret_cast<float2*>(at += piece_ml * (dim / 2));
  p.sums = reinterpret_cast<float*>(at += own_ml);
  p.prefix_len = prefix_len;
  x.line.slots = fp4::kv_prefix_slots(dim);
  x.line.tile = fp4::kv_prefix_tile(dim);
  x.line.blocks = static_cast<int>(shared_blocks(all_rows));
  x.line.items = static_cast<int>(items);
  // no more CTAs than tiles that the table's width could hold
  const int64_t tiles = (static_cast<int64_t>(max_blocks) << p.block_log2) / x.line.tile * cache->kv_heads * items;
  x.line.ctas = tiles < 1 ? 1 : tiles < sms ? static_cast<int>(tiles) : sms;
  x.k_codes = cache->k_codes;
  x.v_codes = cache->v_codes;
  x.k_scale = cache->k_scale;
  x.v_scale = cache->v_scale;
  x.q = p.q;
  x.ldq = ldq;
  x.table = block_table;
  x.lens = seq_lens;
  x.prefix_len = prefix_len;
  x.err = p.err;
  x.B = B;
  x.max_blocks = max_blocks;
  x.num_blocks = cache->num_blocks;
  x.block_log2 = p.block_log2;
  x.kv_heads = cache->kv_heads;
  x.group = p.group;
  x.group_magic = p.group_magic;
  x.skip_tile = fp4::skipped_stage();
  x.inv_rows = 1.0f / static_cast<float>(q_len * p.group);
  x.q_len = q_len;
  x.f16 = p.f16;
  x.sm_scale = sm_scale;
  fp4::KvJoinParams y = {};
  y.line = x.line;
  y.sums = p.sums;
  y.ml = p.ml;
  y.lens = seq_lens;
  y.out = p.out;
  y.ldo = ldo;
  y.lse = lse;
  y.B = B;
  y.kv_heads = cache->kv_heads;
  y.group = p.group;
  y.q_len = q_len;
  y.f16 = p.f16;
  // the own tokens first: the beginning's kernel, which needs whole SMs, starts where its CTAs end
  fp4::count_launch();
  cudaError_t e = fp4::launch_kv_attention_rest(p, dim, int8, row_units, sms, pdl, stream);
  if (e != cudaSuccess) return from_cuda(e);
  fp4::count_launch();
  e = fp4::launch_kv_prefix(x, dim, int8, pdl, stream);
  if (e != cudaSuccess) return from_cuda(e);
  fp4::count_launch();
  return from_cuda(fp4::launch_kv_join(y, dim, sms, pdl, stream));
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
