/*
 * fp4gemv_decode.h -- the decode step's operators around the products of
 * fp4gemv.h: a paged key/value cache held in 8 bits (append, attention,
 * also with first tokens that stay visible in a window or with a beginning that
 * the sequences share, and reading it back), the residual stream with its
 * norms, routing of tokens to experts (what fp4gemv_moe_gate_up takes as ids and
 * fp4gemv_moe_down_combine as tw), and the log probabilities of the answer.
 *
 * The conventions of fp4gemv.h hold: device pointers owned by the caller,
 * nothing allocated, asynchronous on `stream`, argument errors returned
 * before any launch (sizes and flags first, then alignment, then null
 * pointers), conditions that only the device can see recorded in the error
 * word of fp4gemv_get_device_error().  With pdl = 1 a launch starts early
 * and waits for the previous grid before it reads or writes anything.
 */
#ifndef FP4GEMV_DECODE_H
#define FP4GEMV_DECODE_H

#include "fp4gemv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of activations and logits. */
typedef enum { FP4GEMV_BF16 = 0, FP4GEMV_F16 = 1, FP4GEMV_F32 = 2 } fp4gemv_dtype;

/* ---- the 8-bit paged cache -------------------------------------------- */

/* Code formats.  value = code * scale, one fp32 scale for each page and KV
 * head, keys and values apart:
 *   E4M3  scale = the least power of two, not below 2^-100, with
 *         amax <= 448 * scale: joining a page moves older codes by exact
 *         powers of two;
 *   INT8  scale = max(amax * (1 / 127), 2^-100), 1 / 127 rounded to binary32;
 *         codes -127 .. 127. */
typedef enum { FP4GEMV_KV_E4M3 = 0, FP4GEMV_KV_INT8 = 1 } fp4gemv_kv_format;

/* Pages of block_size tokens: codes uint8 [num_blocks, kv_heads, block_size,
 * head_dim] (16-byte aligned), scales fp32 [num_blocks, kv_heads].
 * block_size 16, 32, 64 or 128; head_dim 64, 96, 128 or 256. */
typedef struct {
    uint8_t* k_codes;
    uint8_t* v_codes;
    float* k_scale;
    float* v_scale;
    int num_blocks;
    int kv_heads;
    int block_size;
    int head_dim;
    int format; /* fp4gemv_kv_format */
} fp4gemv_kv_cache;

/* Largest batch of the two calls below. */
#define FP4GEMV_KV_MAX_BATCH 1024
/* Largest q_len, and largest heads / kv_heads, of fp4gemv_kv_attention. */
#define FP4GEMV_KV_MAX_QLEN 16
#define FP4GEMV_KV_MAX_GROUP 64

/* Appends new tokens to B sequences.  Sequence b brings tokens cu_new[b] ..
 * cu_new[b + 1] of k, v (cu_new int32 [B + 1] device, not decreasing, from 0
 * to T), or T / B tokens each with cu_new = NULL.  They end at position
 * seq_lens[b] (int32 [B], the length with them); position p lies on page
 * block_table[b, p / block_size] (int32 [B, max_blocks]).
 * k, v bf16 or f16 [T, kv_heads, head_dim] with token strides ldk, ldv in
 * elements (multiples of 8).  For every page and head that gets tokens, K and
 * V apart: amax = the largest finite |x| of its new tokens, scale as above;
 * a page that already held tokens before the first new one keeps the larger
 * of its scale and that, and where it grew its older codes become
 * round(code * old / scale); new codes are round(x / scale), to nearest,
 * ties to even, infinities saturating, NaN to the E4M3 NaN (INT8: 0).  In
 * binary32, no operation fused.
 * A page that gets tokens must belong to one sequence of the call.  Tokens
 * at positions outside the table's row, or on a page id outside [0,
 * num_blocks), are not stored and raise FP4GEMV_ERR_BAD_INDEX.
 * Shapes: 1 <= B <= FP4GEMV_KV_MAX_BATCH, T >= 0 (with cu_new = NULL a
 *   multiple of B), max_blocks >= 1, max_blocks * block_size and T at most
 *   2^30. */
fp4gemv_status fp4gemv_kv_append(const fp4gemv_kv_cache* cache, const void* k, int64_t ldk, const void* v, int64_t ldv,
                                 int dtype, int T, const int32_t* cu_new, const int32_t* block_table, int max_blocks,
                                 const int32_t* seq_lens, int B, int pdl, cudaStream_t stream);

/* Bytes of the workspace fp4gemv_kv_attention needs on the current device
 * for any call with this cache's head_dim.  The workspace must be zero-filled
 * once before its first call and every call leaves it ready for the next;
 * calls that may run concurrently on the GPU must not share one. */
size_t fp4gemv_kv_attention_workspace_bytes(int head_dim);

/* The number of the capture that `stream` is being recorded into, 0 where it
 * is not (no two captures of a process have the same).  A workspace that is
 * zero-filled during a capture is so in that graph alone: calls captured into
 * another graph, and calls outside captures, must not use it. */
uint64_t fp4gemv_stream_capture_id(cudaStream_t stream);

/* Attention of the newest q_len tokens of every sequence over the cache:
 * query i of sequence b stands at position p = seq_lens[b] - q_len + i and
 * sees the tokens max(0, p - window + 1) .. p (window = 0: 0 .. p):
 *   out[b, i, h] = softmax_t(q[b, i, h] . k_t * sm_scale) v_t,
 *   lse[b, i, h] = log sum_t exp(q . k_t * sm_scale)      (natural log)
 * with k, v of KV head h / (heads / kv_heads).  A query that sees no token
 * (an empty sequence, or p < 0) gives zeros and lse = -inf.
 * q, out bf16 or f16 [B * q_len, heads, head_dim], token strides ldq, ldo in
 * elements (multiples of 8); lse fp32 [B * q_len, heads] or NULL.
 * Numerics: codes and queries are exact f16 operands (queries scaled by a
 * power of two for each row), sums, maxima and statistics fp32,
 * probabilities rounded to f16 for the product with V (below 2^-21 of the
 * largest, at 2^-32 of it), one final rounding.  The sum of probabilities
 * counts every token seen, those on pages whose V scale is 2^-100 (all zeros)
 * beside scales of 2^20 included.  A V scale below 2^-100, which no append
 * leaves, is taken as 2^-100.
 * With E4M3, head_dim 128 and more than 16 rows (q_len heads / kv_heads) both
 * become sums of 8-bit parts, which hold f16's probabilities exactly; entries
 * of a query below 2^-14 (f16: 2^-11) of its largest are rounded at 2^-22 of
 * that, and an infinite entry counts as NaN.
 * What a query does not see has no part in its row, whatever it holds: NaN
 * codes of later tokens or of tokens before the window, page memory past
 * seq_lens.  Lengths outside [0, max_blocks * block_size] are clamped, and
 * tokens on a page id outside [0, num_blocks) read as zeros; both raise
 * FP4GEMV_ERR_BAD_INDEX.
 * workspace: at least fp4gemv_kv_attention_workspace_bytes(head_dim) bytes,
 * 16-byte aligned.
 * Shapes: 1 <= B <= FP4GEMV_KV_MAX_BATCH, 1 <= q_len <= FP4GEMV_KV_MAX_QLEN,
 *   heads a multiple of kv_heads, at most FP4GEMV_KV_MAX_GROUP times it,
 *   window >= 0, sm_scale finite.  FP4GEMV_ERR_UNSUPPORTED_SHAPE also where
 *   max_blocks * block_size is above 2^30, or, with the passes over 8, 16 or
 *   32 rows that a KV head takes, kv_heads * passes is 2^20 or more or
 *   (max_blocks * block_size / 16 + 72) * B * kv_heads * passes 1.2e9. */
fp4gemv_status fp4gemv_kv_attention(const fp4gemv_kv_cache* cache, const void* q, int64_t ldq, int dtype, int heads,
                                    int q_len, const int32_t* block_table, int max_blocks, const int32_t* seq_lens,
                                    int B, float sm_scale, int window, void* out, int64_t ldo, float* lse,
                                    void* workspace, size_t workspace_bytes, int pdl, cudaStream_t stream);

/* fp4gemv_kv_attention with first tokens that stay visible: the query at
 * position p sees the tokens t <= p with t > p - window or t < sinks.  Pages
 * of tokens that no query of a sequence sees are not looked at.  window = 0:
 * all of 0 .. p.  sinks >= 0, at most 2^30; the rest as
 * fp4gemv_kv_attention. */
fp4gemv_status fp4gemv_kv_attention_sinks(const fp4gemv_kv_cache* cache, const void* q, int64_t ldq, int dtype,
                                          int heads, int q_len, const int32_t* block_table, int max_blocks,
                                          const int32_t* seq_lens, int B, float sm_scale, int window, int sinks,
                                          void* out, int64_t ldo, float* lse, void* workspace, size_t workspace_bytes,
                                          int pdl, cudaStream_t stream);

/* Bytes of fp4gemv_kv_attention_shared's scratch on the current device, 0 for
 * sizes that the call refuses.  It needs no initialisation and holds nothing
 * between calls; calls that may run concurrently must not share it. */
size_t fp4gemv_kv_attention_shared_scratch_bytes(int kv_heads, int head_dim, int heads, int q_len, int B);

/* fp4gemv_kv_attention (window = 0) of sequences that begin with the same
 * tokens, that beginning read and multiplied once for all of them.
 * prefix_len int32 [1], device: how many first tokens are the same.  Their
 * whole pages hold the same for every sequence of the call that is not empty
 * (usually they are the same pages); what is on them is read through the first
 * such sequence's row of block_table alone, the rest through each one's own.
 * How many tokens are taken together is prefix_len rounded down to a multiple
 * of 128, less where a sequence's first query stands before that; none is not an
 * error, nor is a negative prefix_len.  Three launches; with always = 0 only
 * where it pays, by the sizes that the host knows: up to
 * FP4GEMV_KV_SHARE_FROM bytes of codes that B - 1 sequences as long as the
 * table have, times the blocks of 16 rows to a KV head (q_len * heads /
 * kv_heads), every sequence is attended to by itself, as fp4gemv_kv_attention
 * does.
 * scratch: 16-byte aligned, fp4gemv_kv_attention_shared_scratch_bytes; the
 * workspace is fp4gemv_kv_attention's.
 * Numerics of three launches: fp4gemv_kv_attention's of up to 16 rows, whatever
 * the rows (exact f16 operands, probabilities rounded to f16, sums fp32); where
 * every sequence is attended to by itself, fp4gemv_kv_attention's for these rows,
 * which above 16 with E4M3 and head_dim 128 are sums of 8-bit parts.
 * What the host knows is the table's width: with a table much wider than the
 * lengths, or a short beginning before long own parts, three launches take
 * longer than fp4gemv_kv_attention, which is then the call to make.  us, that
 * one's / these: 16 sequences of 700, 512 common, 8 rows of 128 on 8, a table of
 * 131072 10 / 21; 32 of 16640, 256 common, E4M3, 8 rows 185 / 191, 32 rows, whose
 * own parts lack the kernel on the 5th-generation tensor core, 172 / 283.
 * Shapes as fp4gemv_kv_attention; kv_heads * (B * q_len * heads / kv_heads
 *   rows in blocks of 128) * (max_blocks * block_size / 64) at most 2^30. */
#define FP4GEMV_KV_SHARE_FROM 140000000ll
fp4gemv_status fp4gemv_kv_attention_shared(const fp4gemv_kv_cache* cache, const void* q, int64_t ldq, int dtype,
                                           int heads, int q_len, const int32_t* block_table, int max_blocks,
                                           const int32_t* seq_lens, int B, const int32_t* prefix_len, float sm_scale,
                                           void* out, int64_t ldo, float* lse, void* workspace,
                                           size_t workspace_bytes, void* scratch, size_t scratch_bytes, int always,
                                           int pdl, cudaStream_t stream);

/* The last tokens of B sequences out of the cache: rows cu[b] .. cu[b + 1] of
 * k and v (cu int32 [B + 1] device, not decreasing, within 0 .. T), or T / B
 * rows each with cu = NULL, receive the tokens that end at position
 * seq_lens[b], value = code * scale in binary32 rounded to `dtype` (bf16, f16
 * or f32).  k, v [T, kv_heads, head_dim], token strides ldk, ldv in elements
 * (multiples of 8; f32: of 4).  The other way of fp4gemv_kv_append.
 * Rows of positions below 0, outside the table's row, or on a page id outside
 * [0, num_blocks) become zeros and raise FP4GEMV_ERR_BAD_INDEX; rows that cu
 * does not name stay as they were.
 * Shapes as fp4gemv_kv_append. */
fp4gemv_status fp4gemv_kv_read(const fp4gemv_kv_cache* cache, void* k, int64_t ldk, void* v, int64_t ldv, int dtype,
                               int T, const int32_t* cu, const int32_t* block_table, int max_blocks,
                               const int32_t* seq_lens, int B, int pdl, cudaStream_t stream);

/* ---- the residual stream and its norms ---------------------------------- */

/* Largest H. */
#define FP4GEMV_NORM_MAX_WIDTH 32768

typedef enum { FP4GEMV_GATE_CHANNEL = 0, FP4GEMV_GATE_TOKEN = 1 } fp4gemv_gate_kind;

/* Per token t, in binary32 (sums of squares as well):
 *   u = y[t], or with post_weight y[t] / sqrt(mean(y[t]^2) + eps) *
 *       (weight_offset + post_weight)
 *   r = x[t] + scale * g * u     g: 1 with gate = NULL, else the gate, or
 *       1 / (1 + exp(-gate)) with gate_sigmoid
 *   residual[t] = r
 *   out[t] = r / sqrt(mean(r^2) + eps) * (weight_offset + weight)
 * each rounded once (out from r before its rounding).  y = NULL: out is the
 * norm of x; post_weight and gate have to be NULL, and residual is not used.
 * x, residual [M, H] of x_dtype (dtype or f32); y, out [M, H] of dtype (bf16
 * or f16); weight, post_weight [H] of weight_dtype, gate of gate_dtype (dtype
 * or f32).  gate_kind CHANNEL: gate [M, H] with row stride ldg, 0 for one row
 * that all tokens take; TOKEN: gate[t * ldg] for all of a token's values.
 * Row strides in elements, at least H; nothing needs more alignment than its
 * element's, and 16-byte aligned rows of H a multiple of 8 are faster.
 * residual may be x, and out may be y, with the same stride.  One launch.
 * Shapes: M >= 1, 1 <= H <= FP4GEMV_NORM_MAX_WIDTH; scale, weight_offset
 *   finite, eps finite and not negative. */
fp4gemv_status fp4gemv_add_norm(const void* x, int64_t ldx, int x_dtype, const void* y, int64_t ldy, int dtype,
                                const void* weight, const void* post_weight, int weight_dtype, const void* gate,
                                int64_t ldg, int gate_dtype, int gate_kind, int gate_sigmoid, float scale, float eps,
                                float weight_offset, void* residual, int64_t ldr, void* out, int64_t ldo, int M, int H,
                                int pdl, cudaStream_t stream);

/* ---- routing to experts ------------------------------------------------ */

typedef enum { FP4GEMV_ROUTE_SOFTMAX = 0, FP4GEMV_ROUTE_SIGMOID = 1 } fp4gemv_route_scores;

/* Per token t, logits x = logits[t, 0 .. E) (bf16, f16 or f32, row stride ldl
 * in elements):
 *   score[e] = softmax(x)[e] or 1 / (1 + exp(-x[e]))
 *   key[e]   = score[e] + bias[e]; with bias = NULL and group_top = 1 the
 *              logits themselves (the scores are monotone in them)
 * With n_group > 1 the experts form n_group consecutive groups; a group's
 * strength is the sum of its group_top (1 or 2) largest keys, and only the
 * topk_group strongest groups take part.  ids[t] = the topk largest keys in
 * descending order (every tie to the lower index),
 *   weights[t, j] = score[ids[t, j]] * scale, the scores divided by their
 *   sum over j before that with renormalize (a zero sum gives zeros).
 * ids int32 [M, topk] and weights fp32 [M, topk] are what
 * fp4gemv_moe_gate_up and fp4gemv_moe_down_combine take.
 * A NaN logit counts as -inf; -inf scores 0 (a row of nothing else: ids of
 * the best keys, weights 0); keys that are NaN count as -inf.  Scores are
 * binary32; the softmax's sum is carried in 48 bits, so keys do not depend
 * on its order.  One launch.
 * Shapes: 1 <= E <= 512, 1 <= topk <= 32, topk <= topk_group * E / n_group,
 *   n_group <= 32 dividing E, 1 <= topk_group <= n_group, group_top <= the
 *   group's size, M >= 1, scale finite. */
fp4gemv_status fp4gemv_moe_route(const void* logits, int64_t ldl, int dtype, int M, int E, int topk, int scores,
                                 const float* bias, int n_group, int topk_group, int group_top, int renormalize,
                                 float scale, int32_t* ids, float* weights, int pdl, cudaStream_t stream);

/* ---- log probabilities -------------------------------------------------- */

/* Largest top_n. */
#define FP4GEMV_MAX_TOP_N 32

/* Per row t, x = logits[t, 0 .. V) (bf16, f16 or f32, row stride ldl in
 * elements, no alignment needed beyond the element's), lp = log softmax(x *
 * inv_temperature):
 *   logprob[t] = lp[tokens[t]]
 *   rank[t]    = 1 + the number of logits above that of tokens[t]
 *   entropy[t] = -sum_i exp(lp[i]) lp[i]
 *   top_ids[t, j], top_logprobs[t, j]: the top_n largest logits in
 *   descending order (ties to the lower id)
 * tokens int32 [T]; logprob, entropy fp32 [T]; rank int32 [T]; top_* [T,
 * top_n] (may be NULL with top_n = 0).  A token id outside [0, V) raises
 * FP4GEMV_ERR_BAD_INDEX and leaves that row's logprob and rank unwritten.
 * Logits at or below -2^100 (-inf, bf16's and fp32's lowest value; f16's,
 * -65504, is a logit like others) are masked: their
 * probability is 0 and their log probability -inf; a row of nothing else has
 * entropy 0.  +inf or NaN logits make the row's logprobs and entropy NaN; NaN
 * is ordered like -inf.
 * The logits are read once, and again near the top_n largest.  One launch.
 * Shapes: T >= 1, V >= 1, 0 <= top_n <= min(V, FP4GEMV_MAX_TOP_N),
 *   1e-20 <= inv_temperature <= 1e6. */
fp4gemv_status fp4gemv_token_logprobs(const void* logits, int64_t ldl, int dtype, int T, int V, const int32_t* tokens,
                                      float inv_temperature, int top_n, float* logprob, int32_t* rank, float* entropy,
                                      int32_t* top_ids, float* top_logprobs, int pdl, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP4GEMV_DECODE_H */
