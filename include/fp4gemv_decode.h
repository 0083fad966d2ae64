/*
 * fp4gemv_decode.h -- the decode step's operators around the products of
 * fp4gemv.h: a paged key/value cache held in 8 bits (append, attention),
 * routing of tokens to experts (what fp4gemv_moe_gate_up takes as ids and
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
 * largest, at 2^-32 of it), one final rounding.
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
