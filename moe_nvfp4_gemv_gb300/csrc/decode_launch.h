// decode_launch.h -- host-side interface between the C API of the decode
// step's operators (decode_api.cu) and their kernel translation units, and
// what those share with fp4gemv_api.cu.
#pragma once

#include "fp4gemv.h"
#include "k_add_norm.cuh"
#include "k_kv_append.cuh"
#include "k_kv_attention.cuh"
#include "k_kv_read.cuh"
#include "k_logprobs.cuh"

namespace fp4 {

// fp4gemv_api.cu: the current device's error word and SM count, and the
// launch counter.
fp4gemv_status current_device_state(uint32_t** err, int* sms);
void count_launch();
// The test hook's stage (fp4gemv_debug_skip_stage), -1: none.
int skipped_stage();
// A tensor map of [pages][block_size][128] bytes in boxes of a page.
bool encode_pages_128(CUtensorMap* m, const void* base, int block_size, int64_t pages);

cudaError_t launch_moe_route(const RouteParams& p, int dtype, int sms, int pdl, cudaStream_t stream);
cudaError_t launch_token_logprobs(const LogprobParams& p, int dtype, int T, int sms, int pdl, cudaStream_t stream);
cudaError_t launch_kv_append(const KvAppendParams& p, int int8, int f16, int pdl, cudaStream_t stream);
cudaError_t launch_kv_read(const KvReadParams& p, int int8, int dtype, int sms, int pdl, cudaStream_t stream);
// part: values that all rows hold side by side on boundaries of their size, 8 (16 bytes), 2 or 1.
cudaError_t launch_add_norm(const AddNormParams& p, int f16, int part, int sms, int pdl, cudaStream_t stream);
// CTAs of the attention kernel at most (the workspace is sized for them).
int kv_attention_max_ctas(int sms);
// row_units: row tiles of 8, 16 or 32 rows: 1, 2 or 4 (4 not with head_dim 256).
cudaError_t launch_kv_attention(const KvAttnParams& p, int dim, int int8, int row_units, int sms, int pdl,
                                cudaStream_t stream);

// ... with first tokens that stay visible, and behind a beginning that is taken; row tiles of 32 for every head_dim but
// 256.
cudaError_t launch_kv_attention_sinks(const KvAttnSinksParams& p, int dim, int int8, int row_units, int sms, int pdl,
                                      cudaStream_t stream);
cudaError_t launch_kv_attention_rest(const KvAttnRestParams& p, int dim, int int8, int row_units, int sms, int pdl,
                                     cudaStream_t stream);

// The common beginning of shared attention (k_kv_prefix.cuh).  The line's slots and tile by head_dim; its ctas and the
// scratch's pieces by the SMs.
struct KvPrefixParams;
int kv_prefix_slots(int dim);
int kv_prefix_tile(int dim);
cudaError_t launch_kv_prefix(const KvPrefixParams& p, int dim, int int8, int pdl, cudaStream_t stream);
struct KvJoinParams;
cudaError_t launch_kv_join(const KvJoinParams& p, int dim, int sms, int pdl, cudaStream_t stream);

// E4M3, head_dim 128, row tiles of 32.
cudaError_t launch_kv_attention_tc(const KvAttnTcParams& p, int sms, int pdl, cudaStream_t stream);
cudaError_t launch_kv_attention_tc_sinks(const KvAttnSinksParams& p, const CUtensorMap& k_map, const CUtensorMap& v_map,
                                         int skip_tile, int sms, int pdl, cudaStream_t stream);

}  // namespace fp4
