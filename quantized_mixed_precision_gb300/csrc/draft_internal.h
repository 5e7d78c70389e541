// Internal launchers behind include/bq_draft.h.  Arguments are validated by
// draft_api.cu; every launcher enqueues work on `stream` and returns the CUDA
// error of the launch.
#pragma once

#include "bq_draft.h"
#include "decode_internal.h"

namespace bq {

// Few query rows a kv head: the kernels of bq_attn_kv4.
size_t attn_tree_rows_workspace(int64_t q_heads, int64_t kv_heads, int64_t D, int64_t max_q, int64_t max_len);
cudaError_t launch_attn_tree_rows(const AttnKv4Args& a, const uint64_t* tree, int words, cudaStream_t stream);

// Many of them, on tcgen05: whether that is the better fit (a rule of sizes alone).
bool attn_tree_tc_applies(int64_t B, int64_t q_heads, int64_t kv_heads, int64_t D, int64_t max_q, int64_t max_len);
size_t attn_tree_tc_workspace(int64_t q_heads, int64_t kv_heads, int64_t D, int64_t max_q);
cudaError_t launch_attn_tree_tc(const AttnKv4Args& a, const uint64_t* tree, int words, cudaStream_t stream);

struct SampleArgs {
  const void* logits;
  int ltype;
  int64_t R, V, ld;
  const float *u, *temperature;
  const int32_t* top_k;
  const float *top_p, *min_p;
  int32_t* tokens;
  float* logprob;
};
cudaError_t launch_sample(const SampleArgs& a, cudaStream_t stream);

struct AcceptArgs {
  const int32_t *tokens, *targets;
  const uint64_t* tree;
  int words;
  int64_t T;
  const int32_t* cu_q;
  int64_t B, each, max_q;       // each: nodes of a sequence where cu_q is null
  const int32_t* table;
  int64_t ld_table;
  const int32_t* lens;
  int64_t max_len;
  Kv4Pool pool;                 // of the first layer
  int64_t layers;
  int32_t *path, *accepted, *next, *new_lens;
};
cudaError_t launch_kv4_accept(const AcceptArgs& a, cudaStream_t stream);

}  // namespace bq
