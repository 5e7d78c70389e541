// bq_attn_kv4_tree with few query rows (the kernels are in attn_kv4.cuh).
#include "attn_kv4.cuh"

namespace bq {

size_t attn_tree_rows_workspace(int64_t q_heads, int64_t kv_heads, int64_t D, int64_t max_q, int64_t max_len) {
  return workspace_bytes(q_heads, kv_heads, D, max_q, max_len);
}

cudaError_t launch_attn_tree_rows(const AttnKv4Args& a, const uint64_t* tree, int words, cudaStream_t stream) {
  return launch_rows<true>(a, tree, words, stream);
}

}  // namespace bq
