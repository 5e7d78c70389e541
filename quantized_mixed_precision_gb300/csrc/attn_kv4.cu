// bq_attn_kv4: causal attention of new tokens over the 4-bit cache (the kernels are in attn_kv4.cuh).
#include "attn_kv4.cuh"

namespace bq {

size_t attn_kv4_workspace(int64_t, int64_t q_heads, int64_t kv_heads, int64_t D, int64_t max_q, int64_t max_len) {
  return workspace_bytes(q_heads, kv_heads, D, max_q, max_len);
}

cudaError_t launch_attn_kv4(const AttnKv4Args& a, cudaStream_t stream) {
  return launch_rows<false>(a, nullptr, 0, stream);
}

}  // namespace bq
