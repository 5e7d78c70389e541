// C ABI of the decoder-layer operators (declared in include/bq_decode.h):
// host-side validation only.  Nothing here allocates device memory.
#include <cstdint>

#include "decode_internal.h"

namespace {

using namespace bq;

constexpr int64_t MAX_ROWS = 1LL << 24;
constexpr int64_t MAX_HEADS = 65536;
constexpr int64_t MAX_KV_HEADS = 4096;   // a page's bytes stay below 2**32
constexpr int64_t MAX_LEN = 1LL << 30;   // keys of a sequence
constexpr int64_t MAX_QUERY_ROWS = 1LL << 31;   // tokens times heads, counted in 32 bits

inline bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned(p, 16); }
inline bq_status from_cuda(cudaError_t e) { return e == cudaSuccess ? BQ_OK : BQ_ERR_CUDA; }

bool valid_pool(int64_t D, int64_t group, int64_t page_size, int64_t num_pages) {
  if (D != 64 && D != 128 && D != 256) return false;
  if (group != 32 && group != 64 && group != 128) return false;
  if (group > D || D / group > 4) return false;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128 && page_size != 256) return false;
  return num_pages * page_size < (1LL << 31);
}

}  // namespace

using namespace bq;

extern "C" {

bq_status bq_gemm_f16xi4_group(const uint16_t* X, int64_t ld_x, const uint8_t* Wp, int layout, int64_t M, int64_t N,
                               int64_t K, int group, const uint16_t* scale, const uint16_t* zero_point,
                               int activation, uint16_t* Y, void* stream) {
  if (M < 0 || N < 0 || K < 0 || ld_x < K) return BQ_ERR_INVALID_ARG;
  if (layout != BQ_LAYOUT_PLAIN && layout != BQ_LAYOUT_INTERLEAVED) return BQ_ERR_INVALID_ARG;
  if (activation != BQ_ACT_NONE && activation != BQ_ACT_RELU && activation != BQ_ACT_GELU) return BQ_ERR_INVALID_ARG;
  if (group != 32 && group != 64 && group != 128) return BQ_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return BQ_OK;
  if (!Y || (K > 0 && (!X || !Wp || !scale))) return BQ_ERR_INVALID_ARG;
  if (K % group != 0 || K > 65536 || M > MAX_ROWS || N > MAX_ROWS) return BQ_ERR_UNSUPPORTED;
  if (!aligned16(Y)) return BQ_ERR_ALIGNMENT;
  if (K > 0 && (!aligned16(X) || !aligned16(Wp) || !aligned16(scale))) return BQ_ERR_ALIGNMENT;
  if ((zero_point && !aligned16(zero_point)) || (K > 0 && M > 1 && ld_x % 8 != 0)) return BQ_ERR_ALIGNMENT;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (K == 0) return from_cuda(cudaMemsetAsync(Y, 0, (size_t)M * (size_t)N * 2, s));
  return from_cuda(launch_gemm_group(
      GroupGemmArgs{X, ld_x, Wp, layout, M, N, K, group, scale, zero_point, activation, Y}, s));
}

bq_status bq_qk_norm_rope_kv4(const uint16_t* q, int64_t ld_q, const uint16_t* k, int64_t ld_k, const uint16_t* v,
                              int64_t ld_v, int64_t T, int64_t q_heads, int64_t kv_heads, int64_t D,
                              const uint16_t* q_weight, const uint16_t* k_weight, float eps, const float* cos,
                              const float* sin, int64_t max_pos, int64_t rot, int pairs, const int32_t* positions,
                              const int32_t* slots, uint8_t* codes, uint16_t* params, int64_t num_pages,
                              int64_t page_size, int64_t group, uint16_t* q_out, uint16_t* k_values,
                              uint16_t* v_values, void* stream) {
  if (T < 0 || q_heads < 0 || kv_heads < 1 || D < 1 || num_pages < 0 || max_pos < 0 || rot < 0)
    return BQ_ERR_INVALID_ARG;
  if (rot > D || (pairs != 0 && pairs != 1) || !(eps >= 0.0f)) return BQ_ERR_INVALID_ARG;
  if (T == 0) return BQ_OK;
  if (!k || !v || !slots || !codes || !params || (q_heads > 0 && (!q || !q_out))) return BQ_ERR_INVALID_ARG;
  if (rot > 0 ? (!cos || !sin || !positions) : (cos || sin)) return BQ_ERR_INVALID_ARG;
  if (q_heads > MAX_HEADS || kv_heads > MAX_KV_HEADS || T > MAX_ROWS || rot % 16 != 0) return BQ_ERR_UNSUPPORTED;
  if (!valid_pool(D, group, page_size, num_pages)) return BQ_ERR_UNSUPPORTED;
  if (ld_k < kv_heads * D || ld_v < kv_heads * D || (q_heads > 0 && ld_q < q_heads * D)) return BQ_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || ld_k % 8 != 0 || ld_v % 8 != 0) return BQ_ERR_ALIGNMENT;
  if (q_heads > 0 && (!aligned16(q) || !aligned16(q_out) || ld_q % 8 != 0)) return BQ_ERR_ALIGNMENT;
  if ((q_weight && !aligned16(q_weight)) || (k_weight && !aligned16(k_weight))) return BQ_ERR_ALIGNMENT;
  if ((cos && !aligned16(cos)) || (sin && !aligned16(sin))) return BQ_ERR_ALIGNMENT;
  if (!aligned16(codes) || !aligned16(params) || (k_values && !aligned16(k_values)) ||
      (v_values && !aligned16(v_values)))
    return BQ_ERR_ALIGNMENT;
  if (!aligned(slots, 4) || (positions && !aligned(positions, 4))) return BQ_ERR_ALIGNMENT;
  Kv4WriteArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.ld_q = ld_q;
  a.ld_k = ld_k;
  a.ld_v = ld_v;
  a.T = T;
  a.q_heads = (int)q_heads;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.eps = eps;
  a.cos = cos;
  a.sin = sin;
  a.max_pos = max_pos;
  a.rot = (int)rot;
  a.pairs = pairs;
  a.positions = positions;
  a.slots = slots;
  a.pool = Kv4Pool{codes, params, num_pages, (int)page_size, (int)kv_heads, (int)D, (int)group};
  a.q_out = q_out;
  a.k_values = k_values;
  a.v_values = v_values;
  return from_cuda(launch_kv4_write(a, static_cast<cudaStream_t>(stream)));
}

size_t bq_attn_kv4_workspace(int64_t B, int64_t q_heads, int64_t kv_heads, int64_t D, int64_t max_q,
                             int64_t max_len) {
  if (B < 1 || kv_heads < 1 || q_heads < 1 || D < 1 || max_q < 1 || max_len < 0 || q_heads % kv_heads != 0) return 0;
  if (B > MAX_ROWS || q_heads > MAX_HEADS || D > 256 || max_q > MAX_ROWS || max_len > MAX_LEN) return 0;
  return attn_kv4_workspace(B, q_heads, kv_heads, D, max_q, max_len);
}

bq_status bq_attn_kv4(const uint16_t* q, int64_t ld_q, int64_t T, int64_t q_heads, int64_t kv_heads, int64_t D,
                      const uint8_t* codes, const uint16_t* params, int64_t num_pages, int64_t page_size,
                      int64_t group, const int32_t* block_table, int64_t ld_table, const int32_t* seq_lens,
                      const int32_t* cu_q, int64_t B, int64_t max_q, int64_t max_len, float scale, int64_t window,
                      uint16_t* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (T < 0 || B < 0 || q_heads < 1 || kv_heads < 1 || D < 1 || num_pages < 0 || ld_table < 0 || max_len < 0 ||
      window < 0 || max_q < 0)
    return BQ_ERR_INVALID_ARG;
  if (q_heads % kv_heads != 0 || !(scale == scale)) return BQ_ERR_INVALID_ARG;
  if (T == 0 || B == 0) return BQ_OK;
  if (max_q < 1 || (!cu_q && T != B)) return BQ_ERR_INVALID_ARG;
  if (!q || !out || !seq_lens || (max_len > 0 && (!codes || !params || !block_table || num_pages < 1)))
    return BQ_ERR_INVALID_ARG;
  if (q_heads > MAX_HEADS || kv_heads > MAX_KV_HEADS || T > MAX_ROWS || B > MAX_ROWS || max_q > MAX_ROWS ||
      max_len > MAX_LEN || T * q_heads >= MAX_QUERY_ROWS)
    return BQ_ERR_UNSUPPORTED;
  if (!valid_pool(D, group, page_size, num_pages)) return BQ_ERR_UNSUPPORTED;
  if (ld_q < q_heads * D || max_len > ld_table * page_size) return BQ_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || ld_q % 8 != 0 || !aligned16(codes) || !aligned16(params))
    return BQ_ERR_ALIGNMENT;
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(cu_q, 4) || !aligned(lse, 4) ||
      !aligned16(workspace))
    return BQ_ERR_ALIGNMENT;
  // No sequence has more than T query tokens, and one each without cu_q, whatever the bound says: the grids, the records
  // of the parts and the workspace follow what there can be (never more workspace than a larger max_q asks for).
  max_q = cu_q ? (max_q < T ? max_q : T) : 1;
  const size_t need = attn_kv4_workspace(B, q_heads, kv_heads, D, max_q, max_len);
  if (need > 0 && (!workspace || workspace_bytes < need)) return BQ_ERR_INVALID_ARG;
  AttnKv4Args a{};
  a.q = q;
  a.ld_q = ld_q;
  a.T = T;
  a.q_heads = (int)q_heads;
  a.pool = Kv4Pool{const_cast<uint8_t*>(codes), const_cast<uint16_t*>(params), num_pages, (int)page_size,
                   (int)kv_heads, (int)D, (int)group};
  a.table = block_table;
  a.ld_table = ld_table;
  a.lens = seq_lens;
  a.cu_q = cu_q;
  a.B = B;
  a.max_q = max_q;
  a.max_len = max_len;
  a.scale = scale;
  a.window = window;
  a.out = out;
  a.lse = lse;
  a.workspace = workspace;
  return from_cuda(launch_attn_kv4(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
