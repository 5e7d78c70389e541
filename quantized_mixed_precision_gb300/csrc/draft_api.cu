// C ABI of the operators on drafted tokens (declared in include/bq_draft.h):
// host-side validation only.  Nothing here allocates device memory.
#include <cstdint>

#include "draft_internal.h"

namespace {

using namespace bq;

constexpr int64_t MAX_ROWS = 1LL << 24;
constexpr int64_t MAX_HEADS = 65536;
constexpr int64_t MAX_KV_HEADS = 4096;   // a page's bytes stay below 2**32
constexpr int64_t MAX_LAYERS = 65536;
constexpr int64_t MAX_LEN = 1LL << 30;   // keys of a sequence
constexpr int64_t MAX_QUERY_ROWS = 1LL << 31;   // tokens times heads, counted in 32 bits
constexpr int64_t MAX_WORDS = 16;        // 1024 nodes
constexpr int64_t MAX_VOCAB = 1LL << 19; // sums of 2**44 units a token stay below 2**64

inline bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned(p, 16); }
inline bq_status from_cuda(cudaError_t e) { return e == cudaSuccess ? BQ_OK : BQ_ERR_CUDA; }

bool valid_pool(int64_t D, int64_t group, int64_t page_size, int64_t num_pages) {
  if (D != 64 && D != 128 && D != 256) return false;
  if (group != 32 && group != 64 && group != 128) return false;
  if (group > D || D / group > 4) return false;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128 && page_size != 256) return false;
  return num_pages < (1LL << 31) && num_pages * page_size < (1LL << 31);
}

}  // namespace

using namespace bq;

extern "C" {

size_t bq_attn_kv4_tree_workspace(int64_t B, int64_t q_heads, int64_t kv_heads, int64_t D, int64_t max_q,
                                  int64_t max_len) {
  if (B < 1 || kv_heads < 1 || q_heads < 1 || D < 1 || max_q < 1 || max_len < 0 || q_heads % kv_heads != 0) return 0;
  if (B > MAX_ROWS || q_heads > MAX_HEADS || D > 256 || max_q > 64 * MAX_WORDS || max_len > MAX_LEN) return 0;
  // (the call takes the smaller of max_q and T: enough for either form)
  const size_t rows = attn_tree_rows_workspace(q_heads, kv_heads, D, max_q, max_len);
  const size_t tc = attn_tree_tc_applies(B, q_heads, kv_heads, D, max_q, max_len)
                        ? attn_tree_tc_workspace(q_heads, kv_heads, D, max_q) : 0;
  return rows > tc ? rows : tc;
}

bq_status bq_attn_kv4_tree(const uint16_t* q, int64_t ld_q, int64_t T, int64_t q_heads, int64_t kv_heads, int64_t D,
                           const uint8_t* codes, const uint16_t* params, int64_t num_pages, int64_t page_size,
                           int64_t group, const int32_t* block_table, int64_t ld_table, const int32_t* seq_lens,
                           const uint64_t* tree, int64_t words, const int32_t* cu_q, int64_t B, int64_t max_q,
                           int64_t max_len, float scale, int64_t window, uint16_t* out, float* lse, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (T < 0 || B < 0 || q_heads < 1 || kv_heads < 1 || D < 1 || num_pages < 0 || ld_table < 0 || max_len < 0 ||
      window < 0 || max_q < 0 || words < 1)
    return BQ_ERR_INVALID_ARG;
  if (q_heads % kv_heads != 0 || !(scale == scale)) return BQ_ERR_INVALID_ARG;
  if (T == 0 || B == 0) return BQ_OK;
  if (max_q < 1 || (!cu_q && T % B != 0)) return BQ_ERR_INVALID_ARG;
  if (!q || !out || !seq_lens || !tree || (max_len > 0 && (!codes || !params || !block_table || num_pages < 1)))
    return BQ_ERR_INVALID_ARG;
  if (q_heads > MAX_HEADS || kv_heads > MAX_KV_HEADS || T > MAX_ROWS || B > MAX_ROWS || max_len > MAX_LEN ||
      T * q_heads >= MAX_QUERY_ROWS || words > MAX_WORDS)
    return BQ_ERR_UNSUPPORTED;
  if (!valid_pool(D, group, page_size, num_pages)) return BQ_ERR_UNSUPPORTED;
  if (ld_q < q_heads * D || ld_table > MAX_QUERY_ROWS || max_len > ld_table * page_size) return BQ_ERR_INVALID_ARG;
  // no sequence has more nodes than there are rows, and all the same number without cu_q
  if (!cu_q && T / B > max_q) return BQ_ERR_INVALID_ARG;
  max_q = cu_q ? (max_q < T ? max_q : T) : T / B;
  if (max_q > 64 * words) return BQ_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || ld_q % 8 != 0 || !aligned16(codes) || !aligned16(params))
    return BQ_ERR_ALIGNMENT;
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(cu_q, 4) || !aligned(lse, 4) ||
      !aligned(tree, 8) || !aligned16(workspace))
    return BQ_ERR_ALIGNMENT;
  const size_t need = bq_attn_kv4_tree_workspace(B, q_heads, kv_heads, D, max_q, max_len);
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
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (attn_tree_tc_applies(B, q_heads, kv_heads, D, max_q, max_len))
    return from_cuda(launch_attn_tree_tc(a, tree, (int)words, s));
  return from_cuda(launch_attn_tree_rows(a, tree, (int)words, s));
}

bq_status bq_sample(const void* logits, int ltype, int64_t R, int64_t V, int64_t ld, const float* u,
                    const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                    int32_t* tokens, float* logprob, void* stream) {
  if (R < 0 || V < 0 || ld < V || (ltype != BQ_LOGITS_F16 && ltype != BQ_LOGITS_F32 && ltype != BQ_LOGITS_BF16))
    return BQ_ERR_INVALID_ARG;
  if (R == 0) return BQ_OK;
  if (!u || !tokens || (V > 0 && !logits)) return BQ_ERR_INVALID_ARG;
  if (V > MAX_VOCAB || R > MAX_ROWS) return BQ_ERR_UNSUPPORTED;
  if (!aligned(logits, ltype == BQ_LOGITS_F32 ? 4 : 2) || !aligned(u, 4) || !aligned(temperature, 4) ||
      !aligned(top_k, 4) || !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(tokens, 4) || !aligned(logprob, 4))
    return BQ_ERR_ALIGNMENT;
  return from_cuda(launch_sample(SampleArgs{logits, ltype, R, V, ld, u, temperature, top_k, top_p, min_p, tokens, logprob},
                                 static_cast<cudaStream_t>(stream)));
}

bq_status bq_kv4_accept(const int32_t* tokens, const int32_t* targets, const uint64_t* tree, int64_t words, int64_t T,
                        const int32_t* cu_q, int64_t B, int64_t max_q, const int32_t* block_table, int64_t ld_table,
                        const int32_t* seq_lens, int64_t max_len, uint8_t* codes, uint16_t* params, int64_t layers,
                        int64_t num_pages, int64_t kv_heads, int64_t page_size, int64_t D, int64_t group,
                        int32_t* path, int32_t* accepted, int32_t* next, int32_t* new_lens, void* stream) {
  if (T < 0 || B < 0 || words < 1 || max_q < 0 || ld_table < 0 || max_len < 0 || layers < 0 || num_pages < 0 ||
      kv_heads < 1 || D < 1)
    return BQ_ERR_INVALID_ARG;
  if (B == 0) return BQ_OK;
  if (!cu_q && (T % B != 0 || T / B > max_q)) return BQ_ERR_INVALID_ARG;
  if (!seq_lens || !accepted || !next || !new_lens || (max_q > 0 && !path) || new_lens == seq_lens ||
      accepted == seq_lens || next == seq_lens)
    return BQ_ERR_INVALID_ARG;
  if (T > 0 && (!tokens || !targets || !tree)) return BQ_ERR_INVALID_ARG;
  if (max_len > 0 && !block_table) return BQ_ERR_INVALID_ARG;
  if (layers > 0 && num_pages > 0 && (!codes || !params)) return BQ_ERR_INVALID_ARG;
  if (words > MAX_WORDS || layers > MAX_LAYERS || kv_heads > MAX_KV_HEADS || T > MAX_ROWS || B > MAX_ROWS ||
      max_len > MAX_LEN)
    return BQ_ERR_UNSUPPORTED;
  if (!valid_pool(D, group, page_size, num_pages)) return BQ_ERR_UNSUPPORTED;
  if (ld_table > MAX_QUERY_ROWS || max_len > ld_table * page_size || max_q > 64 * words) return BQ_ERR_INVALID_ARG;
  if (!aligned(tokens, 4) || !aligned(targets, 4) || !aligned(tree, 8) || !aligned(cu_q, 4) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned16(codes) || !aligned16(params) ||
      !aligned(path, 4) || !aligned(accepted, 4) || !aligned(next, 4) || !aligned(new_lens, 4))
    return BQ_ERR_ALIGNMENT;
  AcceptArgs a{};
  a.tokens = tokens;
  a.targets = targets;
  a.tree = tree;
  a.words = (int)words;
  a.T = T;
  a.cu_q = cu_q;
  a.B = B;
  a.each = cu_q ? 0 : T / B;
  a.max_q = max_q;
  a.table = block_table;
  a.ld_table = ld_table;
  a.lens = seq_lens;
  a.max_len = max_len;
  a.pool = Kv4Pool{codes, params, num_pages, (int)page_size, (int)kv_heads, (int)D, (int)group};
  a.layers = layers;
  a.path = path;
  a.accepted = accepted;
  a.next = next;
  a.new_lens = new_lens;
  return from_cuda(launch_kv4_accept(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
