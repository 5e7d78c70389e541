// Internal launchers behind include/bq_decode.h.  Arguments are validated by
// decode_api.cu; every launcher enqueues work on `stream` and returns the
// CUDA error of the launch.
#pragma once

#include <cuda.h>

#include "bq_decode.h"
#include "bq_internal.h"

namespace bq {

// As make_map (gemm_common.cuh), with rows `ld` elements apart (a multiple of 16 bytes).
cudaError_t make_map_rows(CUtensorMap* map, const void* base, int elem, uint64_t row_elems, uint64_t ld, uint64_t rows,
                          uint32_t box_x, uint32_t box_rows, CUtensorMapSwizzle swz);

struct GroupGemmArgs {
  const uint16_t* x;
  int64_t ld_x;
  const uint8_t* w;
  int layout;
  int64_t M, N, K;
  int group;
  const uint16_t* scale;
  const uint16_t* zero_point;   // or null: signed codes
  int actfn;
  uint16_t* y;
};
cudaError_t launch_gemm_group(const GroupGemmArgs& g, cudaStream_t stream);

// The 4-bit cache pool: codes [page][2][heads][page_size][D / 2], params
// [page][2][heads][page_size][D / group][2].
struct Kv4Pool {
  uint8_t* codes;
  uint16_t* params;
  int64_t num_pages;
  int page_size, heads, D, group;
};

struct Kv4WriteArgs {
  const uint16_t *q, *k, *v;
  int64_t ld_q, ld_k, ld_v;
  int64_t T;
  int q_heads;
  const uint16_t *q_weight, *k_weight;
  float eps;
  const float *cos, *sin;
  int64_t max_pos;
  int rot, pairs;
  const int32_t *positions, *slots;
  Kv4Pool pool;
  uint16_t *q_out, *k_values, *v_values;
};
cudaError_t launch_kv4_write(const Kv4WriteArgs& a, cudaStream_t stream);

struct AttnKv4Args {
  const uint16_t* q;
  int64_t ld_q, T;
  int q_heads;
  Kv4Pool pool;
  const int32_t* table;
  int64_t ld_table;
  const int32_t *lens, *cu_q;
  int64_t B, max_q, max_len;
  float scale;
  int64_t window;
  uint16_t* out;
  float* lse;
  void* workspace;
};
size_t attn_kv4_workspace(int64_t B, int64_t q_heads, int64_t kv_heads, int64_t D, int64_t max_q, int64_t max_len);
cudaError_t launch_attn_kv4(const AttnKv4Args& a, cudaStream_t stream);

}  // namespace bq
