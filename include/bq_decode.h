/*
 * bq_decode.h -- C ABI of the decoder-layer operators of libbq.so: 4-bit
 * weights with group scales, and attention over a cache held in 4 bits.
 *
 * The conventions are those of bq.h: device pointers owned by the caller,
 * asynchronous launches on the caller's stream, no allocation, fp16 as
 * uint16_t bit patterns, host validation before any launch, a bq_status.
 * Pointers must be 16-byte aligned unless a call says otherwise.
 *
 * The 4-bit cache.  Keys and values of every token live in pages:
 *   codes   uint8 [num_pages][2][kv_heads][page_size][D / 2]
 *   params  fp16  [num_pages][2][kv_heads][page_size][D / group][2]
 * with index 0 of the second axis the keys and 1 the values.  Byte j of a
 * code row holds dims 2 j (low four bits) and 2 j + 1; a group of `group`
 * consecutive dims has params (step, low) and stands for the values
 *   x[d] = low + step * code[d],   code in [0, 15].
 * Token `slot` of the pool is row slot % page_size of page slot / page_size.
 * Supported: D 64, 128 or 256; group 32, 64 or 128 with group <= D and
 * D / group <= 4; page_size 16, 32, 64, 128 or 256; at most 4096 kv_heads;
 * num_pages * page_size below 2**31.  Byte offsets into the pool are 64 bits wide.
 */
#ifndef BQ_DECODE_H_
#define BQ_DECODE_H_

#include "bq.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * bq_gemm_f16xi4_group -- fp16 activations times 4-bit weights with a scale
 * (and optionally a zero point) for each group of `group` consecutive k.
 *
 *   w[j, k] = scale[j, k / group] * (c[j, k] - zero_point[j, k / group])
 *   Y[i, j] = fp16_rne( act( sum_k X[i, k] * w[j, k] ) )
 *   zero_point NULL: c are the signed codes -8..7 and the zero point is 0.
 *   zero_point given: c are the unsigned codes 0..15, as in
 *   bq_gemm_f16xu4_zp.
 *   The codes are exact in the products; each group's sum is accumulated in
 *   fp32 and multiplied by its scale in fp32, so nothing is rounded to 16
 *   bits before Y.  bq_quantize_sym over the (N * K / group, group) view of
 *   a weight matrix gives signed codes and scales in this layout.
 *
 *   X           device fp16, M rows of K elements, leading dimension ld_x
 *               (elements, >= K, a multiple of 8 when M > 1)
 *   Wp          device packed 4-bit codes (N, K) in layout `layout`
 *   scale       device fp16 (N, K / group), contiguous
 *   zero_point  device fp16 (N, K / group), contiguous, or NULL
 *   Y           device fp16 (M, N), contiguous
 *   X is finite: with M <= 8 or zero points the sums of X, and of X times the
 *   codes, are made apart, so that an infinity makes its row NaN also where the
 *   product would be infinite.
 *   Any M and any N.  M = 0 or N = 0 is an empty call; K = 0 writes zeros.
 *   With M > 8 the waits for copies are bounded (bq_set_wait_timeout_ns); one
 *   that gives up is reported as BQ_ERR_TIMEOUT by bq_device_status.
 *   Limits: group 32, 64 or 128, K a multiple of it, K <= 65536.
 *   Errors: INVALID_ARG (null pointers, negative sizes, ld_x < K, bad
 *   group, layout or activation), ALIGNMENT, UNSUPPORTED (K not a multiple
 *   of the group, sizes beyond the limits), CUDA.
 */
bq_status bq_gemm_f16xi4_group(const uint16_t* X, int64_t ld_x, const uint8_t* Wp, int layout, int64_t M, int64_t N,
                               int64_t K, int group, const uint16_t* scale, const uint16_t* zero_point,
                               int activation, uint16_t* Y, void* stream);

/*
 * bq_qk_norm_rope_kv4 -- between a decoder layer's QKV projection and its
 * attention: the RMS norm of every head of the queries and keys, their
 * rotation by position, and the write of keys and values into the 4-bit
 * cache, in one pass.
 *
 *   For a head x of D fp16 values, in IEEE fp32 operations, each rounded:
 *     ss   = sum of x[d] * x[d], by neighbouring pairs: ((x0^2 + x1^2) +
 *            (x2^2 + x3^2)) + ..., a binary tree over the head
 *     r    = 1 / sqrt(ss * (1 / D) + eps)
 *     y[d] = (x[d] * r) * weight[d]                (weight NULL: y = x)
 *   The first `rot` dims turn by the angles of the token's position:
 *     (a, b) -> (a * cos[p, i] - b * sin[p, i], b * cos[p, i] + a * sin[p, i])
 *   with (a, b) = (y[i], y[i + rot / 2]), or (y[2 i], y[2 i + 1]) if `pairs`.
 *   The result is rounded once to fp16: q_out for queries.  Keys so
 *   rounded, and the values as they came, go to the cache by groups:
 *     low  = min, step = fp16_rne((max - min) / 15),
 *     code = clamp(rne((x - low) / step), 0, 15)   (step 0: code 0)
 *   with IEEE fp32 subtraction and division.
 *
 *   q, k, v     device fp16; token t's heads are contiguous at t * ld_* (in
 *               elements, multiples of 8): views of one QKV matrix will do
 *   q_weight, k_weight  device fp16 (D) or NULL
 *   cos, sin    device fp32 (max_pos, rot / 2), or both NULL with rot = 0
 *   positions   device int32 (T); may be NULL when rot = 0
 *   slots       device int32 (T): the token's place in the pool; a negative
 *               slot writes nothing to the cache.  Two tokens of one call
 *               must not share a slot.
 *   q_out       device fp16 (T, q_heads, D)
 *   k_values, v_values  device fp16 (T, kv_heads, D) or NULL: the values
 *               that the cache holds after the call, fp16_rne(low + step *
 *               code), for attention over the prompt itself
 *   4-byte alignment is enough for positions and slots.
 *   A position outside [0, max_pos) or a slot past the pool is not used:
 *   the token's q_out and values are zero, its cache row is not written,
 *   and bq_device_status reports BQ_ERR_INVALID_ARG.
 *   NaN / Inf inputs are not supported.  kv_heads >= 1, q_heads >= 0; T = 0
 *   is an empty call.  rot is a multiple of 16, at most D.
 *   Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED (the pool's shape, rot not
 *   a multiple of 16, more than 65536 q_heads or 2**24 tokens), CUDA.
 */
bq_status bq_qk_norm_rope_kv4(const uint16_t* q, int64_t ld_q, const uint16_t* k, int64_t ld_k, const uint16_t* v,
                              int64_t ld_v, int64_t T, int64_t q_heads, int64_t kv_heads, int64_t D,
                              const uint16_t* q_weight, const uint16_t* k_weight, float eps, const float* cos,
                              const float* sin, int64_t max_pos, int64_t rot, int pairs, const int32_t* positions,
                              const int32_t* slots, uint8_t* codes, uint16_t* params, int64_t num_pages,
                              int64_t page_size, int64_t group, uint16_t* q_out, uint16_t* k_values,
                              uint16_t* v_values, void* stream);

/*
 * bq_attn_kv4 -- causal attention of new tokens over the 4-bit cache.
 *
 *   Sequence b has len = seq_lens[b] tokens in the cache, the last of them
 *   its n query tokens, which are rows cu_q[b] .. cu_q[b + 1] - 1 of q (cu_q
 *   NULL: one query token for each sequence, row b).  Query token i of the
 *   sequence stands at position p = len - n + i and sees the keys 0..p, or
 *   with window > 0 the keys p - window + 1 .. p.  Query head h reads kv head
 *   h / (q_heads / kv_heads).
 *     out = sum_t softmax_t(scale * q . k[t]) * v[t]
 *     lse = log sum_t exp(scale * q . k[t])         (natural log, fp32)
 *   A row that sees no key (len = 0, or p < 0) gives out = 0 and lse = -inf.
 *   Scores, the running maximum and sum, and the accumulators are fp32; the
 *   weight of a key, times its value's step, is rounded to fp16 for the
 *   tensor cores, with a power of two that follows the steps of each group of
 *   dims, 32 keys at a time (16 with D = 256 and several query rows): a weight
 *   (of the row's largest so far) times a step that is below 2**-14 of the
 *   largest step beside it is held to 2**-25 of that step instead of 11 bits.
 *   What the pool holds past a sequence's length (NaN included) does not
 *   reach the result.  NaN in what a row sees makes its result NaN; NaN in the
 *   params of a key may also reach query tokens of the same sequence that
 *   stand before the key, whose weight for it is 0.
 *
 *   q            device fp16, T rows of q_heads * D contiguous elements, leading
 *                dimension ld_q (a multiple of 8)
 *   block_table  device int32 (B, ld_table): page of tokens [j * page_size,
 *                (j + 1) * page_size) of a sequence; entries past its length
 *                are not read
 *   seq_lens     device int32 (B);  cu_q device int32 (B + 1) or NULL
 *   max_q        at least every sequence's number of query tokens (taken as 1
 *                where cu_q is NULL)
 *   max_len      at least every sequence's length (the size of the grid and
 *                of the workspace follow it), at most ld_table * page_size
 *   out          device fp16 (T, q_heads, D), contiguous
 *   lse          device fp32 (T, q_heads) or NULL
 *   workspace    device, bq_attn_kv4_workspace(...) bytes (may be NULL if that
 *                is 0); it need not be cleared, and calls that share one run
 *                in stream order
 *   4-byte alignment is enough for block_table, seq_lens and cu_q.
 *   Lengths beyond max_len and more than max_q query tokens are cut off, a
 *   sequence whose rows are not in [0, T) is left out, a page outside the pool
 *   is read as page 0, and bq_device_status reports BQ_ERR_INVALID_ARG.  Rows
 *   of out and lse that are cut off, left out or in no sequence are not written.
 *   T = 0 or B = 0 is an empty call.
 *   Errors: INVALID_ARG (null pointers, q_heads not a multiple of kv_heads,
 *   negative sizes, max_len above ld_table * page_size, an empty pool with
 *   max_len > 0, a workspace that is too small), ALIGNMENT, UNSUPPORTED (the
 *   pool's shape, max_len above 2**30, T * q_heads of 2**31 or more), CUDA.
 */
size_t bq_attn_kv4_workspace(int64_t B, int64_t q_heads, int64_t kv_heads, int64_t D, int64_t max_q,
                             int64_t max_len);
bq_status bq_attn_kv4(const uint16_t* q, int64_t ld_q, int64_t T, int64_t q_heads, int64_t kv_heads, int64_t D,
                      const uint8_t* codes, const uint16_t* params, int64_t num_pages, int64_t page_size,
                      int64_t group, const int32_t* block_table, int64_t ld_table, const int32_t* seq_lens,
                      const int32_t* cu_q, int64_t B, int64_t max_q, int64_t max_len, float scale, int64_t window,
                      uint16_t* out, float* lse, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BQ_DECODE_H_ */
