// Norm and rotation of queries and keys with the write of keys and values
// into the 4-bit cache (bq_qk_norm_rope_kv4), one pass over the QKV rows.
//
// One warp per head of a token: the head is staged in shared memory as fp32
// after the norm, rotated, rounded to fp16 and, for keys and values, coded by
// groups.  Every step is one IEEE fp32 operation in the order the header
// states, so codes and steps are bit-exact.
#include <cuda_fp16.h>

#include "bq_device.cuh"
#include "decode_internal.h"

namespace bq {

namespace {

constexpr int KW_WARPS = 4;

__global__ void __launch_bounds__(KW_WARPS * 32) kv4_write_kernel(Kv4WriteArgs a, int* status) {
  __shared__ float head[KW_WARPS][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int D = a.pool.D, heads = a.pool.heads;
  const int64_t per = a.q_heads + 2 * heads;
  const int64_t item = (int64_t)blockIdx.x * KW_WARPS + warp;
  if (item >= a.T * per) return;
  const int64_t t = item / per;
  int h = (int)(item - t * per);
  const int what = h < a.q_heads ? 0 : (h < a.q_heads + heads ? 1 : 2);   // query, key, value
  h -= what == 0 ? 0 : (what == 1 ? a.q_heads : a.q_heads + heads);
  const __half* src = reinterpret_cast<const __half*>(what == 0 ? a.q + t * a.ld_q
                                                                : (what == 1 ? a.k + t * a.ld_k : a.v + t * a.ld_v)) +
                      (int64_t)h * D;
  const __half* wt = reinterpret_cast<const __half*>(what == 0 ? a.q_weight : (what == 1 ? a.k_weight : nullptr));
  float* y = head[warp];
  const int slot = a.slots[t];
  const int pos = a.rot ? a.positions[t] : 0;
  const bool ok = (a.rot == 0 || (pos >= 0 && pos < a.max_pos)) && slot < a.pool.num_pages * a.pool.page_size;
  if (!ok && lane == 0) record_error(status, BQ_ERR_INVALID_ARG);

  for (int d = lane; d < D; d += 32) y[d] = __half2float(src[d]);
  __syncwarp();
  if (wt) {
    // tree over neighbouring pairs: lane owns D / 32 consecutive dims
    const int per_lane = D / 32;
    float part[8];
    for (int i = 0; i < per_lane; ++i) part[i] = __fmul_rn(y[lane * per_lane + i], y[lane * per_lane + i]);
    for (int n = per_lane; n > 1; n >>= 1)
      for (int i = 0; i < n / 2; ++i) part[i] = __fadd_rn(part[2 * i], part[2 * i + 1]);
    float ss = part[0];
    for (int o = 1; o < 32; o <<= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, o));
    const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(ss, 1.0f / (float)D), a.eps)));
    for (int d = lane; d < D; d += 32) y[d] = __fmul_rn(__fmul_rn(y[d], r), __half2float(wt[d]));
  }
  __syncwarp();
  if (what < 2 && ok) {
    for (int i = lane; i < a.rot / 2; i += 32) {
      const int ia = a.pairs ? 2 * i : i, ib = a.pairs ? 2 * i + 1 : i + a.rot / 2;
      const float c = a.cos[(int64_t)pos * (a.rot / 2) + i], s = a.sin[(int64_t)pos * (a.rot / 2) + i];
      const float ya = y[ia], yb = y[ib];
      y[ia] = __fsub_rn(__fmul_rn(ya, c), __fmul_rn(yb, s));
      y[ib] = __fadd_rn(__fmul_rn(yb, c), __fmul_rn(ya, s));
    }
  }
  __syncwarp();
  if (what == 0) {
    __half* o = reinterpret_cast<__half*>(a.q_out) + (t * a.q_heads + h) * (int64_t)D;
    for (int d = lane; d < D; d += 32) o[d] = __float2half_rn(ok ? y[d] : 0.0f);
    return;
  }
  const int groups = D / a.pool.group;
  const bool store = ok && slot >= 0;
  const int64_t page = store ? slot / a.pool.page_size : 0;
  const int off = store ? slot % a.pool.page_size : 0;
  const int64_t row = ((page * 2 + (what - 1)) * heads + h) * a.pool.page_size + off;
  uint16_t* vals = what == 1 ? a.k_values : a.v_values;
  for (int g = 0; g < groups; ++g) {
    const int G = a.pool.group;
    float lo = INFINITY, hi = -INFINITY;
    for (int d = lane; d < G; d += 32) {
      const float v = __half2float(__float2half_rn(y[g * G + d]));
      y[g * G + d] = v;
      lo = fminf(lo, v);
      hi = fmaxf(hi, v);
    }
    for (int o = 16; o > 0; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    lo = __fadd_rn(lo, 0.0f);   // -0 becomes +0
    __syncwarp();
    const __half step = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.0f));
    const float st = __half2float(step);
    for (int j = lane; j < G / 2; j += 32) {
      uint32_t byte = 0;
      for (int e = 0; e < 2; ++e) {
        const int d = g * G + 2 * j + e;
        float c = st > 0.0f ? rintf(__fdiv_rn(__fsub_rn(y[d], lo), st)) : 0.0f;
        c = fminf(fmaxf(c, 0.0f), 15.0f);
        byte |= (uint32_t)c << (4 * e);
        if (vals)
          reinterpret_cast<__half*>(vals)[(t * heads + h) * (int64_t)D + d] =
              __float2half_rn(ok ? __fadd_rn(__fmul_rn(c, st), lo) : 0.0f);
      }
      if (store) a.pool.codes[row * (D / 2) + g * (G / 2) + j] = (uint8_t)byte;
    }
    if (store && lane == 0)
      reinterpret_cast<__half2*>(a.pool.params)[row * groups + g] = __halves2half2(step, __float2half_rn(lo));
  }
}

}  // namespace

cudaError_t launch_kv4_write(const Kv4WriteArgs& a, cudaStream_t stream) {
  int* status = nullptr;
  cudaError_t e = device_status_ptr(&status);
  if (e != cudaSuccess) return e;
  const int64_t items = a.T * (a.q_heads + 2 * (int64_t)a.pool.heads);
  const int64_t blocks = (items + KW_WARPS - 1) / KW_WARPS;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  kv4_write_kernel<<<(unsigned)blocks, KW_WARPS * 32, 0, stream>>>(a, status);
  return cudaGetLastError();
}

}  // namespace bq
