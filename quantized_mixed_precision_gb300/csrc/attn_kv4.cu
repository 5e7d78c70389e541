// Attention of new tokens over the 4-bit cache (bq_attn_kv4).
//
// One block per (query token, query head): the threads score 128 keys at a
// time, keep a running maximum and sum, and accumulate one output dim each.
#include <cuda_fp16.h>

#include "bq_device.cuh"
#include "decode_internal.h"

namespace bq {

namespace {

constexpr int AT = 128;

__device__ __forceinline__ float block_reduce(float v, bool max, float* red) {
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = max ? fmaxf(v, u) : v + u;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
  for (int w = 1; w < AT / 32; ++w) v = max ? fmaxf(v, red[w]) : v + red[w];
  return v;
}

__global__ void __launch_bounds__(AT) attn_kv4_kernel(AttnKv4Args a, int* status) {
  __shared__ float qs[256], ps[AT], red[AT / 32];
  __shared__ int64_t rows[AT];
  const int64_t t = blockIdx.x;
  const int h = blockIdx.y, tid = threadIdx.x;
  const int D = a.pool.D, heads = a.pool.heads, P = a.pool.page_size, G = a.pool.group, groups = D / G;
  const int kvh = h / (a.q_heads / heads);
  // the token's sequence: the last b with cu_q[b] <= t
  int64_t b = t, first = t, count = 1;
  if (a.cu_q) {
    int64_t lo = 0, hi = a.B - 1;
    while (lo < hi) {
      const int64_t mid = (lo + hi + 1) / 2;
      if (a.cu_q[mid] <= t) lo = mid; else hi = mid - 1;
    }
    b = lo;
    first = a.cu_q[b];
    count = a.cu_q[b + 1] - first;
  }
  if (t < first || t >= first + count) return;
  int64_t len = a.lens[b];
  if ((len > a.max_len || count > a.max_q) && tid == 0) record_error(status, BQ_ERR_INVALID_ARG);
  if (t - first >= a.max_q) return;
  const int64_t p = len - count + (t - first);
  int64_t end = p + 1 < a.max_len ? p + 1 : a.max_len;
  int64_t begin = a.window > 0 && p + 1 - a.window > 0 ? p + 1 - a.window : 0;
  for (int d = tid; d < D; d += AT) qs[d] = __half2float(reinterpret_cast<const __half*>(a.q)[t * a.ld_q + h * D + d]);
  float m = -INFINITY, l = 0.0f, acc[2] = {};
  __syncthreads();
  for (int64_t k0 = begin; k0 < end; k0 += AT) {
    const int64_t key = k0 + tid;
    float s = -INFINITY;
    int64_t vrow = -1;
    if (key < end) {
      const int page = a.table[b * a.ld_table + key / P];
      if (page >= 0 && page < a.pool.num_pages) {
        const int64_t krow = (((int64_t)page * 2) * heads + kvh) * P + key % P;
        vrow = krow + (int64_t)heads * P;
        const uint8_t* c = a.pool.codes + krow * (D / 2);
        const __half2* pr = reinterpret_cast<const __half2*>(a.pool.params) + krow * groups;
        s = 0.0f;
        for (int g = 0; g < groups; ++g) {
          float u = 0.0f, qsum = 0.0f;
          for (int j = 0; j < G / 2; ++j) {
            const uint32_t byte = c[g * (G / 2) + j];
            const float q0 = qs[g * G + 2 * j], q1 = qs[g * G + 2 * j + 1];
            u += q0 * (float)(byte & 15) + q1 * (float)(byte >> 4);
            qsum += q0 + q1;
          }
          s += __low2float(pr[g]) * u + __high2float(pr[g]) * qsum;
        }
        s *= a.scale;
      } else {
        record_error(status, BQ_ERR_INVALID_ARG);
      }
    }
    const float mn = fmaxf(m, block_reduce(s, true, red));
    const float keep = mn == -INFINITY ? 1.0f : __expf(m - mn);
    const float pe = s == -INFINITY ? 0.0f : __expf(s - mn);
    ps[tid] = pe;
    rows[tid] = vrow;
    l = l * keep + block_reduce(pe, false, red);
    m = mn;
    for (int i = 0; i < 2; ++i) {
      const int d = tid + i * AT;
      if (d >= D) break;
      acc[i] *= keep;
      for (int j = 0; j < AT; ++j) {
        if (rows[j] < 0) continue;
        const uint32_t byte = a.pool.codes[rows[j] * (D / 2) + d / 2];
        const __half2 pr = reinterpret_cast<const __half2*>(a.pool.params)[rows[j] * groups + d / G];
        acc[i] += ps[j] * (__low2float(pr) * (float)((byte >> (4 * (d & 1))) & 15) + __high2float(pr));
      }
    }
    __syncthreads();
  }
  for (int i = 0; i < 2; ++i) {
    const int d = tid + i * AT;
    if (d < D)
      reinterpret_cast<__half*>(a.out)[(t * a.q_heads + h) * D + d] = __float2half_rn(l > 0.0f ? acc[i] / l : 0.0f);
  }
  if (a.lse && tid == 0) a.lse[t * a.q_heads + h] = l > 0.0f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t attn_kv4_workspace(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

cudaError_t launch_attn_kv4(const AttnKv4Args& a, cudaStream_t stream) {
  int* status = nullptr;
  cudaError_t e = device_status_ptr(&status);
  if (e != cudaSuccess) return e;
  attn_kv4_kernel<<<dim3((unsigned)a.T, (unsigned)a.q_heads), AT, 0, stream>>>(a, status);
  return cudaGetLastError();
}

}  // namespace bq
