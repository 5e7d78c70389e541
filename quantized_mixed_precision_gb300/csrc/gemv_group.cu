// fp16 activations times 4-bit weights with group scales (bq_gemm_f16xi4_group).
//
//   Y[i, j] = act( sum_g s[j, g] * ( sum_{k in g} x[i, k] c[j, k] - z[j, g] * sum_{k in g} x[i, k] ) )
//
// One warp per output column j and up to 8 rows i: the lanes stride over the
// 32-bit words of the column's packed codes.
#include <cuda_fp16.h>

#include "bq_device.cuh"
#include "decode_internal.h"

namespace bq {

namespace {

constexpr int GG_ROWS = 8;

__global__ void __launch_bounds__(128) gemm_group_kernel(const __half* __restrict__ x, int64_t ld_x,
                                                         const uint32_t* __restrict__ w, bool inter, int M, int N,
                                                         int K, int group, const __half* __restrict__ scale,
                                                         const __half* __restrict__ zero, int actfn,
                                                         __half* __restrict__ y) {
  const int lane = threadIdx.x & 31;
  const int n = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int m0 = blockIdx.y * GG_ROWS;
  if (n >= N) return;
  const int rows = min(GG_ROWS, M - m0);
  float acc[GG_ROWS] = {};
  for (int i = lane; i < K / 8; i += 32) {
    const uint32_t word = w[(size_t)n * (K / 8) + i];
    const int g = i * 8 / group;
    const float s = __half2float(scale[(size_t)n * (K / group) + g]);
    const float z = zero ? __half2float(zero[(size_t)n * (K / group) + g]) : 0.0f;
    for (int e = 0; e < 8; ++e) {
      const int pos = inter ? ((e & 1) * 4 + (e >> 1)) : e;
      int c = (word >> (4 * pos)) & 15;
      if (!zero && c > 7) c -= 16;
      const float wv = ((float)c - z) * s;
      for (int m = 0; m < rows; ++m) acc[m] += wv * __half2float(x[(m0 + m) * ld_x + 8 * i + e]);
    }
  }
  for (int m = 0; m < rows; ++m) {
    float v = acc[m];
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) y[(size_t)(m0 + m) * N + n] = __float2half_rn(apply_act(v, actfn));
  }
}

}  // namespace

cudaError_t launch_gemm_group(const GroupGemmArgs& g, cudaStream_t stream) {
  const int64_t by = (g.M + GG_ROWS - 1) / GG_ROWS;
  for (int64_t y0 = 0; y0 < by; y0 += 65535) {
    const int64_t ny = by - y0 < 65535 ? by - y0 : 65535;
    const dim3 grid((unsigned)((g.N + 3) / 4), (unsigned)ny);
    gemm_group_kernel<<<grid, 128, 0, stream>>>(
        reinterpret_cast<const __half*>(g.x) + y0 * GG_ROWS * g.ld_x, g.ld_x, reinterpret_cast<const uint32_t*>(g.w),
        g.layout == BQ_LAYOUT_INTERLEAVED, (int)(g.M - y0 * GG_ROWS), (int)g.N, (int)g.K, g.group,
        reinterpret_cast<const __half*>(g.scale), reinterpret_cast<const __half*>(g.zero_point), g.actfn,
        reinterpret_cast<__half*>(g.y) + y0 * GG_ROWS * g.N);
  }
  return cudaGetLastError();
}

}  // namespace bq
