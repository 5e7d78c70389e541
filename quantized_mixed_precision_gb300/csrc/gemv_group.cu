// fp16 activations times 4-bit weights with group scales (bq_gemm_f16xi4_group).
//
//   Y[i, j] = act( sum_g s[j, g] * ( sum_{k in g} x[i, k] u[j, k] - z[j, g] * sum_{k in g} x[i, k] ) )
// with unsigned codes u; signed codes are u - 8 once their top bit is flipped, so
// they are the case z = 8.  The tensor cores multiply the codes as fp16
// subnormals (kv4_device.cuh: one LOP3 for two codes, exact), weights as the A
// operand (16 columns j a tile) and up to 8 rows i as its columns.  Beside each
// product an MMA with A = 1 sums the same activations, so that the zero point
// costs no pass over X.  A group's sums start from zero, are scaled in fp32 and
// added to fp32 accumulators: nothing is rounded to 16 bits before Y.
#include <cuda_fp16.h>

#include "bq_device.cuh"
#include "decode_internal.h"
#include "kv4_device.cuh"

namespace bq {

namespace {

// D = A * B with a zero C.
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// ---------------------------------------------------------------------------
// Up to 8 rows of X: bound by one read of the weights.  A block owns 16 columns
// and its warps take stages of K in turn, each through a ring of its own, so
// that no warp waits for another before the end.  A stage is 512 k (256 with
// more than two rows of X, whose share of the ring would leave fewer blocks on
// an SM): N = 11008, K = 4096 takes 7.9 us at M = 1 with 512, 8.5 with 1024, and
// 18.1 at M = 8 with 256, 23 with 512 (two blocks fewer an SM).
// ---------------------------------------------------------------------------
constexpr int SMEM_MAX = 227 * 1024;

struct StagePlan {
  int k_log2;        // k of a stage: 256 or 512
  int stages;        // of a warp's ring
  int groups;        // most groups a warp meets
  // ring, then (step, zero) of 16 rows for each of the warp's groups
  int warp_bytes(int M) const { return stages * ((8 + 2 * M) << k_log2) + 64 * groups; }
};

// XOR of the address bits of weight row r: loads of 16, 8 or 4 bytes of each
// quad lane of rows 0..7 (a multiple of 128 bytes apart) then touch every bank once.
__device__ __forceinline__ int row_swizzle(int r) { return (r & 1) << 6 | (r & 2) << 4 | (r & 4) << 2; }

// Codes of a word as MMA operands; signed codes become u = c + 8 by flipping their top bit, in the same LOP3.  The
// masks come in registers that the compiler cannot see through: with constants it put one of the two into a register
// again for every LOP3.
struct Masks {
  uint32_t lo, hi, flip_lo, flip_hi;
  uint32_t one[4];   // an A operand of ones, in registers of its own
};
__device__ __forceinline__ Masks make_masks() {
  Masks m;
  asm volatile("mov.b32 %0, 0x000f000f;" : "=r"(m.lo));
  asm volatile("mov.b32 %0, 0x00f000f0;" : "=r"(m.hi));
  asm volatile("mov.b32 %0, 0x00080008;" : "=r"(m.flip_lo));
  asm volatile("mov.b32 %0, 0x00800080;" : "=r"(m.flip_hi));
#pragma unroll
  for (int i = 0; i < 4; ++i) asm volatile("mov.b32 %0, 0x3c003c00;" : "=r"(m.one[i]));
  return m;
}
template <bool ZP>
__device__ __forceinline__ uint32_t codes(uint32_t w, uint32_t mask, uint32_t flip) {
  uint32_t r;
  if constexpr (ZP) r = w & mask;
  else asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(r) : "r"(w), "r"(mask), "r"(flip));   // (w & mask) ^ flip
  return r;
}

// (640 threads bound the registers at 96, which lets five blocks of four warps share an SM)
template <int G, bool ZP, int KLOG>
__global__ void __launch_bounds__(640, 1) gemv_group_kernel(const __half* __restrict__ x, int64_t ld_x,
                                                            const uint8_t* __restrict__ w, bool inter, int M, int N,
                                                            int K, const uint16_t* __restrict__ scale,
                                                            const uint16_t* __restrict__ zero, int actfn,
                                                            __half* __restrict__ y, StagePlan plan) {
  constexpr int SG = (1 << KLOG) / G;                    // groups of a stage
  constexpr int WB = 8 << KLOG;                          // bytes of a stage's weights
  constexpr int WROW = 1 << (KLOG - 1), XROW = 2 << KLOG;   // bytes of a row of weights, of X
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * 16;
  const int ngroups = K / G, nst = (K + (1 << KLOG) - 1) >> KLOG;
  const int mine_n = nst > warp ? (nst - warp + warps - 1) / warps : 0;
  const int stage = WB + M * XROW;
  uint8_t* const mine = smem + warp * (plan.stages * stage + 64 * plan.groups);
  uint32_t* const sz = reinterpret_cast<uint32_t*>(mine + plan.stages * stage);   // [group][16 rows] (scale, zero)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- scales and zero points of this warp's groups: the first loads go out before the stages' ----
  const int sn = 16 * SG * mine_n;
  const size_t s_row = (size_t)min(n0 + (lane & 15), N - 1) * ngroups;
  auto sz_load = [&](int i) -> uint32_t {
    const int j = i >> 4;                    // group of this warp; the row is lane & 15
    const int group = (warp + j / SG * warps) * SG + j % SG;
    if (i >= sn || group >= ngroups) return 0;
    return ZP ? scale[s_row + group] | (uint32_t)zero[s_row + group] << 16 : scale[s_row + group];
  };
  uint32_t first[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) first[i] = sz_load(lane + 32 * i);

  // ---- copies of a stage: weight rows in pieces of 16 bytes, lanes along a row; the same k of X ----
  constexpr int LROW = WROW / 16;                        // pieces of a weight row: 8, 16 or 32
  constexpr int RSTEP = 32 / LROW;                       // rows of one copy of the warp
  const int row_b = K / 2;
  const int wr0 = lane / LROW, wc = lane % LROW * 16;
  const uint32_t ring = smem_u32(mine);
  const uint32_t x_off = (lane / (G / 8) * (G / 8) + lane % (G / 32) * 4 + lane % (G / 8) / (G / 32)) * 16;
  const uint8_t* const wsrc = w + (size_t)(n0 + wr0) * row_b + wc;
  const int last = N - 1 - n0 - wr0;                     // rows past the last column repeat it
  auto issue = [&](int i) {
    if (i < mine_n) {
      const int s = warp + i * warps;
      const uint32_t ro = plan.stages == 1 ? 0 : (i & 1) * stage;
      if (s * WROW + wc < row_b) {
        const uint8_t* src = wsrc + s * WROW;
#pragma unroll
        for (int r = 0; r < 16; r += RSTEP)
          cp_async_16_u(ring + ro + (((wr0 + r) * WROW + wc) ^ row_swizzle(wr0 + r)),
                        src + (int64_t)min(r, last) * row_b);
      }
      // X: pieces of 8 k, those of a group in the order of the loads (word i, quad lane t)
      const __half* xsrc = x + (s << KLOG) + 8 * lane;
      for (int m = 0; m < M; ++m, xsrc += ld_x)
#pragma unroll
        for (int c = 0; c < 1 << (KLOG - 8); ++c)
          if ((s << KLOG) + 8 * (32 * c + lane) < K)
            cp_async_16_l1(ring + ro + WB + m * XROW + (x_off ^ ((m & 1) << 6)) + c * 512, xsrc + c * 256);
    }
    cp_async_commit();
  };
  issue(0);
  if (plan.stages == 2) issue(1);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (lane + 32 * i < sn) sz[lane + 32 * i] = first[i];
  for (int i = lane + 128; i < sn; i += 32) sz[i] = sz_load(i);
  __syncwarp();

  const Masks mk = make_masks();
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  // columns of B past the last row of X repeat row 0: they are not stored
  const int xm = g < M ? g : 0;
  const int xo = WB + xm * XROW + t * 16;
  for (int q = 0; q < mine_n; ++q) {
    if (plan.stages == 2) cp_async_wait<1>(); else cp_async_wait<0>();
    __syncwarp();
    uint8_t* const st = mine + (plan.stages == 1 ? 0 : (q & 1) * stage);
    // Each 8 values of X into the order of the masks, as register pairs of a B operand: the low codes of a word stand
    // for k 0, 1 and 4, 5 (plain words: 0, 4 and 2, 6), the high ones for 2, 3 and 6, 7 (1, 5 and 3, 7).
    for (int c = lane; c < M * (XROW / 16); c += 32) {
      uint4* const p = reinterpret_cast<uint4*>(st + WB) + c;
      const uint4 v = *p;
      *p = inter ? make_uint4(v.x, v.z, v.y, v.w)
                 : make_uint4(prmt(v.x, v.z, 0x5410u), prmt(v.y, v.w, 0x5410u), prmt(v.x, v.z, 0x7632u),
                              prmt(v.y, v.w, 0x7632u));
    }
    __syncwarp();
    const uint8_t* const ws = st + g * WROW;
    const uint8_t* const xs0 = st + xo + ((xm & 1) << 6);
    const uint8_t* const xs1 = st + xo + (((xm & 1) ^ 1) << 6);
    const int count = min(SG, ngroups - (warp + q * warps) * SG);
    const uint32_t* const sg = sz + q * SG * 16 + g;
#pragma unroll
    for (int j = 0; j < SG; ++j) {
      if (j >= count) break;                 // uniform
      // lane t of a quad holds k [t G / 4, (t + 1) G / 4) of the group: G / 32 words
      constexpr int WORDS = G / 32;
      uint32_t w0[WORDS], w1[WORDS];
      {
        const uint8_t* p = ws + ((j * (G / 2) + t * (G / 8)) ^ row_swizzle(g));
        if constexpr (WORDS == 4) {
          *reinterpret_cast<uint4*>(w0) = *reinterpret_cast<const uint4*>(p);
          *reinterpret_cast<uint4*>(w1) = *reinterpret_cast<const uint4*>(p + WB / 2);
        } else if constexpr (WORDS == 2) {
          *reinterpret_cast<uint2*>(w0) = *reinterpret_cast<const uint2*>(p);
          *reinterpret_cast<uint2*>(w1) = *reinterpret_cast<const uint2*>(p + WB / 2);
        } else {
          w0[0] = *reinterpret_cast<const uint32_t*>(p);
          w1[0] = *reinterpret_cast<const uint32_t*>(p + WB / 2);
        }
      }
      float lo[4], hi[4], sum[2][4];
#pragma unroll
      for (int i = 0; i < WORDS; ++i) {
        // odd rows have the halves of each 128 bytes swapped
        constexpr int STEP = 64;             // bytes of the quad's pieces of one word
        const int at = (j * (G / 32) + i) * STEP;
        const uint4 v = *reinterpret_cast<const uint4*>((at & 64 ? xs1 : xs0) + (at & ~64));
        const uint32_t a = w0[i], b = w1[i], a8 = a >> 8, b8 = b >> 8;
        const uint32_t l0 = codes<ZP>(a, mk.lo, mk.flip_lo), l1 = codes<ZP>(b, mk.lo, mk.flip_lo);
        const uint32_t l2 = codes<ZP>(a8, mk.lo, mk.flip_lo), l3 = codes<ZP>(b8, mk.lo, mk.flip_lo);
        const uint32_t h0 = codes<ZP>(a, mk.hi, mk.flip_hi), h1 = codes<ZP>(b, mk.hi, mk.flip_hi);
        const uint32_t h2 = codes<ZP>(a8, mk.hi, mk.flip_hi), h3 = codes<ZP>(b8, mk.hi, mk.flip_hi);
        if (i == 0) {
          mma_f16_zero(lo, l0, l1, l2, l3, v.x, v.y);
          mma_f16_zero(hi, h0, h1, h2, h3, v.z, v.w);
          mma_f16_zero(sum[0], mk.one[0], mk.one[1], mk.one[2], mk.one[3], v.x, v.y);
          mma_f16_zero(sum[1], mk.one[0], mk.one[1], mk.one[2], mk.one[3], v.z, v.w);
        } else {
          mma_f16(lo, l0, l1, l2, l3, v.x, v.y);
          mma_f16(hi, h0, h1, h2, h3, v.z, v.w);
          mma_f16(sum[0], mk.one[0], mk.one[1], mk.one[2], mk.one[3], v.x, v.y);
          mma_f16(sum[1], mk.one[0], mk.one[1], mk.one[2], mk.one[3], v.z, v.w);
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float2 p = unpack_h2(sg[16 * j + 8 * r]);
        const float z = ZP ? p.y : 8.0f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int i = 2 * r + c;
          const float u = fmaf(hi[i], 0.0625f, lo[i]);
          acc[i] = fmaf(p.x, fmaf(u, 16777216.0f, -z * (sum[0][i] + sum[1][i])), acc[i]);
        }
      }
    }
    __syncwarp();                            // the stage is read before it is filled again
    if (plan.stages == 2) issue(q + 2); else issue(q + 1);
  }

  // ---- join the warps' shares of K in warp order ----
  cp_async_wait<0>();
  __syncthreads();
  float* const red = reinterpret_cast<float*>(smem);        // [warp][8 rows of X][16 columns]
#pragma unroll
  for (int i = 0; i < 4; ++i) red[warp * 128 + (2 * t + (i & 1)) * 16 + g + 8 * (i >> 1)] = acc[i];
  __syncthreads();
  const int m = threadIdx.x >> 4, n = n0 + (threadIdx.x & 15);
  if (threadIdx.x < 128 && m < M && n < N) {
    float v = 0.0f;
    for (int i = 0; i < warps; ++i) v += red[i * 128 + threadIdx.x];
    y[(size_t)m * N + n] = __float2half_rn(apply_act(v, actfn));
  }
}

template <int G, bool ZP>
cudaError_t launch_gemv(const GroupGemmArgs& a, cudaStream_t stream) {
  const int64_t tiles = (a.N + 15) / 16;
  const int M = (int)a.M, K = (int)a.K;
  StagePlan plan{};
  plan.k_log2 = K >= 2048 && M <= 2 ? 9 : 8;
  // 4 warps a block; where the tiles are few, up to 16, each with at least one stage of at least 256 k
  int warps = 4;
  while (warps < 16 && tiles * warps < sm_count() * 8 && K >= 512 * warps) {
    warps *= 2;
    if (plan.k_log2 > 8 && K < warps << plan.k_log2) --plan.k_log2;
  }
  auto fit = [&]() {
    const int nst = (K + (1 << plan.k_log2) - 1) >> plan.k_log2, each = (nst + warps - 1) / warps;
    plan.stages = each > 1 ? 2 : 1;
    plan.groups = each * (1 << plan.k_log2) / G;
    return warps * plan.warp_bytes(M) <= SMEM_MAX;
  };
  while (!fit()) {
    if (plan.k_log2 > 8) --plan.k_log2; else warps /= 2;
  }
  auto kern = plan.k_log2 == 9 ? gemv_group_kernel<G, ZP, 9> : gemv_group_kernel<G, ZP, 8>;
  cudaError_t e = set_smem_once(kern, SMEM_MAX);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)tiles);
  cfg.blockDim = dim3(warps * 32);
  cfg.dynamicSmemBytes = (size_t)(warps * plan.warp_bytes(M));
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, reinterpret_cast<const __half*>(a.x), a.ld_x, a.w,
                            a.layout == BQ_LAYOUT_INTERLEAVED, M, (int)a.N, K, a.scale, a.zero_point, a.actfn,
                            reinterpret_cast<__half*>(a.y), plan);
}

}  // namespace

cudaError_t launch_gemm_group(const GroupGemmArgs& g, cudaStream_t stream) {
  const bool zp = g.zero_point != nullptr;
  for (int64_t m = 0; m < g.M; m += 8) {
    GroupGemmArgs a = g;
    a.x = g.x + m * g.ld_x;
    a.y = g.y + m * g.N;
    a.M = g.M - m < 8 ? g.M - m : 8;
    cudaError_t e;
    if (g.group == 128)
      e = zp ? launch_gemv<128, true>(a, stream) : launch_gemv<128, false>(a, stream);
    else if (g.group == 64)
      e = zp ? launch_gemv<64, true>(a, stream) : launch_gemv<64, false>(a, stream);
    else
      e = zp ? launch_gemv<32, true>(a, stream) : launch_gemv<32, false>(a, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace bq
