// fp16 activations times 4-bit weights with group scales (bq_gemm_f16xi4_group).
//
//   Y[i, j] = act( sum_g s[j, g] * ( sum_{k in g} x[i, k] u[j, k] - z[j, g] * sum_{k in g} x[i, k] ) )
// with unsigned codes u; signed codes are u - 8 once their top bit is flipped, so
// they are the case z = 8.  The tensor cores multiply the codes as fp16
// subnormals (kv4_device.cuh: one LOP3 for two codes, exact), weights as the A
// operand (16 columns j a tile) and up to 8 rows i as its columns.  The sums of X
// over a group, which the zero point needs, are made from the same tiles, so that
// it costs no pass over X.  A group's sums start from zero, are scaled in fp32 and
// added to fp32 accumulators: nothing is rounded to 16 bits before Y.
#include <cuda_fp16.h>

#include "bq_device.cuh"
#include "decode_internal.h"
#include "gemm_common.cuh"
#include "kv4_device.cuh"

namespace bq {

namespace {

// ---------------------------------------------------------------------------
// Up to 8 rows of X: one read of the weights is what it cannot do without.  A
// block owns 16 columns and its warps take stages of K in turn, each through a
// ring of its own, so that no warp waits for another before the end.  A stage is
// 512 k (256 with more than two rows of X, whose share of the ring would leave
// fewer blocks on an SM): 512 against 1024 at M = 1 was 7.9 against 8.5 us, 256
// against 512 at M = 8 18.1 against 23 (two blocks fewer an SM; 16.1 and 19.9 now,
// groups of 128 and groups of 64 with zero points).
// 1 x 11008 x 4096 in groups of 128, one call after another on weights larger
// than L2: 7.1 us, 3.3 TB/s.  The copies alone take 3.7; the arithmetic, about 170
// instructions for 16 columns and 128 k in a warp, 3.8 after a block's data has
// come, and the blocks of the next call get their shared memory when this one's
// are done, so that the two overlap in part only.
// ---------------------------------------------------------------------------
constexpr int SMEM_MAX = 227 * 1024;

constexpr int SUM_BYTES = 2 * 16 * 4;        // sums of two rows over a stage's groups of 32

struct StagePlan {
  int k_log2;        // k of a stage: 256 or 512
  int stages;        // of a warp's ring
  int groups;        // most groups a warp meets
  // ring, then (step, zero) of 16 rows for each of the warp's groups
  int warp_bytes(int M) const { return stages * ((8 + 2 * M) << k_log2) + 64 * groups + SUM_BYTES; }
};

// XOR of the address bits of weight row r: loads of 16, 8 or 4 bytes of each
// quad lane of rows 0..7 (a multiple of 128 bytes apart) then touch every bank once.
__device__ __forceinline__ int row_swizzle(int r) { return (r & 1) << 6 | (r & 2) << 4 | (r & 4) << 2; }

// TMA's swizzle of rows of 64 bytes.
__device__ __forceinline__ int weight_swizzle(int r) { return (r & 6) << 3; }

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
  // The sums of X over a group: with one or two rows (the long stages) from the pieces as they are put in order, else
  // from an MMA with A = 1 beside each product.  That MMA cost 1.3 of 8.2 us at M = 1.
  constexpr bool SUMS = KLOG == 9;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * 16;
  const int ngroups = K / G, nst = (K + (1 << KLOG) - 1) >> KLOG;
  const int mine_n = nst > warp ? (nst - warp + warps - 1) / warps : 0;
  const int stage = WB + M * XROW;
  uint8_t* const mine = smem + warp * (plan.stages * stage + 64 * plan.groups + SUM_BYTES);
  uint32_t* const sz = reinterpret_cast<uint32_t*>(mine + plan.stages * stage);   // [group][16 rows] (scale, zero)
  float* const xsum = reinterpret_cast<float*>(sz + 16 * plan.groups);            // [row of X][group of the stage]
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
      if constexpr (SUMS) {
        // (whole warps come here; past K the pieces are stale, in groups that are not used)
        float s = sum_h8(v);
#pragma unroll
        for (int d = 1; d < G / 8; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        const int m = c / (XROW / 16), at = c % (XROW / 16) ^ (m & 1) << 2;
        if (c % (G / 8) == 0) xsum[m * SG + at / (G / 8)] = s;
      }
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
      float lo[4], hi[4];
      [[maybe_unused]] float sum[2][4];
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
          if constexpr (!SUMS) {
            mma_f16_zero(sum[0], mk.one[0], mk.one[1], mk.one[2], mk.one[3], v.x, v.y);
            mma_f16_zero(sum[1], mk.one[0], mk.one[1], mk.one[2], mk.one[3], v.z, v.w);
          }
        } else {
          mma_f16(lo, l0, l1, l2, l3, v.x, v.y);
          mma_f16(hi, h0, h1, h2, h3, v.z, v.w);
          if constexpr (!SUMS) {
            mma_f16(sum[0], mk.one[0], mk.one[1], mk.one[2], mk.one[3], v.x, v.y);
            mma_f16(sum[1], mk.one[0], mk.one[1], mk.one[2], mk.one[3], v.z, v.w);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float2 p = unpack_h2(sg[16 * j + 8 * r]);
        const float z = ZP ? p.y : 8.0f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (c > 0 && M == 1) break;        // uniform; odd columns are not stored then
          const int i = 2 * r + c;
          const float u = fmaf(hi[i], 0.0625f, lo[i]);
          const float all = SUMS ? xsum[c * SG + j] : sum[0][i] + sum[1][i];
          acc[i] = fmaf(p.x, fmaf(u, 16777216.0f, -z * all), acc[i]);
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

// ---------------------------------------------------------------------------
// More rows of X: blocks of 128 columns j and up to 64 rows i, K split over a
// cluster.  A warp owns 32 columns and up to 32 rows; the warps of a block share
// X, a slab of 128 k at a time, and two warps with the same columns their
// weights.  The codes are converted to exact signed fp16 (a conversion serves all
// rows of a warp, so its subtraction is cheap here and one accumulator a group is
// enough).  A slab comes by TMA, which one thread asks for: with 16-byte copies by
// all of them a third of a slab's time went into issuing those (61 x 8192 x 8192
// took 41.9 us, 256 rows 138).  What a slab needs besides (the order of X for plain codes, its sums
// over groups for zero points, which add (8 - z) s sum) is made while the slab
// before it is multiplied, so that a slab costs one barrier.
// What bounds it is mma.sync, whose pipe is busy 42 % of a launch at 61 rows and
// what most warps wait for, with the fill of the ring before and the cluster's
// sum after it; at 16 rows (15 %) it is those two and the latency of a slab.
// 61 x 8192 x 8192 in groups of 128 takes 38.3 us (214 TFLOP/s, 0.9 TB/s of
// weights), 16 x 11008 x 4096 in groups of 64 with zero points 16.0 (1.6 TB/s).  Every
// 64 rows convert the weights again, which bounds prompts: 256 x 8192 x 8192 122 us
// (282 TFLOP/s), 256 x 11008 x 4096 100 (231), 2048 x 4096 x 4096 269 (255).
// ---------------------------------------------------------------------------
constexpr int GB_SLAB = 128;                 // k of a slab
constexpr int GB_COLS = 128;                 // columns j of a block
constexpr int GB_STAGES = 4;                 // slabs in the ring
constexpr uint64_t DRAIN_NS = 2000000000;    // limit of the wait for copies in flight after another wait gave up

// Blocks an SM: NT row tiles of 8 a warp, RG warps along the rows
constexpr int block_slots(int nt, int rg) { return rg == 2 ? 2 : (nt == 4 ? 3 : 4); }

template <int NT, int RG, int G>
struct BlockCfg {
  static constexpr int THREADS = 128 * RG;
  static constexpr int ROWS = 8 * NT * RG;
  static constexpr int X_B = ROWS * GB_SLAB * 2;
  static constexpr int W_B = GB_COLS * GB_SLAB / 2;
  static constexpr int SG = GB_SLAB / G;
  static constexpr int SUMS = ROWS * SG;                             // sums of X over a slab's groups
  static constexpr int SB = 8 / SG;                                  // slabs with 8 groups
  static constexpr int STEPS = GB_COLS * 8;                          // (step, zero) of 8 groups
  static constexpr int STAGE_B = X_B + W_B;
  static constexpr int RING = GB_STAGES * STAGE_B + 2 * SUMS * 4 + 2 * STEPS * 4;
  static constexpr int ACC = ROWS * (GB_COLS + 4) * 4;               // partial results, for the cluster
  static constexpr int SMEM = (RING > ACC ? RING : ACC) + 1024;      // TMA's swizzles repeat every 1024 bytes
};

// Exact signed fp16 pairs of a word's codes, in the order of its masks: signed codes c, or unsigned ones less 8.
template <bool ZP>
__device__ __forceinline__ void signed_codes(uint32_t w, uint32_t (&h)[4]) {
  const uint32_t y = w >> 8;
  if constexpr (ZP) {
    h[0] = hsub2_u32((w & CODE_LO) | H2_MAGIC, H2_1032);
    h[1] = hfma2_u32((w & CODE_HI) | H2_MAGIC, H2_INV16, H2_NEG72);
    h[2] = hsub2_u32((y & CODE_LO) | H2_MAGIC, H2_1032);
    h[3] = hfma2_u32((y & CODE_HI) | H2_MAGIC, H2_INV16, H2_NEG72);
  } else {
    cvt_i4x8_f16(w, h);
  }
}

template <int NT, int RG, int G, bool ZP>
__global__ void __launch_bounds__(128 * RG, block_slots(NT, RG))
    gemm_group_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w, bool inter,
                      int M, int N, int K, const uint16_t* __restrict__ scale, const uint16_t* __restrict__ zero, int actfn,
                      __half* __restrict__ y, int parts, uint64_t timeout_ns, int* status) {
  using C = BlockCfg<NT, RG, G>;
  constexpr int WORDS = G / 32;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[GB_STAGES];
  uint8_t* const smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int wcol = warp & 3, wrow = warp >> 2;              // this warp's columns and rows
  const int part = blockIdx.x % parts, unit = blockIdx.x / parts;   // a cluster is the parts of a unit
  const int m0 = blockIdx.y * C::ROWS, rows = min(C::ROWS, M - m0);
  const int slabs = (K + GB_SLAB - 1) / GB_SLAB, ngroups = K / G;
  const int s0 = slabs * part / parts, s1 = slabs * (part + 1) / parts;   // this part's slabs (at most 512 in all)
  float* const sums = reinterpret_cast<float*>(smem + GB_STAGES * C::STAGE_B);
  uint32_t* const steps = reinterpret_cast<uint32_t*>(sums + 2 * C::SUMS);

  // A slab is three TMA boxes: two of 64 k of X (rows of 128 bytes, 16-byte piece c of row r at c ^ (r & 7)) and the
  // codes (rows of 64 bytes, piece c at c ^ (r >> 1 & 3)).  What lies past M, N and K comes as zeros.
  if (tid == 0) {
#pragma unroll
    for (int i = 0; i < GB_STAGES; ++i) mbar_init(&full[i], 1);
    mbar_fence_init();
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  auto issue = [&](int s) {                                 // (thread 0)
    if (s >= s1) return;
    const int st = (s - s0) & (GB_STAGES - 1);
    uint8_t* const to = smem + st * C::STAGE_B;
    mbar_arrive_expect_tx(&full[st], C::STAGE_B);
    tma_load_2d(to, &tmap_x, s * GB_SLAB, m0, &full[st]);
    tma_load_2d(to + C::X_B / 2, &tmap_x, s * GB_SLAB + 64, m0, &full[st]);
    tma_load_2d(to + C::X_B, &tmap_w, s * (GB_SLAB / 2), unit * GB_COLS, &full[st]);
  };
  auto arrived = [&](int s) {                               // every thread sees the copies of slab s
    return s >= s1 || mbar_wait(&full[(s - s0) & (GB_STAGES - 1)], ((s - s0) / GB_STAGES) & 1, timeout_ns, status);
  };
  const int xc = tid & 15, x_row = tid >> 4;                // a piece of a row of X
  constexpr int XR = C::THREADS / 16;
  // What slab s needs besides its copies
  auto ready = [&](int s) {
    if (s >= s1) return;
    uint8_t* const xs = smem + ((s - s0) & (GB_STAGES - 1)) * C::STAGE_B;
    if (ZP || !inter) {
      float* const to = sums + ((s - s0) & 1) * C::SUMS;
#pragma unroll
      for (int r = x_row; r < C::ROWS; r += XR) {           // (whole warps: rows past the last are not used)
        uint4* const at = reinterpret_cast<uint4*>(xs + (xc >> 3) * (C::X_B / 2) + r * 128 + (((xc ^ r) & 7) << 4));
        const uint4 p = *at;
        if (ZP) {
          // a group's pieces are those of G / 8 neighbouring lanes
          float v = sum_h8(p);
#pragma unroll
          for (int o = 1; o < G / 8; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o, 16);
          if (xc % (G / 8) == 0) to[r * C::SG + xc / (G / 8)] = v;
        }
        if (!inter)
          *at = make_uint4(prmt(p.x, p.z, 0x5410u), prmt(p.x, p.z, 0x7632u), prmt(p.y, p.w, 0x5410u),
                           prmt(p.y, p.w, 0x7632u));
      }
    }
  };
  if (tid == 0) {
    issue(s0);
    issue(s0 + 1);
    issue(s0 + 2);
  }

  float acc[2][NT][4];
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[r][nt][i] = 0.0f;
  // (step, zero) of the block's columns, 8 groups at a time (16 bytes of a column; two bytes a load, as many sectors as
  // the weights have, took 700 cycles a slab), loaded a whole eight before they are passed on through shared memory
  const size_t s_at = (size_t)min(unit * GB_COLS + (tid & 127), N - 1) * ngroups;
  const bool whole = (ngroups & 7) == 0;                    // 16-byte loads of 8 groups are aligned
  uint4 es = make_uint4(0, 0, 0, 0), ez = es;
  auto load_eight = [&](int e) {
    if (tid >= GB_COLS || e * 8 >= ngroups || e * C::SB >= s1) return;
    if (whole) {
      es = __ldg(reinterpret_cast<const uint4*>(scale + s_at + e * 8));
      if (ZP) ez = __ldg(reinterpret_cast<const uint4*>(zero + s_at + e * 8));
      return;
    }
    uint32_t a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int g0 = min(e * 8 + 2 * i, ngroups - 1), g1 = min(e * 8 + 2 * i + 1, ngroups - 1);
      a[i] = scale[s_at + g0] | (uint32_t)scale[s_at + g1] << 16;
      if (ZP) b[i] = zero[s_at + g0] | (uint32_t)zero[s_at + g1] << 16;
    }
    es = make_uint4(a[0], a[1], a[2], a[3]);
    if (ZP) ez = make_uint4(b[0], b[1], b[2], b[3]);
  };
  auto store_eight = [&](int e) {
    if (tid >= GB_COLS) return;
    uint32_t* const to = steps + (e & 1) * C::STEPS + tid;
    const uint32_t a[4] = {es.x, es.y, es.z, es.w}, b[4] = {ez.x, ez.y, ez.z, ez.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      to[2 * i * GB_COLS] = prmt(a[i], b[i], 0x5410u);
      to[(2 * i + 1) * GB_COLS] = prmt(a[i], b[i], 0x7632u);
    }
  };
  load_eight(s0 / C::SB);
  // A wait that gives up is reported and nothing is copied from then on; the sums go on with what is there.
  bool ok = true;
  int lost = s0;
  auto await = [&](int s) {
    if (!ok) return;
    ok = arrived(s);
    lost = s;
  };
  await(s0);
  ready(s0);
  store_eight(s0 / C::SB);
  load_eight(s0 / C::SB + 1);

  // Word i of group j: piece t * WORDS + i of the group.  With four words (groups of 128) the lanes 2 and 3, whose
  // pieces lie in the other box, take them in the order 2, 3, 0, 1, which keeps eight lanes' loads on different banks.
  const uint32_t x_row0 = g * 128;
  auto x_at = [&](int i, int j) -> uint32_t {
    const int piece = j * (G / 8) + t * WORDS + (WORDS == 4 ? i ^ (t & 2) : i);
    return x_row0 + (piece >> 3) * (C::X_B / 2) + (((piece ^ g) & 7) << 4);
  };
  for (int s = s0; s < s1; ++s) {
    if (!inter) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // X was put in order before the next copy
    __syncthreads();                         // slab s is ready, and slab s - 1 has been read
    if (tid == 0 && ok) issue(s + 3);
    await(s + 1);
    ready(s + 1);
    if ((s + 1) % C::SB == 0) {              // the next slab begins an eight: its steps, and the loads of the one after
      store_eight((s + 1) / C::SB);
      load_eight((s + 1) / C::SB + 1);
    }
    const uint32_t* const sp = steps + ((s / C::SB) & 1) * C::STEPS + s % C::SB * C::SG * GB_COLS + wcol * 32 + g;
    const uint8_t* const xs = smem + ((s - s0) & (GB_STAGES - 1)) * C::STAGE_B + wrow * NT * 8 * 128;
    const float* const sum = sums + ((s - s0) & 1) * C::SUMS + wrow * NT * 8 * C::SG;
    const uint8_t* const ws = smem + ((s - s0) & (GB_STAGES - 1)) * C::STAGE_B + C::X_B + wcol * 32 * 64;
#pragma unroll
    for (int j = 0; j < C::SG; ++j) {
      if (s * C::SG + j >= ngroups) break;           // uniform
      float c[2][NT][4];
      uint32_t wd[4][WORDS];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* p = ws + (((g * 64) + j * (G / 2) + t * (G / 8)) ^ weight_swizzle(g)) + i * 512;
        if constexpr (WORDS == 4) {
          const uint4 q = *reinterpret_cast<const uint4*>(p);
          wd[i][0] = t & 2 ? q.z : q.x;
          wd[i][1] = t & 2 ? q.w : q.y;
          wd[i][2] = t & 2 ? q.x : q.z;
          wd[i][3] = t & 2 ? q.y : q.w;
        }
        else if constexpr (WORDS == 2) *reinterpret_cast<uint2*>(wd[i]) = *reinterpret_cast<const uint2*>(p);
        else wd[i][0] = *reinterpret_cast<const uint32_t*>(p);
      }
#pragma unroll
      for (int i = 0; i < WORDS; ++i) {
        uint32_t h[4][4];
#pragma unroll
        for (int r = 0; r < 4; ++r) signed_codes<ZP>(wd[r][i], h[r]);
        // blocks of four tiles: all first halves of the word before the second, so that no MMA waits for the last
        constexpr int NB = NT < 4 ? NT : 4;
#pragma unroll
        for (int nb = 0; nb < NT; nb += NB) {
          uint4 v[NB];
#pragma unroll
          for (int n = 0; n < NB; ++n)
            v[n] = *reinterpret_cast<const uint4*>(xs + 8 * (nb + n) * 128 + x_at(i, j));
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float(&d)[4] = c[r][nb + n];
              if (i == 0) mma_f16_zero(d, h[2 * r][0], h[2 * r + 1][0], h[2 * r][1], h[2 * r + 1][1], v[n].x, v[n].y);
              else mma_f16(d, h[2 * r][0], h[2 * r + 1][0], h[2 * r][1], h[2 * r + 1][1], v[n].x, v[n].y);
            }
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r)
              mma_f16(c[r][nb + n], h[2 * r][2], h[2 * r + 1][2], h[2 * r][3], h[2 * r + 1][3], v[n].z, v[n].w);
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float2 p0 = unpack_h2(sp[j * GB_COLS + 16 * r]), p1 = unpack_h2(sp[j * GB_COLS + 16 * r + 8]);
        const float a0 = p0.x, a1 = p1.x, b0 = 8.0f - p0.y, b1 = 8.0f - p1.y;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float x0 = 0.0f, x1 = 0.0f;
          if (ZP) {
            x0 = sum[(8 * nt + 2 * t) * C::SG + j];
            x1 = sum[(8 * nt + 2 * t + 1) * C::SG + j];
          }
          acc[r][nt][0] = fmaf(a0, ZP ? fmaf(b0, x0, c[r][nt][0]) : c[r][nt][0], acc[r][nt][0]);
          acc[r][nt][1] = fmaf(a0, ZP ? fmaf(b0, x1, c[r][nt][1]) : c[r][nt][1], acc[r][nt][1]);
          acc[r][nt][2] = fmaf(a1, ZP ? fmaf(b1, x0, c[r][nt][2]) : c[r][nt][2], acc[r][nt][2]);
          acc[r][nt][3] = fmaf(a1, ZP ? fmaf(b1, x1, c[r][nt][3]) : c[r][nt][3], acc[r][nt][3]);
        }
      }
    }
  }

  // ---- add the cluster's shares of K in rank order, each block a share of the columns ----
  if (tid == 0 && !ok)                                      // copies in flight end before their memory is used again
    for (int s = lost; s < min(lost + 3, s1); ++s)
      mbar_wait(&full[(s - s0) & (GB_STAGES - 1)], ((s - s0) / GB_STAGES) & 1, DRAIN_NS, status);
  __syncthreads();
  float* const pa = reinterpret_cast<float*>(smem);         // [row of X][column], padded
  constexpr int LD = GB_COLS + 4;
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        pa[(8 * (wrow * NT + nt) + 2 * t + (i & 1)) * LD + wcol * 32 + 16 * r + g + 8 * (i >> 1)] = acc[r][nt][i];
  if (parts > 1) cluster_sync_all(); else __syncthreads();
  const int c0 = GB_COLS * part / parts, c1 = GB_COLS * (part + 1) / parts, cols = c1 - c0;
  const uint32_t pa_u = smem_u32(pa);
  for (int i = tid; i < rows * cols; i += C::THREADS) {
    const int r = i / cols, cc = c0 + i - r * cols;
    const int n = unit * GB_COLS + cc;
    if (n >= N) continue;
    float v = 0.0f;
    if (parts == 1) {
      v = pa[r * LD + cc];
    } else {
      for (int p = 0; p < parts; ++p) {
        float u;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(u) : "r"(mapa_shared(pa_u + (r * LD + cc) * 4, p)));
        v += u;
      }
    }
    y[(size_t)(m0 + r) * N + n] = __float2half_rn(apply_act(v, actfn));
  }
  if (parts > 1) cluster_sync_all();                        // nobody leaves while its shares are read
}

template <int NT, int RG, int G, bool ZP>
cudaError_t launch_block(const GroupGemmArgs& a, cudaStream_t stream) {
  using C = BlockCfg<NT, RG, G>;
  const int64_t units = (a.N + GB_COLS - 1) / GB_COLS, zs = (a.M + C::ROWS - 1) / C::ROWS;
  // K is split over up to four blocks with at least two slabs each, so that the fullest block's share times the rounds
  // of the grid is least; where that is equal, over more blocks.  61 x 8192 x 8192 takes 38.3 us with four parts, 45.3 with
  // two; 61 x 11008 x 4096 in groups of 64 43.9 with four (40 blocks wait for a second round), 36.7 with three; 256 x 8192 x
  // 8192 121.6 with four, 133.1 with two; 16 x 4096 x 1024 8.6 with two, 5.7 with four.  Clusters of eight cost more than
  // they bring (44.4, and 16 x 11008 x 4096 19.1 instead of 16.2).
  const int slabs = (int)((a.K + GB_SLAB - 1) / GB_SLAB);
  constexpr int FIT = 228 * 1024 / (C::SMEM + 1024);
  const int64_t slots = (int64_t)sm_count() * (FIT < block_slots(NT, RG) ? FIT : block_slots(NT, RG));
  int parts = 1;
  int64_t least = INT64_MAX;
  for (int p = 1; p <= 4 && (p == 1 || slabs >= 2 * p); ++p) {
    const int64_t time = (units * zs * p + slots - 1) / slots * ((slabs + p - 1) / p);
    if (time <= least) {
      least = time;
      parts = p;
    }
  }
  auto kern = gemm_group_kernel<NT, RG, G, ZP>;
  cudaError_t e = set_smem_once(kern, C::SMEM);
  if (e != cudaSuccess) return e;
  CUtensorMap tmap_x, tmap_w;
  e = make_map_rows(&tmap_x, a.x, 2, a.K, a.ld_x, a.M, 64, C::ROWS, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e == cudaSuccess) e = make_map(&tmap_w, a.w, 1, a.K / 2, a.N, 64, GB_COLS, CU_TENSOR_MAP_SWIZZLE_64B);
  int* status = nullptr;
  if (e == cudaSuccess) e = device_status_ptr(&status);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(parts * units), (unsigned)zs);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)parts;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, tmap_x, tmap_w, a.layout == BQ_LAYOUT_INTERLEAVED, (int)a.M, (int)a.N, (int)a.K,
                            a.scale, a.zero_point, a.actfn, reinterpret_cast<__half*>(a.y), parts,
                            (uint64_t)wait_timeout_ns(), status);
}

// Up to 8 rows the GEMV, for more the blocks.  Both measured, us of the GEMV / of the blocks:
//   rows                               1            2            4            6            8
//   11008 x 4096, groups of 128     7.1 / 10.6  10.2 / 10.6  10.6 / 10.7  12.5 / 10.9  16.1 / 11.0
//   the same, 64 with zero points   9.6 / 14.5  13.1 / 14.5  13.1 / 14.7  14.7 / 15.1  19.9 / 15.0
//   8192 x 8192, groups of 128     12.7 / 17.8  13.0 / 17.9  19.3 / 17.9  23.3 / 18.3  23.2 / 18.4
//   1000 x 1024, 32 with zeros      2.8 / 4.3    2.8 / 4.4    2.8 / 4.4    2.9 / 4.9    2.9 / 4.8
// With many tiles the blocks are ahead from 4 to 7 rows on, with few never: the bound stands where the small call needs it,
// and a rule on rows and tiles would take up to 5 us off 5 to 8 rows.
template <int G, bool ZP>
cudaError_t launch_rows(const GroupGemmArgs& a, cudaStream_t stream) {
  if (a.M <= 8) return launch_gemv<G, ZP>(a, stream);
  if (a.M <= 16) return launch_block<2, 1, G, ZP>(a, stream);
  if (a.M <= 32) return launch_block<4, 1, G, ZP>(a, stream);
  return launch_block<4, 2, G, ZP>(a, stream);
}

}  // namespace

cudaError_t launch_gemm_group(const GroupGemmArgs& g, cudaStream_t stream) {
  const bool zp = g.zero_point != nullptr;
  constexpr int64_t MOST = 32768;          // rows of a launch
  for (int64_t m = 0; m < g.M; m += MOST) {
    GroupGemmArgs a = g;
    a.x = g.x + m * g.ld_x;
    a.y = g.y + m * g.N;
    a.M = g.M - m < MOST ? g.M - m : MOST;
    cudaError_t e;
    if (g.group == 128)
      e = zp ? launch_rows<128, true>(a, stream) : launch_rows<128, false>(a, stream);
    else if (g.group == 64)
      e = zp ? launch_rows<64, true>(a, stream) : launch_rows<64, false>(a, stream);
    else
      e = zp ? launch_rows<32, true>(a, stream) : launch_rows<32, false>(a, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace bq
