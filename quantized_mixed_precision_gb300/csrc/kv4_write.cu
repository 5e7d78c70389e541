// Norm and rotation of queries and keys with the write of keys and values
// into the 4-bit cache (bq_qk_norm_rope_kv4), one pass over the QKV rows.
//
// The work is bound by memory: a head is read once and written once, and its
// norm, rotation and codes are made in registers.  A thread owns 8 consecutive
// dims of a head (one 16-byte load), D / 8 threads a head, and a block of 128
// threads walks the heads of one token, so that the token's angles and the
// norm weights of the thread's dims are loaded once for all heads.  The loads of
// several heads are issued before the first is used.  What then competes with
// memory is the issue of instructions, so the fp32 work runs in packed pairs
// (each lane of a packed operation is an ordinary IEEE operation).
// 8192 tokens of 32 + 2 x 8 heads of 128 dims take 46.6 us: 4.6 TB/s of the 6.8 that
// a plain copy has, with 76 % of the issue slots taken (219 instructions for two
// heads and warp), which is what bounds it; 777 tokens of 16 + 2 x 16 heads of 64
// dims 5.3 us, 5 tokens 2.7, both the latency of one launch.  Bounded at
// 7 blocks an SM (72 registers): 8 took 49.7 us, 6 47.9, unbounded 51.2.
//
// Every step is one IEEE fp32 operation in the order the header states, so
// codes and steps are bit-exact: the sum of squares is a tree over neighbouring
// pairs (three levels in the thread, the rest by shuffles), and the rotation's
// two products and their sum are rounded separately (the sign of a product is
// put into the sine, which is exact; dims that do not turn use cosine 1, sine 0).
//
// Quotients without a division.  For y / s with y of 24 significant bits and s of
// at most 11 (an fp16 step, or 15) and c = 1 / s within 2**-22: t1 = RN(y c),
// e = RN(y - t1 s) in one fma, t2 = RN(t1 + e c).  Before its rounding t2 lies
// within 2**-43 of y / s (relative), and y / s is at least 2**-36 away from every
// midpoint m of two fp32 numbers: y - m s is a multiple of the last place of
// m s, and not 0, since m has 25 bits with an odd last one, so that m s is no
// number of 24 bits.  So t2 = RN(y / s), exactly.
#include <cuda_fp16.h>

#include "bq_device.cuh"
#include "decode_internal.h"
#include "kv4_device.cuh"
#include "quant_math.cuh"

namespace bq {

namespace {

constexpr int WT = 128;   // threads of a block
constexpr int WQ = 4;     // items (a head for each D / 8 threads) of queries whose loads are issued together
constexpr int WKV = 2;    // the same for keys and values

// a * b rounded, for a product that an addition follows: ptxas contracts a packed mul.rn and add.rn into one fma
// (seen as outputs one place off), which an fma with an addend that it does not know keeps apart.  mz: -0.
__device__ __forceinline__ P2 product2(P2 a, P2 b, P2 mz) { return fma2(a, b, mz); }
__device__ __forceinline__ float rcp_near(float x) {   // 1 / x within 2**-22
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The 8 values of a thread as pairs (0, 2), (1, 3), (4, 6), (5, 7), so that the
// neighbouring pairs of the sum of squares meet in packed additions.
__device__ __forceinline__ void unpack8(const uint4& x, P2 (&y)[4]) {
  const float2 a = unpack_h2(x.x), b = unpack_h2(x.y), c = unpack_h2(x.z), d = unpack_h2(x.w);
  y[0] = p2(a.x, b.x);
  y[1] = p2(a.y, b.y);
  y[2] = p2(c.x, d.x);
  y[3] = p2(c.y, d.y);
}
__device__ __forceinline__ uint4 pack8(const P2 (&y)[4]) {
  const float2 a = f2(y[0]), b = f2(y[1]), c = f2(y[2]), d = f2(y[3]);
  return make_uint4(pack_h2(a.x, b.x), pack_h2(a.y, b.y), pack_h2(c.x, d.x), pack_h2(c.y, d.y));
}

// What a thread needs of its token and its 8 dims.
struct Turn {
  P2 c[4], s[4];     // angles, the sine with the sign of its product
  int partner;       // lane with the other dim of each pair (itself where the pairs are its own, or nothing turns)
  bool any, pairs;
  P2 mz;             // (-0, -0)
};

template <int L>
__device__ __forceinline__ void norm8(P2 (&y)[4], const P2 (&w)[4], float eps, P2 mz) {
  P2 q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = product2(y[i], y[i], mz);
  const float2 u = f2(add2(q[0], q[1])), v = f2(add2(q[2], q[3]));   // (0+1, 2+3), (4+5, 6+7)
  float ss = __fadd_rn(__fadd_rn(u.x, u.y), __fadd_rn(v.x, v.y));
#pragma unroll
  for (int o = 1; o < L; o <<= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, o));
  const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(ss, 1.0f / (float)(8 * L)), eps)));
  const P2 rr = p2(r, r);
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = mul2(mul2(y[i], rr), w[i]);
}

__device__ __forceinline__ void turn8(P2 (&y)[4], const Turn& t) {
  P2 o[4];
  if (t.pairs) {     // dims 0 and 1, 2 and 3: y[0] with y[1]; 4 and 5, 6 and 7: y[2] with y[3]
    o[0] = y[1];
    o[1] = y[0];
    o[2] = y[3];
    o[3] = y[2];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = f2(y[i]);
      o[i] = p2(__shfl_sync(0xffffffffu, v.x, t.partner), __shfl_sync(0xffffffffu, v.y, t.partner));
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = add2(product2(y[i], t.c[i], t.mz), product2(o[i], t.s[i], t.mz));
}

template <int D>
__global__ void __launch_bounds__(WT, 7) kv4_write_kernel(const Kv4WriteArgs a, int page_log2, float minus_zero,
                                                          int* status) {
  constexpr int L = D / 8;              // lanes of a head
  constexpr int HEADS = WT / L;         // heads of an item: what the block works on at a time
  const int l = threadIdx.x % L, sub = threadIdx.x / L, lane = threadIdx.x & 31;
  const int64_t t = blockIdx.x;
  const int heads = a.pool.heads, kv_heads2 = 2 * heads, q_heads = a.q_heads;
  const int qi = (q_heads + HEADS - 1) / HEADS, ki = (kv_heads2 + HEADS - 1) / HEADS;
  // this block's share of the items: the queries' first, then the keys' and values'
  int i0 = 0, i1 = qi + ki;
  if (gridDim.y > 1) {
    i0 = (int)((uint32_t)i1 * blockIdx.y / gridDim.y);
    i1 = (int)((uint32_t)i1 * (blockIdx.y + 1) / gridDim.y);
  }
  const int q1 = min(i1, qi), kv0 = max(i0 - qi, 0), kv1 = i1 - qi;

  // head `h` of keys and values counts on from the keys' to the values': one pointer for each, less the keys' heads
  const uint16_t* const qsrc = a.q + t * a.ld_q + 8 * l;
  const uint16_t* const ksrc = a.k + t * a.ld_k + 8 * l;
  const uint16_t* const vsrc = a.v + t * a.ld_v + 8 * l - heads * D;
  uint4 xq[WQ], xkv[WKV];
  auto fetch_q = [&](int base) {
#pragma unroll
    for (int u = 0; u < WQ; ++u) {
      const int h = (base + u) * HEADS + sub;
      if (base + u < q1 && h < q_heads) xq[u] = __ldcs(reinterpret_cast<const uint4*>(qsrc + h * D));
    }
  };
  auto fetch_kv = [&](int base) {
#pragma unroll
    for (int u = 0; u < WKV; ++u) {
      const int h = (base + u) * HEADS + sub;
      if (base + u < kv1 && h < kv_heads2)
        xkv[u] = __ldcs(reinterpret_cast<const uint4*>((h < heads ? ksrc : vsrc) + h * D));
    }
  };
#pragma unroll
  for (int u = 0; u < WQ; ++u) xq[u] = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int u = 0; u < WKV; ++u) xkv[u] = make_uint4(0, 0, 0, 0);
  fetch_q(i0);
  fetch_kv(kv0);

  const int slot = a.slots[t];
  const int pos = a.rot ? a.positions[t] : 0;
  uint16_t* const qdst = a.q_out + t * q_heads * D + 8 * l;
  uint16_t* const kval = a.k_values ? a.k_values + t * heads * D + 8 * l : nullptr;
  uint16_t* const vval = a.v_values ? a.v_values + (t - 1) * heads * D + 8 * l : nullptr;
  if ((a.rot != 0 && (pos < 0 || pos >= a.max_pos)) || slot >= a.pool.num_pages << page_log2) {
    // a position or slot that does not exist (uniform)
    if (threadIdx.x == 0) record_error(status, BQ_ERR_INVALID_ARG);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int h = i0 * HEADS + sub; h < min(q1 * HEADS, q_heads); h += HEADS) *reinterpret_cast<uint4*>(qdst + h * D) = zero;
    for (int h = kv0 * HEADS + sub; h < min(kv1 * HEADS, kv_heads2); h += HEADS) {
      uint16_t* const val = h < heads ? kval : vval;
      if (val) *reinterpret_cast<uint4*>(val + h * D) = zero;
    }
    return;
  }

  Turn turn;
  turn.pairs = a.pairs != 0;
  turn.any = a.rot != 0;
  turn.mz = p2(minus_zero, minus_zero);
  {
    const int half = a.rot / 2;
    const bool mine = 8 * l < a.rot, second = mine && 8 * l >= half;
    turn.partner = !mine ? lane : (second ? lane - half / 8 : lane + half / 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      turn.c[i] = p2(1.0f, 1.0f);
      turn.s[i] = p2(0.0f, 0.0f);
    }
    if (mine) {
      const int64_t at = (int64_t)pos * half + (turn.pairs ? 4 * l : (second ? 8 * l - half : 8 * l));
      const float4 c0 = *reinterpret_cast<const float4*>(a.cos + at), s0 = *reinterpret_cast<const float4*>(a.sin + at);
      if (turn.pairs) {
        turn.c[0] = turn.c[1] = p2(c0.x, c0.y);
        turn.c[2] = turn.c[3] = p2(c0.z, c0.w);
        turn.s[0] = p2(-s0.x, -s0.y);
        turn.s[1] = p2(s0.x, s0.y);
        turn.s[2] = p2(-s0.z, -s0.w);
        turn.s[3] = p2(s0.z, s0.w);
      } else {
        const float4 c1 = *reinterpret_cast<const float4*>(a.cos + at + 4);
        const float4 s1 = *reinterpret_cast<const float4*>(a.sin + at + 4);
        const float sign = second ? 1.0f : -1.0f;
        turn.c[0] = p2(c0.x, c0.z);
        turn.c[1] = p2(c0.y, c0.w);
        turn.c[2] = p2(c1.x, c1.z);
        turn.c[3] = p2(c1.y, c1.w);
        turn.s[0] = p2(sign * s0.x, sign * s0.z);
        turn.s[1] = p2(sign * s0.y, sign * s0.w);
        turn.s[2] = p2(sign * s1.x, sign * s1.z);
        turn.s[3] = p2(sign * s1.y, sign * s1.w);
      }
    }
  }

  // ---- queries ----
  if (i0 < q1) {
    P2 w[4];
    if (a.q_weight) unpack8(*reinterpret_cast<const uint4*>(a.q_weight + 8 * l), w);
    for (int base = i0; base < q1; base += WQ) {
      if (base != i0) fetch_q(base);
#pragma unroll
      for (int u = 0; u < WQ; ++u) {
        if (base + u >= q1) break;                     // uniform
        P2 y[4];
        unpack8(xq[u], y);
        if (a.q_weight) norm8<L>(y, w, a.eps, turn.mz);
        if (turn.any) turn8(y, turn);
        const int h = (base + u) * HEADS + sub;
        if (h < q_heads) __stcs(reinterpret_cast<uint4*>(qdst + h * D), pack8(y));
      }
    }
  }
  if (kv0 >= kv1) return;

  // ---- keys and values ----
  P2 w[4];
  if (a.k_weight) unpack8(*reinterpret_cast<const uint4*>(a.k_weight + 8 * l), w);
  const int gl = a.pool.group / 8, groups = D / a.pool.group;   // lanes of a group, groups of a head
  const bool store = slot >= 0;
  // key row of head 0 in the pool; head h (on to the values') is h << page_log2 rows further
  const int64_t row0 = store ? (((int64_t)(slot >> page_log2) * kv_heads2) << page_log2) + (slot & ((1 << page_log2) - 1)) : 0;
  uint8_t* const code0 = a.pool.codes + row0 * (D / 2) + 4 * l;
  __half2* const param0 = reinterpret_cast<__half2*>(a.pool.params) + row0 * groups + l / gl;
  const bool first_lane = (l & (gl - 1)) == 0;
  for (int base = kv0; base < kv1; base += WKV) {
    if (base != kv0) fetch_kv(base);
#pragma unroll
    for (int u = 0; u < WKV; ++u) {
      if (base + u >= kv1) break;                      // uniform
      const int h = (base + u) * HEADS + sub;          // 0 .. heads - 1: keys, then values
      uint4 o = xkv[u];
      P2 y[4];
      if ((base + u) * HEADS < heads) {                // uniform: some of the item's heads are keys
        unpack8(o, y);
        if (a.k_weight) norm8<L>(y, w, a.eps, turn.mz);
        if (turn.any) turn8(y, turn);
        if (h < heads) o = pack8(y);
      }
      // (minimum, -maximum) of the group in one register: one shuffle and one minimum a level
      const __half2 h0 = *reinterpret_cast<const __half2*>(&o.x), h1 = *reinterpret_cast<const __half2*>(&o.y);
      const __half2 h2 = *reinterpret_cast<const __half2*>(&o.z), h3 = *reinterpret_cast<const __half2*>(&o.w);
      const __half2 mn = __hmin2(__hmin2(h0, h1), __hmin2(h2, h3));
      const __half2 mx = __hneg2(__hmax2(__hmax2(h0, h1), __hmax2(h2, h3)));
      __half2 mm = __hmin2(__lows2half2(mn, mx), __highs2half2(mn, mx));
#pragma unroll
      for (int d = 1; d < 16; d <<= 1)
        if (d < gl) mm = __hmin2(mm, __shfl_xor_sync(0xffffffffu, mm, d));   // uniform
      const float lo = __fadd_rn(__low2float(mm), 0.0f);   // a minimum of -0 is stored as +0
      const float range = __fsub_rn(-__high2float(mm), lo);
      constexpr float C15 = 1.0f / 15.0f;
      const float t1 = __fmul_rn(range, C15);
      const __half step = __float2half_rn(__fmaf_rn(__fmaf_rn(t1, -15.0f, range), C15, t1));
      const float st = __half2float(step);
      const float rcp = st > 0.0f ? rcp_near(st) : 0.0f;
      unpack8(o, y);
      const P2 nlo = p2(-lo, -lo), nst = p2(-st, -st), cc = p2(rcp, rcp), magic = p2(RNE_MAGIC, RNE_MAGIC);
      // a quotient is above 15.5 only where a subnormal step was rounded down
      const bool clamp = __any_sync(0xffffffffu, st < 6.103515625e-05f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const P2 x = add2(y[i], nlo);
        const P2 q = mul2(x, cc);
        P2 z = fma2(fma2(q, nst, x), cc, q);
        if (clamp) {
          const float2 f = f2(z);
          z = p2(fminf(f.x, 15.0f), fminf(f.y, 15.0f));
        }
        y[i] = add2(z, magic);                         // rounds to the code, in the low bits
      }
      if (h >= kv_heads2) continue;
      uint16_t* const val = h < heads ? kval : vval;
      if (val) {
        const P2 unmagic = p2(-RNE_MAGIC, -RNE_MAGIC), plo = p2(lo, lo), pst = p2(st, st);
        P2 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fma2(add2(y[i], unmagic), pst, plo);   // (the product is exact)
        __stcs(reinterpret_cast<uint4*>(val + h * D), pack8(v));
      }
      if (store) {
        // bytes: dims (0, 1), (2, 3), (4, 5), (6, 7)
        const float2 a0 = f2(y[0]), a1 = f2(y[1]), a2 = f2(y[2]), a3 = f2(y[3]);
        const uint32_t b0 = (code_byte(a1.x) << 4) + code_byte(a0.x), b1 = (code_byte(a1.y) << 4) + code_byte(a0.y);
        const uint32_t b2 = (code_byte(a3.x) << 4) + code_byte(a2.x), b3 = (code_byte(a3.y) << 4) + code_byte(a2.y);
        const int64_t rows = (int64_t)h << page_log2;
        *reinterpret_cast<uint32_t*>(code0 + rows * (D / 2)) =
            __byte_perm(__byte_perm(b0, b1, 0x0040), __byte_perm(b2, b3, 0x0040), 0x5410);
        if (first_lane) param0[rows * groups] = __halves2half2(step, __float2half_rn(lo));
      }
    }
  }
}

template <int D>
cudaError_t launch_write(const Kv4WriteArgs& a, int* status, cudaStream_t stream) {
  constexpr int HEADS = WT / (D / 8);
  const int64_t items = (a.q_heads + HEADS - 1) / HEADS + (2 * (int64_t)a.pool.heads + HEADS - 1) / HEADS;
  // one block a token; with few tokens a token's heads are spread over blocks until the GPU has four each SM
  const int64_t want = ((int64_t)sm_count() * 4 + a.T - 1) / a.T;
  const int64_t by = want < items ? want : items;
  kv4_write_kernel<D><<<dim3((unsigned)a.T, (unsigned)by), WT, 0, stream>>>(
      a, __builtin_ctz((unsigned)a.pool.page_size), -0.0f, status);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_write(const Kv4WriteArgs& a, cudaStream_t stream) {
  int* status = nullptr;
  cudaError_t e = device_status_ptr(&status);
  if (e != cudaSuccess) return e;
  if (a.pool.D == 64) return launch_write<64>(a, status, stream);
  if (a.pool.D == 128) return launch_write<128>(a, status, stream);
  return launch_write<256>(a, status, stream);
}

}  // namespace bq
