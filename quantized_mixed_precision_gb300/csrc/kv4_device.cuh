// Device helpers of the 4-bit cache kernels: mma.sync, movmatrix, the base-2
// exponential, and the meaning of 4-bit codes as fp16 subnormals.
//
// A masked word w & 0x000f000f holds two codes u in the low bits of two fp16
// fields, i.e. the fp16 subnormals u * 2**-24, exactly; w & 0x00f000f0 holds
// u * 2**-20.  Tensor cores take subnormals as they are, so one LOP3 turns two
// codes into an exact MMA operand, with no arithmetic; the factor 2**24 (or
// 2**20) returns in the fp32 scale that follows the sum.
#pragma once

#include <cuda_fp16.h>

#include "bq_device.cuh"

namespace bq {

constexpr uint32_t CODE_LO = 0x000f000fu;   // codes worth u * 2**-24
constexpr uint32_t CODE_HI = 0x00f000f0u;   // codes worth u * 2**-20

// D (16 x 8, fp32) += A (16 x 16) * B (16 x 8), fp16.  With g = lane / 4 and
// t = lane % 4: a0, a1 hold rows g, g + 8 at k = 2t, 2t + 1, a2, a3 the same
// rows at k + 8; b0, b1 hold k = 2t, 2t + 1 (+ 8) of column g; d holds
// columns 2t, 2t + 1 of rows g and g + 8.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D = A * B with a zero C.
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// Transpose of an 8 x 8 matrix of 16-bit values, one row pair per register.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// 2**x (2 ulp; exact 0 at -inf)
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float2 unpack_h2(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// 2**e as fp32, for e in [-126, 127]
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

// floor(log2(|x|)) of a positive normal fp32 number
__device__ __forceinline__ int ilog2f(float x) { return ((__float_as_int(x) >> 23) & 255) - 127; }

// Two 16 x 16 byte matrices, transposed: lanes 0..15 give the rows of the
// first, lanes 16..31 those of the second (16 bytes each); r[2 i] and r[2 i + 1]
// hold rows 4t .. 4t + 3 of columns g and g + 8 of matrix i.
__device__ __forceinline__ void ldmatrix_b8_trans_x2(uint32_t saddr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(saddr)
               : "memory");
}

// Packed fp32 arithmetic: each lane of an operation is an ordinary IEEE one.
struct P2 {               // two fp32 values in one 64-bit register
  uint64_t v;
};
__device__ __forceinline__ P2 p2(float a, float b) {
  P2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 f2(P2 p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p.v));
  return r;
}
__device__ __forceinline__ P2 mul2(P2 a, P2 b) {
  P2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ P2 add2(P2 a, P2 b) {
  P2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ P2 fma2(P2 a, P2 b, P2 c) {
  P2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
// Two fp16 values times the fp16 constant c (its bits) added to two fp32 sums
__device__ __forceinline__ P2 fma_h2(uint32_t h, uint16_t c, P2 sum) {
  float2 v = f2(sum);
  asm("{\n\t.reg .f16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "fma.rn.f32.f16 %0, lo, %3, %0;\n\t"
      "fma.rn.f32.f16 %1, hi, %3, %1;\n\t}"
      : "+f"(v.x), "+f"(v.y)
      : "r"(h), "h"(c));
  return p2(v.x, v.y);
}

// Sum of 8 fp16 values in fp32
__device__ __forceinline__ float sum_h8(const uint4& v) {
  float a = 0.0f, b = 0.0f;
  asm("{\n\t.reg .f16 l0, h0, l1, h1, l2, h2, l3, h3;\n\t"
      "mov.b32 {l0, h0}, %2;\n\tmov.b32 {l1, h1}, %3;\n\tmov.b32 {l2, h2}, %4;\n\tmov.b32 {l3, h3}, %5;\n\t"
      "add.rn.f32.f16 %0, l0, %0;\n\tadd.rn.f32.f16 %1, h0, %1;\n\t"
      "add.rn.f32.f16 %0, l1, %0;\n\tadd.rn.f32.f16 %1, h1, %1;\n\t"
      "add.rn.f32.f16 %0, l2, %0;\n\tadd.rn.f32.f16 %1, h2, %1;\n\t"
      "add.rn.f32.f16 %0, l3, %0;\n\tadd.rn.f32.f16 %1, h3, %1;\n\t}"
      : "+f"(a), "+f"(b)
      : "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w));
  return a + b;
}

// 16-byte asynchronous copy to a shared-memory address
__device__ __forceinline__ void cp_async_16_u(uint32_t smem_dst, const void* gmem_src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_dst), "l"(gmem_src) : "memory");
}

// The same through L1, for data that many blocks read: with copies past L1 the 8 KB row of X of a GEMV, read by all 688
// blocks, cost 8 us.
__device__ __forceinline__ void cp_async_16_l1(uint32_t smem_dst, const void* gmem_src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem_dst), "l"(gmem_src) : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace bq
