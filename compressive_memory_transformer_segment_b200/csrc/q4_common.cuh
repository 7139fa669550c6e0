// Shared device code of the kernels that read 4-bit codes: code words to
// bf16 pairs, and the warp's matrix product on them.
//
// A code q in 0..15 becomes a bf16 by bit insertion: 0x4300 | q is 128 + q
// (the 7 mantissa bits of 128 step by 1), and subtracting 128 + zero in bf16
// gives the integer q - zero exactly.  Products of such integers with a bf16
// operand are exact in the fp32 accumulator, so the only roundings of a
// product over a group are the accumulator's own.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "common.cuh"

namespace infini {

constexpr uint32_t kCodeBias2 = 0x43004300u;  // bf16x2 (128, 128)

// The four bf16 pairs of a word of 8 codes: pair p holds the codes of bits
// 4p.. and 4p + 16.., each minus the value that `bias` (bf16x2 of 128 + zero)
// says.
__device__ __forceinline__ void unpack_codes(uint32_t w, uint32_t bias, uint32_t (&out)[4]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const uint32_t t = ((w >> (4 * p)) & 0x000f000fu) | kCodeBias2;
    const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&t),
                                     *reinterpret_cast<const __nv_bfloat162*>(&bias));
    out[p] = *reinterpret_cast<const uint32_t*>(&v);
  }
}

// bf16x2 of (lo, hi), and what it leaves of them: lo and hi become the
// rounding errors.  Three such steps hold all 24 bits of an fp32 (down to 2^-133, bf16's
// least value).  Saturated: fp32's largest values would round to infinity.
__device__ __forceinline__ uint32_t split_bf16(float& lo, float& hi) {
  uint32_t v;
  asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(hi), "f"(lo));
  lo -= __uint_as_float(v << 16);
  hi -= __uint_as_float(v & 0xffff0000u);
  return v;
}

// c += a b: a 16 x 16 (rows x k), b 16 x 8 (k x columns), bf16 with fp32
// accumulation.  Lane 4 i + t holds a rows i (a0, a2) and i + 8 (a1, a3) at k
// 2t, 2t + 1 (a0, a1) and 2t + 8, 2t + 9 (a2, a3), b column i at the same k,
// and c rows i (c0, c1) and i + 8 (c2, c3) at columns 2t, 2t + 1.
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same product alone: c = a b.
__device__ __forceinline__ void mma_bf16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// 2^x by the hardware approximation (relative error 2^-22; 0 below 2^-126).
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Loads of data that passes through once (kept out of L1).
__device__ __forceinline__ uint4 ld_once_16(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

}  // namespace infini
