// e4m3.cuh -- E4M3 codes under E8M0 scales: what the FP8 linear layer, the key/value cache and the attention
// over it share.
#pragma once

#include "sb_device.cuh"

namespace sb {

// Exponent byte of a block with largest magnitude a, given as bf16 bits: the smallest e with
// a <= 448 * 2^e (448 = 1.75 * 2^8), plus 127; a is 1.m * 2^(field - 127). Subnormal and zero a
// give 0.
__device__ __forceinline__ uint32_t e8m0_of_amax(uint32_t bits) {
  const int b = (int)(bits >> 7) - 8 + ((bits & 0x7fu) > 0x60u ? 1 : 0);
  return (uint32_t)max(b, 0);
}

__device__ __forceinline__ float pow2_byte(int byte) {  // 2^(byte - 127)
  return byte <= 0 ? 0x1p-127f : __uint_as_float((uint32_t)byte << 23);
}

// 2^-e for an exponent byte e + 127 (byte <= 253, which every finite bf16 amax gives).
__device__ __forceinline__ float e8m0_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

__device__ __forceinline__ uint32_t cvt_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// E4M3 pairs -> fp16 pairs, exact.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t b) {
  uint32_t h;
  const uint16_t in = (uint16_t)b;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(in));
  return h;
}

// 16 x 8 += (16 x 16) (16 x 8), fp16 with FP32 sums.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

}  // namespace sb
