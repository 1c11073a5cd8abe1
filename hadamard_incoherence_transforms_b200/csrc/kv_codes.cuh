// Stored codes to fp16 matrix operands, in registers and without an error.
#pragma once
#include <stdint.h>

namespace hit {

__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t m, uint32_t o) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(m), "r"(o));
  return r;
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// Eight 4-bit codes -> (0, 4), (1, 5), (2, 6), (3, 7) as fp16 pairs: 0x6400 | u
// is 1024 + u, and 1024 + 16 u for the upper nibble of a byte.
__device__ __forceinline__ void half_of4(uint32_t w, uint32_t (&h)[4]) {
  const uint32_t v = w >> 8;
  h[0] = hadd2(and_or(w, 0x000f000fu, 0x64006400u), 0xe408e408u);               // - 1032
  h[1] = hfma2(and_or(w, 0x00f000f0u, 0x64006400u), 0x2c002c00u, 0xd480d480u);  // / 16 - 72
  h[2] = hadd2(and_or(v, 0x000f000fu, 0x64006400u), 0xe408e408u);
  h[3] = hfma2(and_or(v, 0x00f000f0u, 0x64006400u), 0x2c002c00u, 0xd480d480u);
}
// Four 8-bit codes -> (0, 1), (2, 3) as fp16 pairs.
__device__ __forceinline__ void half_of8(uint32_t w, uint32_t& a, uint32_t& b) {
  a = hadd2(__byte_perm(w, 0x64646464u, 0x4140), 0xe480e480u);  // 1024 + u - 1152
  b = hadd2(__byte_perm(w, 0x64646464u, 0x4342), 0xe480e480u);
}
// x: two runs of 16 bits of codes -> (code n of the low run, code n of the high one).
__device__ __forceinline__ void half_runs4(uint32_t x, uint32_t (&b)[4]) {
#pragma unroll
  for (int n = 0; n < 4; ++n) b[n] = hadd2(and_or(x >> (4 * n), 0x000f000fu, 0x64006400u), 0xe408e408u);  // 1024 + u - 1032
}
__device__ __forceinline__ void half_runs8(uint32_t x, uint32_t& b0, uint32_t& b1) {
  b0 = hadd2(and_or(x, 0x00ff00ffu, 0x64006400u), 0xe480e480u);  // 1024 + u - 1152
  b1 = hadd2(and_or(x >> 8, 0x00ff00ffu, 0x64006400u), 0xe480e480u);
}

// d += A B for 16 x 8 x 16, fp16 operands.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
}  // namespace hit
