// The 4-bit cache's number formats.  A group of 16 values along a head's D
// has E2M1 codes (bias 1: 0, .5, 1, 1.5, 2, 3, 4, 6 and a sign) and one E4M3
// scale.  code * scale has at most 2 + 4 significant bits and lies in
// 2^-10 .. 2688, so it is exact in fp16 (and in bf16 and fp32).
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace mlora {

constexpr int Q4_GROUP = 16;

// Eight fp32 values to eight E2M1 codes (nearest, ties to even, saturating at
// 6), element i in bits 4i .. 4i + 3.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// One fp32 value to an E4M3 code (nearest, ties to even, saturating at 448;
// NaN gives NaN).
__device__ __forceinline__ uint32_t cvt_e4m3(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(v));
  return r & 0xFFu;
}

// The eight codes of a word as fp16 pairs (elements 2i, 2i + 1), exact.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

// Two E4M3 codes (low byte first) as an fp16 pair, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}

__device__ __forceinline__ float e4m3_to_float(uint32_t code) {
  const uint32_t p = e4m3x2_to_f16(code & 0xFFu);
  return __half2float(__ushort_as_half((unsigned short)(p & 0xFFFFu)));
}

__device__ __forceinline__ float f16_lo(uint32_t p) { return __half2float(__ushort_as_half((unsigned short)p)); }
__device__ __forceinline__ float f16_hi(uint32_t p) { return __half2float(__ushort_as_half((unsigned short)(p >> 16))); }

}  // namespace mlora
