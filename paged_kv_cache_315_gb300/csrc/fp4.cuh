// fp4.cuh -- E2M1 codes (1 sign, 2 exponent bits with bias 1, 1 fraction bit; magnitudes
// 0, 0.5, 1, 1.5, 2, 3, 4, 6) to and from wider types.  sm_103a only.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace pkv {

// The code of `lo` in bits 0-3 and of `hi` in bits 4-7: nearest, ties to the even code,
// magnitudes beyond 6 saturate.
__device__ __forceinline__ uint32_t f32x2_to_e2m1x2(float lo, float hi) {
  uint32_t out;
  asm("{\n\t.reg .b8 c;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %2, %1;\n\t"
      "cvt.u32.u8 %0, c;\n\t}"
      : "=r"(out)
      : "f"(lo), "f"(hi));
  return out;
}

// Eight codes (element 0 in the lowest four bits) -> four fp16 pairs (lower element in the
// low half).  Exact.
__device__ __forceinline__ void e2m1x8_to_f16x2x4(uint32_t codes, uint32_t (&out)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3])
      : "r"(codes));
}

// Eight codes times `scale`.
__device__ __forceinline__ void decode8(uint32_t codes, float scale, float (&x)[8]) {
  uint32_t h[4];
  e2m1x8_to_f16x2x4(codes, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h[i]));
    x[2 * i] = f.x * scale;
    x[2 * i + 1] = f.y * scale;
  }
}

// Two E4M3 codes (`lo` in the low byte) of fp16 or fp32 pairs: nearest, ties to even,
// magnitudes beyond 448 saturate, NaN stays NaN.
__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(uint32_t pair) {
  uint16_t out;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(out) : "r"(pair));
  return out;
}

__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t out;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(out) : "f"(hi), "f"(lo));
  return out;
}

}  // namespace pkv
