// The 4-bit cache's numbers: a value is an e2m1 code (0, 0.5, 1, 1.5, 2, 3, 4, 6
// and their negatives) times the e4m3 scale of its group of 16 elements along
// the head dimension, times the caller's gain.  Code and scale have 2 and 4
// significant bits, so their product is exact in float16 (largest 2688,
// smallest 2^-10).
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace sv {

constexpr int kFp4Group = 16;
constexpr uint32_t kFp4NanScale = 0x7f;   // of a group with a NaN or an infinity

// Four bytes of codes as four pairs of float16, the byte's low half first.
__device__ __forceinline__ void fp4_unpack(uint32_t w, uint32_t* r) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
// Eight values, rounded to the nearest code (ties to the even one, saturating).
__device__ __forceinline__ uint32_t fp4_pack(const float* x) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return w;
}
// Two bytes of scales as a pair of float16.
__device__ __forceinline__ uint32_t fp4_scales(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(two));
  return r;
}
__device__ __forceinline__ uint32_t fp4_scale_code(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r;
}
__device__ __forceinline__ float fp4_scale(uint32_t code) {
  const uint32_t pair = fp4_scales(code);
  return __low2float(*(const __half2*)&pair);
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace sv
