// Conversions between e4m3 and wider numbers (four significant bits, 2^-9 to 448),
// two or more at a time.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace cb {

// The low (high) two bytes of x as a pair of f16: exact, the lower byte first.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_hi_to_f16x2(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void f16x2_to_float(uint32_t x, float& lo, float& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}" : "=f"(lo), "=f"(hi) : "r"(x));
}
// Four bytes as floats.
__device__ __forceinline__ void e4m3x4_to_float(uint32_t x, float (&f)[4]) {
  f16x2_to_float(e4m3x2_to_f16x2(x), f[0], f[1]);
  f16x2_to_float(e4m3x2_hi_to_f16x2(x), f[2], f[3]);
}
// Four floats to the nearest e4m3 numbers, ties to even; beyond 448 to 448, NaN stays.
__device__ __forceinline__ uint32_t float_to_e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

}  // namespace cb
