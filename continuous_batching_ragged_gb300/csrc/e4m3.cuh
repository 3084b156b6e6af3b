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

// y, off from an exact value of its sign by `rest` (whose sign counts) and by less than one step: the value cut off towards zero, its
// last bit set where bits were cut off.  Rounded to fewer bits after that, it is rounded once.  NaN stays.
__device__ __forceinline__ float to_odd(float y, float rest) {
  uint32_t u = __float_as_uint(y);
  if (!(rest == 0.f)) u = (u - ((u ^ __float_as_uint(rest)) >> 31)) | 1u;
  return __uint_as_float(u);
}
// The same of a product of numbers with up to 4 and 24 bits, if it is 2^-100 or more.
__device__ __forceinline__ float product_to_odd(float x, float s) {
  const float y = __fmul_rz(x, s);
  return fmaf(x, s, -y) == 0.f ? y : __uint_as_float(__float_as_uint(y) | 1u);
}
__device__ __forceinline__ bool is_power_of_two(float x) { return (__float_as_uint(x) & 0x7fffffu) == 0; }   // of positive ones that are not denormal

}  // namespace cb
