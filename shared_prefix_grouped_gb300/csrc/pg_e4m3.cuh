// e4m3 codes, four to a 32-bit word, lowest address first, and the scales of blocks of them.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace pg {
namespace e4m3 {

// The least power of two 2^e, e >= -126, with amax <= 448 * 2^e (448 = 1.75 * 2^8).
__device__ __forceinline__ float block_scale(float amax) {
  const int b = __float_as_int(amax);
  const int e = (b >> 23) - ((b & 0x7fffff) <= 0x600000 ? 8 : 7);
  return __int_as_float(max(e, 1) << 23);
}
// 2^-e of a scale 2^e, -126 <= e <= 120.
__device__ __forceinline__ float inverse_scale(float s) {
  return __int_as_float((254 << 23) - __float_as_int(s));
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;
}

// Four values as codes, lowest address first (NaN stays one, an infinity becomes 448).
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n"
      " cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n mov.b32 %0, {l, h};\n}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
// Four values times inv as codes; what is not finite becomes NaN.
__device__ __forceinline__ uint32_t encode4(const float (&x)[4], float inv) {
  return pack4(fmaf(x[0], inv, x[0] * 0.f), fmaf(x[1], inv, x[1] * 0.f), fmaf(x[2], inv, x[2] * 0.f),
               fmaf(x[3], inv, x[3] * 0.f));
}
// The same without infinities among them.
__device__ __forceinline__ uint32_t encode4_finite(const float (&x)[4], float inv) {
  return pack4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
}
__device__ __forceinline__ void decode4(uint32_t c, float (&x)[4]) {
  uint32_t a, b;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(a) : "h"((uint16_t)(c & 0xffffu)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"((uint16_t)(c >> 16)));
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}"
      : "=f"(x[0]), "=f"(x[1]) : "r"(a));
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}"
      : "=f"(x[2]), "=f"(x[3]) : "r"(b));
}

}  // namespace e4m3
}  // namespace pg
