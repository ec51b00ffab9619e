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

// Four values times inv as codes, lowest address first; what is not finite becomes NaN.
__device__ __forceinline__ uint32_t encode4(const float (&x)[4], float inv) {
  float y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = fmaf(x[e], inv, x[e] * 0.f);
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y[1]), "f"(y[0]));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y[3]), "f"(y[2]));
  return (uint32_t)lo | (uint32_t)hi << 16;
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
