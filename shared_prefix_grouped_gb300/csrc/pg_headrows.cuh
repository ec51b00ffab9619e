// Rows of one head of one token (head_dim elements) handled by part of a warp: D / 8 lanes per row, so
// a warp takes 2 rows (D = 128) or 4 (D = 64) at a time.  Lane l of a row holds elements
// [4 l, 4 l + 4) and [D/2 + 4 l, D/2 + 4 l + 4): both ends of its four rotate-half pairs, so the
// rotation needs no exchange between lanes, and each half of a row is one contiguous piece per load.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pg_internal.h"

namespace pg {
namespace headrows {

__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&v)[4]) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
  const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  uint2 u;
  u.x = *reinterpret_cast<const uint32_t*>(&a);
  u.y = *reinterpret_cast<const uint32_t*>(&b);
  *reinterpret_cast<uint2*>(p) = u;
}

// Four elements as they are in memory: rows wait for their turn in half the registers (bf16).
template <typename T>
struct Raw4;
template <>
struct Raw4<float> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void get(float (&x)[4]) const {
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  }
};
template <>
struct Raw4<__nv_bfloat16> {
  uint2 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    v = *reinterpret_cast<const uint2*>(p);
  }
  __device__ __forceinline__ void get(float (&x)[4]) const {
    x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xffff0000u);
  }
};
template <typename T, int D>
struct RawRow {
  Raw4<T> lo, hi;
  __device__ __forceinline__ void load(const T* row, int l) {
    lo.load(row + 4 * l);
    hi.load(row + D / 2 + 4 * l);
  }
};

// One row's share of a lane: the low and the high ends of its four pairs.
template <typename T, int D>
struct Row {
  float lo[4], hi[4];
  __device__ __forceinline__ void load(const T* row, int l) {
    load4(row + 4 * l, lo);
    load4(row + D / 2 + 4 * l, hi);
  }
  __device__ __forceinline__ void from(const RawRow<T, D>& r) {
    r.lo.get(lo);
    r.hi.get(hi);
  }
  __device__ __forceinline__ void store(T* row, int l) const {
    store4(row + 4 * l, lo);
    store4(row + D / 2 + 4 * l, hi);
  }
  __device__ __forceinline__ void rotate(const float (&c)[4], const float (&s)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = lo[e], b = hi[e];
      lo[e] = a * c[e] - b * s[e];
      hi[e] = b * c[e] + a * s[e];
    }
  }
};

// Sum over the D / 8 lanes of a row (every lane of the warp takes part).
template <int D>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The cosines and sines of a lane's four angles at a position that the whole warp shares.  Lanes with the
// same elements of different rows need the same angles: each computes its part of the four and passes it
// on.  position x (frequency / 2 pi) modulo one turn is exact in 0.64 fixed point, its upper 32 bits read
// as signed give the angle in half turns, [-1, 1).
template <int D>
struct Angles {
  static constexpr int kLanes = D / 8, kOwn = 4 * kLanes / 32;
  uint64_t turn[kOwn];
  __device__ __forceinline__ void init(const uint64_t* turns, int lane) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) turn[i] = turns[4 * (lane % kLanes) + lane / kLanes * kOwn + i];
  }
  // Every lane of the warp takes part.
  __device__ __forceinline__ void at(int32_t pos, int lane, float (&c)[4], float (&s)[4]) const {
    float own_c[kOwn], own_s[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const uint64_t t = (uint64_t)(int64_t)pos * turn[i];
      sincospif((float)(int32_t)(uint32_t)(t >> 32) * 0x1p-31f, &own_s[i], &own_c[i]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int from = e / kOwn * kLanes + lane % kLanes;
      c[e] = __shfl_sync(0xffffffffu, own_c[e % kOwn], from);
      s[e] = __shfl_sync(0xffffffffu, own_s[e % kOwn], from);
    }
  }
};

}  // namespace headrows
}  // namespace pg
