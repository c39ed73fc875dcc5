// Values in 8-bit integers, on the device: the scale of a group and its codes
// (quant_i8.hip has the definition).
#pragma once
#include "rowops.hpp"

namespace moe {
using row::f32x8;

__device__ __forceinline__ f32x8 bf16x8_to_f32(u32x4 v) {
  row::Raw8<false> r;
  r.a = v;
  return r.get();
}

constexpr uint32_t kInfBits = 0x7F800000u;
constexpr float kTiny = 0x1p-119f;

// Largest magnitude of eight values as bits, which order as the values do, an
// infinity above all numbers and NaN above it.
__device__ __forceinline__ uint32_t top8(const f32x8 v) {
  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) m = max(m, __float_as_uint(v[q]) & 0x7FFFFFFFu);
  return m;
}

struct Scaling {
  float scale, inv;  // inv 0: every code is 0
  __device__ __forceinline__ explicit Scaling(uint32_t top) {
    const float m = __uint_as_float(top);
    const bool bad = top >= kInfBits, zero = m < kTiny;
    scale = bad ? __uint_as_float(0x7FC00000u) : zero ? 0.0f : m / 127.0f;
    inv = bad || zero ? 0.0f : 127.0f / m;
  }
};

__device__ __forceinline__ u32x2 codes8(const f32x8 v, float inv) {
  u32x2 r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      // (a product with inv 0 may be NaN; it is not used)
      const int c = inv == 0.0f ? 0 : (int)__builtin_rintf(v[4 * h + q] * inv);
      w |= (uint32_t)(c & 255) << (8 * q);
    }
    r[h] = w;
  }
  return r;
}

}  // namespace moe
