// Device helpers of the row kernels (norms, combine with residual, token
// sort): a row of d values is held in registers by one block, eight
// consecutive values (a chunk) at a time.
#pragma once
#include "kcommon.hpp"

namespace moe {
namespace row {

typedef float f32x8 __attribute__((ext_vector_type(8)));

// Eight consecutive values of a bf16 or fp32 row, as fp32.
template <bool kF32>
__device__ __forceinline__ f32x8 load8(const void* p, size_t i) {
  f32x8 v;
  if (kF32) {
    const f32x4 a = *(const f32x4*)((const float*)p + i);
    const f32x4 b = *(const f32x4*)((const float*)p + i + 4);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[q] = a[q];
      v[4 + q] = b[q];
    }
  } else {
    const u32x4 a = *(const u32x4*)((const uint16_t*)p + i);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = __uint_as_float(a[q] << 16);
      v[2 * q + 1] = __uint_as_float(a[q] & 0xFFFF0000u);
    }
  }
  return v;
}

// Stored as fp32, or as bf16 (round to nearest even).
template <bool kF32>
__device__ __forceinline__ void store8(void* p, size_t i, const f32x8 v) {
  if (kF32) {
    *(f32x4*)((float*)p + i) = f32x4{v[0], v[1], v[2], v[3]};
    *(f32x4*)((float*)p + i + 4) = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    u32x4 a;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      a[q] = f32_to_bf16_rne(v[2 * q]) | (f32_to_bf16_rne(v[2 * q + 1]) << 16);
    *(u32x4*)((uint16_t*)p + i) = a;
  }
}

__device__ __forceinline__ float sum8(const f32x8 a, const f32x8 b) {
  float s = a[0] * b[0];
#pragma unroll
  for (int q = 1; q < 8; ++q) s = fmaf(a[q], b[q], s);
  return s;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

// Sums of N values over the block's kW waves, in a fixed order; every thread
// gets them.  red: N * kW floats of LDS that the previous call with the same
// array has been read from on the far side of another barrier.
template <int N, int kW>
__device__ __forceinline__ void block_sum(float (&v)[N], float* red) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if (kW == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[i * kW + wave] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float s = red[i * kW];
#pragma unroll
    for (int w = 1; w < kW; ++w) s += red[i * kW + w];
    v[i] = s;
  }
}

}  // namespace row
}  // namespace moe
