// Device helpers of the row kernels (norms, combine with residual, token
// sort): a row of d values is held in registers by one block, eight
// consecutive values (a chunk) at a time.
#pragma once
#include <type_traits>

#include "kcommon.hpp"

namespace moe {
namespace row {

typedef float f32x8 __attribute__((ext_vector_type(8)));

// Eight consecutive values of a bf16 or fp32 row, as loaded and as fp32.
template <bool kF32>
struct Raw8 {
  u32x4 a, b;
  __device__ __forceinline__ void load(const void* p, size_t i) {
    if (kF32) {
      a = *(const u32x4*)((const float*)p + i);
      b = *(const u32x4*)((const float*)p + i + 4);
    } else {
      a = *(const u32x4*)((const uint16_t*)p + i);
    }
  }
  // mask 0: zeros, whatever was loaded
  __device__ __forceinline__ f32x8 get(uint32_t mask = ~0u) const {
    f32x8 v;
    if (kF32) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[q] = __uint_as_float(a[q] & mask);
        v[4 + q] = __uint_as_float(b[q] & mask);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[2 * q] = __uint_as_float((a[q] & mask) << 16);
        v[2 * q + 1] = __uint_as_float(a[q] & mask & 0xFFFF0000u);
      }
    }
    return v;
  }
};

template <bool kF32>
__device__ __forceinline__ f32x8 load8(const void* p, size_t i) {
  Raw8<kF32> r;
  r.load(p, i);
  return r.get();
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

// Eight 8-bit codes as fp32.
__device__ __forceinline__ f32x8 i8x8_to_f32(u32x2 w) {
  f32x8 v;
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q] = (float)((int)(w[q >> 2] << (24 - 8 * (q & 3))) >> 24);
  return v;
}

// What a row is stored as: its values, or 8-bit codes with a scale for each 128
// (a chunk's codes and its group's scale; restored as quant_i8.hip says).
enum RowKind { kRowBf16, kRowF32, kRowI8 };

template <int kKind>
struct RowChunk {
  Raw8<kKind == kRowF32> r;
  __device__ __forceinline__ void load(const void* p, const float*, size_t row, int d, int at) {
    r.load(p, row * d + at);
  }
  __device__ __forceinline__ f32x8 get() const { return r.get(); }
};
template <>
struct RowChunk<kRowI8> {
  u32x2 q;
  float s;
  __device__ __forceinline__ void load(const void* p, const float* scales, size_t row, int d,
                                       int at) {
    q = *(const u32x2*)((const int8_t*)p + row * d + at);
    s = scales[row * ((d + 127) >> 7) + (at >> 7)];
  }
  __device__ __forceinline__ f32x8 get() const { return i8x8_to_f32(q) * s; }
};

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

// The k <= KM pairs of one token.  A dropped pair (slot outside [0, P)) has
// weight 0, mask 0 and slot 0, so that the rows of all pairs can be asked for
// without a branch on the routing between the loads; the mask keeps what the
// dropped pair's load returned out of every sum.
template <int KM>
struct Pairs {
  int slot[KM > 0 ? KM : 1];
  uint32_t mask[KM > 0 ? KM : 1];
  float w[KM > 0 ? KM : 1];
  __device__ __forceinline__ void load(const int32_t* pair_pos, const float* topk_w, int P, int k,
                                       int t) {
#pragma unroll
    for (int j = 0; j < KM; ++j) {
      slot[j] = 0;
      mask[j] = 0;
      w[j] = 0.0f;
      if (j < k) {
        const int s = pair_pos[(size_t)t * k + j];
        const float f = topk_w ? topk_w[(size_t)t * k + j] : 1.0f;
        const bool live = (unsigned)s < (unsigned)P;
        slot[j] = live ? s : 0;
        mask[j] = live ? ~0u : 0u;
        w[j] = live ? f : 0.0f;
      }
    }
  }
};

// Threads of a row's block and the chunks each holds: 256 threads while two
// chunks each hold the row, then 512; a batch of no more rows than CUs, where
// only latency counts, takes 512 from one chunk on.
constexpr int kWideRows = 256;
template <typename F>
inline void with_shape(int T, int d, F&& f) {
  using std::integral_constant;
  const int nch = d >> 3;
  if (nch <= 256)
    f(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  else if (nch <= 512 && T > kWideRows)
    f(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  else if (nch <= 512)
    f(integral_constant<int, 512>{}, integral_constant<int, 1>{});
  else
    f(integral_constant<int, 512>{}, integral_constant<int, 2>{});
}

// Calls f with the smallest of the kernels' pair counts that holds k.
template <typename F>
inline void with_pairs(int k, F&& f) {
  if (k == 0)
    f(std::integral_constant<int, 0>{});
  else if (k <= 2)
    f(std::integral_constant<int, 2>{});
  else if (k <= 4)
    f(std::integral_constant<int, 4>{});
  else if (k <= 8)
    f(std::integral_constant<int, 8>{});
  else
    f(std::integral_constant<int, 16>{});
}

}  // namespace row
}  // namespace moe
