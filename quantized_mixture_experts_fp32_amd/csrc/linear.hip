// Linear map with int4 weights: y = x W'^T (+ bias) for dense projections,
// with the codes and group scales of the experts (W' = s q, group 128).
//
// Arithmetic.  A code word becomes eight bf16 values 192 + 8 q (w4_top); the
// MFMA accumulator of every 128-group starts from -192 * sum(x over the
// group), so the group's sum is 8 sum(q x) in fp32, and the fp16 scale / 8
// (exact) weights it into the running fp32 total.  Weights are never rounded.
//
// Layout.  Lane (row r, quarter kq) of a wave reads bytes [16 kq, 16 kq + 16)
// of row r of a 16-row tile's group: one 16-byte load per lane takes the
// whole 1 KiB block.  The activations of token c sit in lanes (c, kq).
#include "launch.hpp"
#include "kcommon.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr uint32_t kOffset = 0x4340u;     // 192.0, the conversion offset
constexpr uint32_t kNegOffset = 0xC340u;  // -192.0

// One block: 16 output features of 16 tokens.  The waves take the 128-groups
// of K in turn and their totals are joined in wave order.
template <bool kOutF32>
__global__ __launch_bounds__(kThreads) void linear_w4_kernel(
    const uint16_t* __restrict__ x, const uint8_t* __restrict__ codes,
    const uint16_t* __restrict__ scales, const float* __restrict__ bias, int T, int N, int K,
    void* __restrict__ out) {
  __shared__ f32x4 red[kWaves][64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int col = lane & 15, kq = lane >> 4;
  const int n0 = blockIdx.x * 16, t = blockIdx.y * 16 + col, G = K >> 7;
  const uint8_t* cd = codes + (size_t)n0 * (K >> 1) + 64 * col + 16 * kq;
  const uint16_t* xr = x + (size_t)(t < T ? t : 0) * K + 32 * kq;
  const uint16_t* sr = scales + (size_t)(n0 + 4 * kq) * G;
  u32x4 neg;
  neg = kNegOffset | (kNegOffset << 16);
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int g = wave; g < G; g += kWaves) {
    const u32x4 q = *(const u32x4*)(cd + (size_t)1024 * g);
    f32x4 p = {0.0f, 0.0f, 0.0f, 0.0f};
    bf16x8 xf[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      xf[j] = as_bf16x8(*(const u32x4*)(xr + 128 * g + 8 * j));
      p = mfma16(as_bf16x8(neg), xf[j], p);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) p = mfma16(w4_top(q[j], kOffset | (kOffset << 16)), xf[j], p);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc[i] = fmaf(0.125f * f16_bits_to_f32(sr[(size_t)i * G + g]), p[i], acc[i]);
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (wave != 0 || t >= T) return;
#pragma unroll
  for (int w = 1; w < kWaves; ++w) acc += red[w][lane];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = n0 + 4 * kq + i;
    const float v = bias ? acc[i] + bias[n] : acc[i];
    if (kOutF32)
      ((float*)out)[(size_t)t * N + n] = v;
    else
      ((uint16_t*)out)[(size_t)t * N + n] = (uint16_t)f32_to_bf16_rne(v);
  }
}

}  // namespace

size_t linear_w4_ws_bytes(int, int, int) { return 0; }

hipError_t launch_linear_w4(const uint16_t* x, const uint8_t* codes, const uint16_t* scales,
                            const float* bias, int T, int N, int K, void* out, int out_f32,
                            void*, hipStream_t s) {
  auto kern = out_f32 ? linear_w4_kernel<true> : linear_w4_kernel<false>;
  hipLaunchKernelGGL(kern, dim3(N / 16, (T + 15) / 16), dim3(kThreads), 0, s, x, codes, scales,
                     bias, T, N, K, out);
  return hipGetLastError();
}

}  // namespace moe
