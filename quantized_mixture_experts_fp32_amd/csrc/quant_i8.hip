// Rows in 8-bit integers: activation checkpoints (a scale for each 128 values
// of a row) and the operands of the 8-bit linear map (one scale a row).
//   m = max |x| over the group, scale = m / 127, q = rne(x * (127 / m)),
//   restored as q * scale
// (fp32 divisions and one fp32 product, correctly rounded, so codes and scales
// are the same everywhere).  |x - q scale| <= scale / 2 and the roundings of
// three fp32 steps.  A group below 2^-119 is stored as zeros (127 / m stays
// finite), one with an infinity or NaN restores as NaN.
//
// HBM-bound: x is read once and the codes are written once.  8192 x 4096 (bf16):
// 22.7 us in groups (4.5 TB/s), 20.4 us by row (4.9 TB/s), restored in 18.7 us (5.4
// TB/s; a large copy: 5.1); 8192 x 4096 (fp32) 30 us (5.6 TB/s, partly from the
// last cache); 16 rows 2.9 us, a launch.
#include "i8.hpp"
#include "launch.hpp"

namespace moe {
namespace {
using namespace row;

// Sixteen lanes a group of 128, eight values each; the last group of a row may
// be shorter.
template <bool kF32>
__global__ __launch_bounds__(256) void quantize_i8_groups(const void* __restrict__ x, int K, int G,
                                                          long long groups,
                                                          int8_t* __restrict__ codes,
                                                          float* __restrict__ scales) {
  const long long i = (long long)blockIdx.x * 16 + (threadIdx.x >> 4);
  if (i >= groups) return;
  const int l = threadIdx.x & 15;
  const uint32_t row = (uint32_t)i / (uint32_t)G, g = (uint32_t)i - row * (uint32_t)G;
  const int at = (int)g * 128 + 8 * l;
  const size_t p = (size_t)row * K + at;
  f32x8 v = 0.0f;
  if (at < K) v = load8<kF32>(x, p);
  uint32_t m = top8(v);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 16));
  const Scaling s(m);
  if (at < K) *(u32x2*)(codes + p) = codes8(v, s.inv);
  if (l == 0) scales[i] = s.scale;
}

// A row by W waves, which hold it in registers (kNC chunks of eight a lane), or
// read it twice (kNC = 0); blocks of four waves.
template <bool kF32, int kNC, int W>
__global__ __launch_bounds__(256) void quantize_i8_rows(const void* __restrict__ x, int T, int K,
                                                        int8_t* __restrict__ codes,
                                                        float* __restrict__ scales) {
  __shared__ uint32_t red[4];
  const int wave = threadIdx.x >> 6, t = blockIdx.x * (4 / W) + wave / W;
  const int first = threadIdx.x % (64 * W), nch = K >> 3;
  if (t >= T) return;  // (a whole row's waves, and with W = 4 none)
  const size_t base = (size_t)t * K;
  f32x8 v[kNC > 0 ? kNC : 1];
  uint32_t m = 0;
  if (kNC > 0) {
#pragma unroll
    for (int i = 0; i < kNC; ++i) {
      const int c = first + 64 * W * i;
      v[i] = 0.0f;
      if (c < nch) v[i] = load8<kF32>(x, base + 8 * c);
    }
#pragma unroll
    for (int i = 0; i < kNC; ++i) m = max(m, top8(v[i]));
  } else {
    for (int c = first; c < nch; c += 64 * W) m = max(m, top8(load8<kF32>(x, base + 8 * c)));
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, kWave));
  if (W > 1) {
    if ((threadIdx.x & 63) == 0) red[wave] = m;
    __syncthreads();
    m = max(max(red[0], red[1]), max(red[2], red[3]));
  }
  const Scaling s(m);
  if (kNC > 0) {
#pragma unroll
    for (int i = 0; i < kNC; ++i) {
      const int c = first + 64 * W * i;
      if (c < nch) *(u32x2*)(codes + base + 8 * c) = codes8(v[i], s.inv);
    }
  } else {
    for (int c = first; c < nch; c += 64 * W)
      *(u32x2*)(codes + base + 8 * c) = codes8(load8<kF32>(x, base + 8 * c), s.inv);
  }
  if (first == 0) scales[t] = s.scale;
}

// Codes back to values, eight a thread; G groups a row (128 each, or one).
template <bool kF32>
__global__ __launch_bounds__(256) void dequantize_i8(const int8_t* __restrict__ codes,
                                                     const float* __restrict__ scales, int nch,
                                                     int G, long long chunks,
                                                     void* __restrict__ out) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= chunks) return;
  const uint32_t row = (uint32_t)i / (uint32_t)nch, c = (uint32_t)i - row * (uint32_t)nch;
  const float s = scales[(size_t)row * G + (G == 1 ? 0 : c >> 4)];
  store8<kF32>(out, 8 * (size_t)i, i8x8_to_f32(*(const u32x2*)(codes + 8 * (size_t)i)) * s);
}

// Checkpoint rows as the gated block's gradient multiplies them (launch_unpack_i8); a
// block takes a group of 16 rows, so that their units are stored together.  A code has
// seven bits: its product with a power of two is exact in bf16.  HBM-bound, two bf16
// arrays from one of codes: 4093 x 2048 11.9 us, 3.5 TB/s (the rounded one alone 7.5).
__global__ __launch_bounds__(256) void unpack_i8(const int8_t* __restrict__ codes,
                                                 const float* __restrict__ scales, int T, int K,
                                                 int G, uint16_t* __restrict__ whole,
                                                 float* __restrict__ unit,
                                                 uint16_t* __restrict__ restored) {
  const int g = blockIdx.x % G, row = blockIdx.x / G * 16 + (threadIdx.x >> 4);
  const int l = threadIdx.x & 15, at = g * 128 + 8 * l;
  if (row >= T || at >= K) return;
  const size_t p = (size_t)row * K + at;
  const float s = scales[(size_t)row * G + g];
  const f32x8 q = i8x8_to_f32(*(const u32x2*)(codes + p));
  if (whole) {
    // s = m 2^e with m in [0.5, 1); a scale of 0 (its codes are zeros) has unit 1, and
    // NaN stays in the unit
    const int e = __builtin_amdgcn_frexp_expf(s) - 1;
    store8<false>(whole, p, q * __builtin_ldexpf(1.0f, e));
    if (l == 0)
      unit[(size_t)g * T + row] = s == 0.0f ? 1.0f : 2.0f * __builtin_amdgcn_frexp_mantf(s);
  }
  if (restored) store8<false>(restored, p, q * s);
}

}  // namespace

hipError_t launch_unpack_i8(const int8_t* codes, const float* scales, int T, int K,
                            uint16_t* whole, float* unit, uint16_t* restored, hipStream_t s) {
  const int G = (K + 127) / 128;
  hipLaunchKernelGGL(unpack_i8, dim3((uint32_t)(((long long)T + 15) / 16 * G)), dim3(256), 0, s,
                     codes, scales, T, K, G, whole, unit, restored);
  return hipGetLastError();
}

hipError_t launch_quantize_i8(const void* x, int x_f32, int T, int K, int by_row, int8_t* codes,
                              float* scales, hipStream_t s) {
  if (!by_row) {
    const int G = (K + 127) / 128;
    const long long groups = (long long)T * G;
    auto k = x_f32 ? quantize_i8_groups<true> : quantize_i8_groups<false>;
    hipLaunchKernelGGL(k, dim3((uint32_t)((groups + 15) / 16)), dim3(256), 0, s, x, K, G, groups,
                       codes, scales);
    return hipGetLastError();
  }
  auto go = [&](auto nc, auto w) {
    constexpr int NC = decltype(nc)::value, W = decltype(w)::value;
    auto k = x_f32 ? quantize_i8_rows<true, NC, W> : quantize_i8_rows<false, NC, W>;
    hipLaunchKernelGGL(k, dim3((T + 4 / W - 1) / (4 / W)), dim3(256), 0, s, x, T, K, codes,
                       scales);
  };
  using std::integral_constant;
  // A wave a row up to 1024 values: no barrier, and short rows leave no lanes idle
  // (5597 x 336 4.2 us, four waves 6.0; 8192 x 1024 8.3 and 10.0); four waves for
  // longer ones (8192 x 2048 13.0 us, one wave 15.2), which beyond 8192 values are
  // read twice (8192 x 16384 109 us).
  constexpr integral_constant<int, 1> one{};
  constexpr integral_constant<int, 4> four{};
  if (K <= 512)
    go(one, one);
  else if (K <= 1024)
    go(integral_constant<int, 2>{}, one);
  else if (K <= 2048)
    go(one, four);
  else if (K <= 4096)
    go(integral_constant<int, 2>{}, four);
  else if (K <= 8192)
    go(four, four);
  else
    go(integral_constant<int, 0>{}, four);
  return hipGetLastError();
}

hipError_t launch_dequantize_i8(const int8_t* codes, const float* scales, int T, int K, int by_row,
                                void* out, int out_f32, hipStream_t s) {
  const int nch = K >> 3, G = by_row ? 1 : (K + 127) / 128;
  const long long chunks = (long long)T * nch;
  auto k = out_f32 ? dequantize_i8<true> : dequantize_i8<false>;
  hipLaunchKernelGGL(k, dim3((uint32_t)((chunks + 255) / 256)), dim3(256), 0, s, codes, scales,
                     nch, G, chunks, out);
  return hipGetLastError();
}

static size_t round_up(size_t n) { return (n + 255) & ~(size_t)255; }

size_t linear_i8_ws_bytes(int T, int N, int K, int x_bf16) {
  if (!x_bf16 || product_i8_quantizes(T, N, K)) return 0;
  return round_up((size_t)T * K) + round_up(4 * (size_t)T);
}

hipError_t launch_linear_i8(const void* x, const float* x_scales, int T, int N, int K,
                            const int8_t* codes, const float* scales, const float* bias, void* out,
                            int out_f32, void* ws, hipStream_t s) {
  if (!x_scales && !product_i8_quantizes(T, N, K)) {
    int8_t* q = (int8_t*)ws;
    float* sx = (float*)((char*)ws + round_up((size_t)T * K));
    const hipError_t e = launch_quantize_i8(x, 0, T, K, 1, q, sx, s);
    if (e != hipSuccess) return e;
    x = q;
    x_scales = sx;
  }
  return launch_product_i8(x, x_scales, T, N, K, codes, scales, bias, out, out_f32, s);
}

}  // namespace moe
