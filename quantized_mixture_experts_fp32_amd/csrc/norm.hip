// The norm in front of a block, and its gradient.
//   out = x * rstd * gain,  rstd = (mean(x^2) + eps)^(-1/2)
// With u = dout * gain and h = x * rstd, the gradient is
//   dx = dres + rstd * (u - h * mean(u h)),   dgain = sum over tokens of dout * h
// (dres: the gradient that reaches x past the norm).  The backward pass has
// the row of x in registers anyway, so it computes rstd again instead of
// reading a saved one: mean(x^2) and mean(u x) are two sums of one pass.
//
// HBM-bound: every row is read once, held in registers by one block as fp32,
// and written once.  All sums are fp32 in a fixed order.  Backward, a block
// takes every 512th row, so that its share of the gain's column sums stays in
// registers, and has the next row's three arrays in flight during the sums of
// this one: 8191 rows of 4096 (bf16) take 55 us with the column sums, 4.9 TB/s,
// the rate of a large copy (76 us without the prefetch).  Forward, 8192 rows of
// 4096 (bf16) 27 us, 4.9 TB/s; 16 rows 2.5 us, a launch.
#include "launch.hpp"
#include "rowops.hpp"

namespace moe {
namespace {
using namespace row;

// Blocks of the backward pass, two a CU; their partial column sums are 512 d
// floats, 3 % of the bytes of 8192 bf16 rows.
constexpr int kBwdBlocks = 512;

template <bool kXF32, bool kOutF32, int NC, int kThreads>
__global__ __launch_bounds__(kThreads) void rmsnorm_kernel(const void* __restrict__ x,
                                                           const float* __restrict__ gain, int d,
                                                           float eps, void* __restrict__ out) {
  constexpr int kWaves = kThreads / kWave;
  __shared__ float red[kWaves];
  const size_t base = (size_t)blockIdx.x * d;
  const int nch = d >> 3;
  f32x8 v[NC], g[NC];
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = threadIdx.x + kThreads * i;
    g[i] = 1.0f;
    if (c < nch) {
      v[i] = load8<kXF32>(x, base + 8 * c);
      if (gain) g[i] = load8<true>(gain, 8 * c);
      s[0] += sum8(v[i], v[i]);
    }
  }
  block_sum<1, kWaves>(s, red);
  const float rstd = rsqrtf(s[0] / d + eps);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = threadIdx.x + kThreads * i;
    if (c < nch) store8<kOutF32>(out, base + 8 * c, v[i] * rstd * g[i]);
  }
}

template <bool kDoF32, bool kXF32, int NC, int kThreads>
__global__ __launch_bounds__(kThreads) void rmsnorm_bwd_kernel(
    const void* __restrict__ dout, const void* __restrict__ x, const float* __restrict__ gain,
    const void* dres, int T, int d, float eps, void* dx, float* __restrict__ partial) {
  constexpr int kWaves = kThreads / kWave;
  __shared__ float red[2][2 * kWaves];
  const int nch = d >> 3;
  f32x8 g[NC], acc[NC];
  int at[NC];  // the chunk's column; threads past the row read its first chunk
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = threadIdx.x + kThreads * i;
    at[i] = c < nch ? 8 * c : 0;
    acc[i] = 0.0f;
    g[i] = 1.0f;
    if (gain && c < nch) g[i] = load8<true>(gain, 8 * c);
  }
  // the next row is asked for before this one's sums (past the last row: the
  // last again, for nothing)
  Raw8<kXF32> rx[NC], rr[NC];
  Raw8<kDoF32> ru[NC];
  auto ask = [&](int t) {
    const size_t base = (size_t)min(t, T - 1) * d;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      rx[i].load(x, base + at[i]);
      ru[i].load(dout, base + at[i]);
      if (dres) rr[i].load(dres, base + at[i]);
    }
  };
  ask(blockIdx.x);
  int turn = 0;
  for (int t = blockIdx.x; t < T; t += gridDim.x, turn ^= 1) {
    const size_t base = (size_t)t * d;
    f32x8 v[NC], u[NC], r[NC];
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      v[i] = rx[i].get();
      u[i] = ru[i].get();
      r[i] = 0.0f;
      if (dres) r[i] = rr[i].get();
    }
    ask(t + gridDim.x);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if ((int)threadIdx.x + kThreads * i < nch) {
        s[0] += sum8(v[i], v[i]);
        s[1] += sum8(u[i] * g[i], v[i]);
      }
    }
    block_sum<2, kWaves>(s, red[turn]);
    const float rstd = rsqrtf(s[0] / d + eps);
    const float a = s[1] / d * rstd * rstd;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = threadIdx.x + kThreads * i;
      if (c < nch) {
        store8<kXF32>(dx, base + 8 * c, (u[i] * g[i] - v[i] * a) * rstd + r[i]);
        acc[i] += u[i] * (v[i] * rstd);
      }
    }
  }
  if (!partial) return;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = threadIdx.x + kThreads * i;
    if (c < nch) store8<true>(partial, (size_t)blockIdx.x * d + 8 * c, acc[i]);
  }
}

// S[c] = sum over n rows of rows[r][c]; out1[c] = S[c] * f1[c] and out2[c] =
// S[c] * f2[c] (a null factor is 1, a null output is skipped).  64 columns per
// block, the rows dealt to its 16 waves, which are joined in wave order.
__global__ __launch_bounds__(1024) void colsum_kernel(const float* __restrict__ rows, int n, int d,
                                                      float* __restrict__ out1,
                                                      const float* __restrict__ f1,
                                                      float* __restrict__ out2,
                                                      const float* __restrict__ f2) {
  __shared__ float red[16][64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int c = blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (c < d) {
#pragma unroll 16
    for (int r = wave; r < n; r += 16) s += rows[(size_t)r * d + c];
  }
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < d) {
#pragma unroll
    for (int w = 1; w < 16; ++w) s += red[w][lane];
    if (out1) out1[c] = f1 ? s * f1[c] : s;
    if (out2) out2[c] = f2 ? s * f2[c] : s;
  }
}

}  // namespace

hipError_t launch_colsum(const float* rows, int n, int d, float* out1, const float* f1,
                         float* out2, const float* f2, hipStream_t s) {
  hipLaunchKernelGGL(colsum_kernel, dim3((d + 63) / 64), dim3(1024), 0, s, rows, n, d, out1, f1,
                     out2, f2);
  return hipGetLastError();
}

hipError_t launch_rmsnorm(const void* x, int x_f32, const float* gain, int T, int d, float eps,
                          void* out, int out_f32, hipStream_t s) {
  with_shape(T, d, [&](auto th, auto nc) {
    with_bools(x_f32, out_f32, [&](auto xf, auto of) {
      constexpr int TH = decltype(th)::value, NC = decltype(nc)::value;
      hipLaunchKernelGGL((rmsnorm_kernel<decltype(xf)::value, decltype(of)::value, NC, TH>),
                         dim3(T), dim3(TH), 0, s, x, gain, d, eps, out);
    });
  });
  return hipGetLastError();
}

size_t rmsnorm_bwd_ws_bytes(int T, int d) {
  return (size_t)(T < kBwdBlocks ? T : kBwdBlocks) * d * sizeof(float);
}

hipError_t launch_rmsnorm_bwd(const void* dout, int do_f32, const void* x, int x_f32,
                              const float* gain, const void* dres, int T, int d, float eps,
                              void* dx, float* dgain, void* ws, hipStream_t s) {
  const int nb = T < kBwdBlocks ? T : kBwdBlocks;
  float* partial = dgain ? (float*)ws : nullptr;
  if (nb) {
    with_shape(kWideRows, d, [&](auto th, auto nc) {
      with_bools(do_f32, x_f32, [&](auto df, auto xf) {
        constexpr int TH = decltype(th)::value, NC = decltype(nc)::value;
        hipLaunchKernelGGL((rmsnorm_bwd_kernel<decltype(df)::value, decltype(xf)::value, NC, TH>),
                           dim3(nb), dim3(TH), 0, s, dout, x, gain, dres, T, d, eps, dx, partial);
      });
    });
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !dgain) return e;
  return launch_colsum(partial, nb, d, dgain, nullptr, nullptr, nullptr, s);
}

}  // namespace moe
