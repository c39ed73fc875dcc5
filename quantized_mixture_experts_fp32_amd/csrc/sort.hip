// Tokens into expert order, and the gradients of that copy and of the
// combine.  pair_pos[t*k + j] is the row that pair (t, j) owns; a pair whose
// row is outside [0, T*k) is dropped, and rows that no pair owns keep what
// they held.
//   dispatch      xs[slot_j] = w_j x                    (or x without weights)
//   dispatch_bwd  dx = sum_j w_j dxs[slot_j],           dw_j = <x, dxs[slot_j]>
//   combine_bwd   dy[slot_j] = w_j dout,                dw_j = <dout, y[slot_j]>
// The kernels go by tokens, not by rows: a token's row is read once for its k
// pairs, and its k routing entries are uniform over the block.  HBM-bound;
// sums are fp32 in a fixed order (ranks ascending).  Top-8: dispatch of 8192
// tokens of 2048 (bf16, 299 MB) 57 us, 5.2 TB/s; dispatch_bwd of 4095 tokens
// with weights (168 MB) 34 us, 5.0 TB/s (the k rows asked for together; 36 us
// one after the other); combine_bwd of 515 tokens of 4096 (fp32, 143 MB) 33 us,
// 4.4 TB/s (one pair after the other, which leaves room for twice the waves;
// 35 us with the pairs' loads together).
#include "launch.hpp"
#include "rowops.hpp"

namespace moe {
namespace {
using namespace row;

constexpr int kThreads = 256;

// 256 threads a token, 512 for a long row while there are few tokens.
template <typename F>
void with_threads(int T, int d, F&& f) {
  if (d > 2048 && T <= 2048)
    f(std::integral_constant<int, 512>{});
  else
    f(std::integral_constant<int, 256>{});
}

template <bool kF32, int kTh>
__global__ __launch_bounds__(kTh) void dispatch_kernel(
    const void* __restrict__ x, const int32_t* __restrict__ pair_pos,
    const float* __restrict__ topk_w, int P, int k, int d, void* __restrict__ xs) {
  const int t = blockIdx.x, nch = d >> 3;
  for (int c = threadIdx.x; c < nch; c += kTh) {
    const f32x8 v = load8<kF32>(x, (size_t)t * d + 8 * c);
    for (int j = 0; j < k; ++j) {
      const int s = pair_pos[(size_t)t * k + j];
      if ((unsigned)s >= (unsigned)P) continue;
      const float w = topk_w ? topk_w[(size_t)t * k + j] : 1.0f;
      store8<kF32>(xs, (size_t)s * d + 8 * c, v * w);
    }
  }
}

template <bool kF32, int KM, int kTh>
__global__ __launch_bounds__(kTh) void dispatch_bwd_kernel(
    const void* __restrict__ dxs, const void* __restrict__ x,
    const int32_t* __restrict__ pair_pos, const float* __restrict__ topk_w, int P, int k, int d,
    void* __restrict__ dx, float* __restrict__ dtopk_w) {
  constexpr int kWaves = kTh / kWave;
  __shared__ float red[KM * kWaves];
  const int t = blockIdx.x, nch = d >> 3;
  Pairs<KM> pr;
  pr.load(pair_pos, topk_w, P, k, t);
  float dot[KM];
#pragma unroll
  for (int j = 0; j < KM; ++j) dot[j] = 0.0f;
  for (int c = threadIdx.x; c < nch; c += kTh) {
    f32x8 v = 0.0f, acc = 0.0f;
    if (dtopk_w) v = load8<kF32>(x, (size_t)t * d + 8 * c);
    Raw8<kF32> g[KM];
#pragma unroll
    for (int j = 0; j < KM; ++j)
      if (j < k) g[j].load(dxs, (size_t)pr.slot[j] * d + 8 * c);
#pragma unroll
    for (int j = 0; j < KM; ++j) {
      if (j >= k) continue;
      const f32x8 r = g[j].get(pr.mask[j]);
      acc += r * pr.w[j];
      dot[j] += sum8(v, r);
    }
    store8<kF32>(dx, (size_t)t * d + 8 * c, acc);
  }
  if (!dtopk_w) return;
  block_sum<KM, kWaves>(dot, red);
#pragma unroll
  for (int j = 0; j < KM; ++j)
    if (j < k && (int)threadIdx.x == j)  // (an infinite x times a dropped row's zeros is NaN)
      dtopk_w[(size_t)t * k + j] = pr.mask[j] ? dot[j] : 0.0f;
}

template <bool kDoF32, bool kDyF32, int KM>
__global__ __launch_bounds__(kThreads) void combine_bwd_kernel(
    const void* __restrict__ dout, const float* __restrict__ y,
    const int32_t* __restrict__ pair_pos, const float* __restrict__ topk_w, int P, int k, int d,
    void* __restrict__ dy, float* __restrict__ dtopk_w) {
  constexpr int kWaves = kThreads / kWave;
  __shared__ float red[KM * kWaves];
  const int t = blockIdx.x, nch = d >> 3;
  Pairs<KM> pr;
  pr.load(pair_pos, topk_w, P, k, t);
  float dot[KM];
#pragma unroll
  for (int j = 0; j < KM; ++j) dot[j] = 0.0f;
  for (int c = threadIdx.x; c < nch; c += kThreads) {
    const f32x8 v = load8<kDoF32>(dout, (size_t)t * d + 8 * c);
#pragma unroll
    for (int j = 0; j < KM; ++j) {
      if (!pr.mask[j]) continue;
      if (dtopk_w) dot[j] += sum8(v, load8<true>(y, (size_t)pr.slot[j] * d + 8 * c));
      if (dy) store8<kDyF32>(dy, (size_t)pr.slot[j] * d + 8 * c, v * pr.w[j]);
    }
  }
  if (!dtopk_w) return;
  block_sum<KM, kWaves>(dot, red);
#pragma unroll
  for (int j = 0; j < KM; ++j)
    if (j < k && (int)threadIdx.x == j) dtopk_w[(size_t)t * k + j] = dot[j];
}

}  // namespace

hipError_t launch_dispatch(const void* x, int f32, const int32_t* pair_pos, const float* topk_w,
                           int T, int k, int d, void* xs, hipStream_t s) {
  with_threads(T, d, [&](auto th) {
    constexpr int TH = decltype(th)::value;
    auto kern = f32 ? dispatch_kernel<true, TH> : dispatch_kernel<false, TH>;
    hipLaunchKernelGGL(kern, dim3(T), dim3(TH), 0, s, x, pair_pos, topk_w, T * k, k, d, xs);
  });
  return hipGetLastError();
}

hipError_t launch_dispatch_bwd(const void* dxs, int f32, const void* x, const int32_t* pair_pos,
                               const float* topk_w, int T, int k, int d, void* dx,
                               float* dtopk_w, hipStream_t s) {
  with_pairs(k, [&](auto km) {
    constexpr int KM = decltype(km)::value > 0 ? decltype(km)::value : 2;
    with_threads(T, d, [&](auto th) {
      constexpr int TH = decltype(th)::value;
      auto kern = f32 ? dispatch_bwd_kernel<true, KM, TH> : dispatch_bwd_kernel<false, KM, TH>;
      hipLaunchKernelGGL(kern, dim3(T), dim3(TH), 0, s, dxs, x, pair_pos, topk_w, T * k, k, d, dx,
                         dtopk_w);
    });
  });
  return hipGetLastError();
}

hipError_t launch_combine_bwd(const void* dout, int do_f32, const float* y,
                              const int32_t* pair_pos, const float* topk_w, int T, int k, int d,
                              void* dy, int dy_f32, float* dtopk_w, hipStream_t s) {
  with_pairs(k, [&](auto km) {
    constexpr int KM = decltype(km)::value > 0 ? decltype(km)::value : 2;
    with_bools(do_f32, dy_f32, [&](auto df, auto yf) {
      hipLaunchKernelGGL((combine_bwd_kernel<decltype(df)::value, decltype(yf)::value, KM>),
                         dim3(T), dim3(kThreads), 0, s, dout, y, pair_pos, topk_w, T * k, k, d, dy,
                         dtopk_w);
    });
  });
  return hipGetLastError();
}

}  // namespace moe
