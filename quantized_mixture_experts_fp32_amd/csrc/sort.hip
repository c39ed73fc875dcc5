// Tokens into expert order, and the gradients of that copy and of the
// combine.  pair_pos[t*k + j] is the row that pair (t, j) owns; a pair whose
// row is outside [0, T*k) is dropped, and rows that no pair owns keep what
// they held.
//   dispatch      xs[slot_j] = w_j x                    (or x without weights)
//   dispatch_bwd  dx = sum_j w_j dxs[slot_j],           dw_j = <x, dxs[slot_j]>
//   combine_bwd   dy[slot_j] = w_j dout,                dw_j = <dout, y[slot_j]>
// The kernels go by tokens, not by rows: a token's row is read once for its k
// pairs, and its k routing entries are uniform over the block.  HBM-bound;
// sums are fp32 in a fixed order (ranks ascending).
#include "launch.hpp"
#include "rowops.hpp"

namespace moe {
namespace {
using namespace row;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

template <bool kF32>
__global__ __launch_bounds__(kThreads) void dispatch_kernel(
    const void* __restrict__ x, const int32_t* __restrict__ pair_pos,
    const float* __restrict__ topk_w, int P, int k, int d, void* __restrict__ xs) {
  const int t = blockIdx.x, nch = d >> 3;
  for (int c = threadIdx.x; c < nch; c += kThreads) {
    const f32x8 v = load8<kF32>(x, (size_t)t * d + 8 * c);
    for (int j = 0; j < k; ++j) {
      const int s = pair_pos[(size_t)t * k + j];
      if ((unsigned)s >= (unsigned)P) continue;
      const float w = topk_w ? topk_w[(size_t)t * k + j] : 1.0f;
      store8<kF32>(xs, (size_t)s * d + 8 * c, v * w);
    }
  }
}

template <bool kF32, int KM>
__global__ __launch_bounds__(kThreads) void dispatch_bwd_kernel(
    const void* __restrict__ dxs, const void* __restrict__ x,
    const int32_t* __restrict__ pair_pos, const float* __restrict__ topk_w, int P, int k, int d,
    void* __restrict__ dx, float* __restrict__ dtopk_w) {
  __shared__ float red[KM * kWaves];
  const int t = blockIdx.x, nch = d >> 3;
  float dot[KM];
#pragma unroll
  for (int j = 0; j < KM; ++j) dot[j] = 0.0f;
  for (int c = threadIdx.x; c < nch; c += kThreads) {
    f32x8 v = 0.0f, acc = 0.0f;
    if (dtopk_w) v = load8<kF32>(x, (size_t)t * d + 8 * c);
#pragma unroll
    for (int j = 0; j < KM; ++j) {
      const int s = j < k ? pair_pos[(size_t)t * k + j] : -1;
      if ((unsigned)s >= (unsigned)P) continue;
      const f32x8 g = load8<kF32>(dxs, (size_t)s * d + 8 * c);
      acc += topk_w ? g * topk_w[(size_t)t * k + j] : g;
      dot[j] += sum8(v, g);
    }
    store8<kF32>(dx, (size_t)t * d + 8 * c, acc);
  }
  if (!dtopk_w) return;
  block_sum<KM, kWaves>(dot, red);
#pragma unroll
  for (int j = 0; j < KM; ++j)
    if (j < k && (int)threadIdx.x == j) dtopk_w[(size_t)t * k + j] = dot[j];
}

template <bool kDoF32, bool kDyF32, int KM>
__global__ __launch_bounds__(kThreads) void combine_bwd_kernel(
    const void* __restrict__ dout, const float* __restrict__ y,
    const int32_t* __restrict__ pair_pos, const float* __restrict__ topk_w, int P, int k, int d,
    void* __restrict__ dy, float* __restrict__ dtopk_w) {
  __shared__ float red[KM * kWaves];
  const int t = blockIdx.x, nch = d >> 3;
  float dot[KM];
#pragma unroll
  for (int j = 0; j < KM; ++j) dot[j] = 0.0f;
  for (int c = threadIdx.x; c < nch; c += kThreads) {
    const f32x8 v = load8<kDoF32>(dout, (size_t)t * d + 8 * c);
#pragma unroll
    for (int j = 0; j < KM; ++j) {
      const int s = j < k ? pair_pos[(size_t)t * k + j] : -1;
      if ((unsigned)s >= (unsigned)P) continue;
      if (dtopk_w) dot[j] += sum8(v, load8<true>(y, (size_t)s * d + 8 * c));
      if (dy) store8<kDyF32>(dy, (size_t)s * d + 8 * c, v * topk_w[(size_t)t * k + j]);
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
  auto kern = f32 ? dispatch_kernel<true> : dispatch_kernel<false>;
  hipLaunchKernelGGL(kern, dim3(T), dim3(kThreads), 0, s, x, pair_pos, topk_w, T * k, k, d, xs);
  return hipGetLastError();
}

hipError_t launch_dispatch_bwd(const void* dxs, int f32, const void* x, const int32_t* pair_pos,
                               const float* topk_w, int T, int k, int d, void* dx,
                               float* dtopk_w, hipStream_t s) {
  with_bools(f32, k <= 8, [&](auto f, auto k8) {
    hipLaunchKernelGGL((dispatch_bwd_kernel<decltype(f)::value, decltype(k8)::value ? 8 : 16>),
                       dim3(T), dim3(kThreads), 0, s, dxs, x, pair_pos, topk_w, T * k, k, d, dx,
                       dtopk_w);
  });
  return hipGetLastError();
}

hipError_t launch_combine_bwd(const void* dout, int do_f32, const float* y,
                              const int32_t* pair_pos, const float* topk_w, int T, int k, int d,
                              void* dy, int dy_f32, float* dtopk_w, hipStream_t s) {
  with_bools(do_f32, dy_f32, [&](auto df, auto yf) {
    constexpr bool D = decltype(df)::value, Y = decltype(yf)::value;
    auto kern = k <= 8 ? combine_bwd_kernel<D, Y, 8> : combine_bwd_kernel<D, Y, 16>;
    hipLaunchKernelGGL(kern, dim3(T), dim3(kThreads), 0, s, dout, y, pair_pos, topk_w, T * k, k,
                       d, dy, dtopk_w);
  });
  return hipGetLastError();
}

}  // namespace moe
