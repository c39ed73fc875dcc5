// End of a block: the combine of the routed pairs' outputs, the norm after
// the block, its gate, the scaled residual and the next block's norm in one
// pass over the rows; and the gradient of all but the last.
//   o   = sum_j w_j y[slot_j] (+ add)          n = o * rstd(o) * post_gain  (or o)
//   out = res_scale * residual + gate * n      next = out * rstd(out) * next_gain
// A pair whose slot is outside [0, T*k) is dropped: its y is not read.
//
// Gradient, for the gradient r of out, with gc the channel gate (or 1), tg
// the token gate (or 1), u = r gc post_gain and h = o rstd(o):
//   do = tg rstd (u - h mean(u h))             (without post norm: do = tg u)
//   dy[slot_j] = w_j do,   dw_j = <do, y[slot_j]>
// dw_j needs do, which needs row sums over o, which needs every y of the
// row; to read y once, the row is reduced to A_j = <u, y_j> and B_j =
// <o, y_j> beside <o, o> and <u, o>, and then
//   dw_j = tg rstd (A_j - rstd^2 <u, o> / d * B_j).
// The gains' column sums are one: with S = sum over tokens of tg r h,
// dpost_gain = gc S and the channel gate's gradient is post_gain S (a layer
// has one of the two gates, so tg = 1 there).
//
// HBM-bound: y (fp32, k rows a token) dominates the bytes.  One block holds a
// row of o in registers; all sums are fp32 in a fixed order.
#include "../../include/moe_wq.h"
#include "launch.hpp"
#include "rowops.hpp"

namespace moe {
namespace {
using namespace row;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kBwdBlocks = 512;

// The pairs of one token: KM >= k of them, dropped and missing ones with
// weight 0 and slot -1.
template <int KM>
struct Pairs {
  int slot[KM > 0 ? KM : 1];
  float w[KM > 0 ? KM : 1];
  __device__ __forceinline__ void load(const BlockOutArgs& a, int t) {
    const int P = a.T * a.k;
#pragma unroll
    for (int j = 0; j < KM; ++j) {
      slot[j] = -1;
      w[j] = 0.0f;
      if (j < a.k) {
        const int s = a.pair_pos[(size_t)t * a.k + j];
        if ((unsigned)s < (unsigned)P) {
          slot[j] = s;
          w[j] = a.topk_w[(size_t)t * a.k + j];
        }
      }
    }
  }
};

template <bool kF32, int KM, int NC>
__global__ __launch_bounds__(kThreads) void combine_residual_kernel(
    BlockOutArgs a, const void* residual, const float* __restrict__ next_gain, void* out,
    void* __restrict__ next_out) {
  __shared__ float red[2][kWaves];
  const int t = blockIdx.x, nch = a.d >> 3;
  const size_t base = (size_t)t * a.d;
  Pairs<KM> pr;
  pr.load(a, t);
  f32x8 o[NC];
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = threadIdx.x + kThreads * i;
    o[i] = 0.0f;
    if (c < nch) {
#pragma unroll
      for (int j = 0; j < KM; ++j)
        if (pr.slot[j] >= 0) o[i] += pr.w[j] * load8<true>(a.y, (size_t)pr.slot[j] * a.d + 8 * c);
      if (a.add) o[i] += load8<kF32>(a.add, base + 8 * c);
      s[0] += sum8(o[i], o[i]);
    }
  }
  float rstd = 1.0f;
  if (a.post_gain) {
    block_sum<1, kWaves>(s, red[0]);
    rstd = rsqrtf(s[0] / a.d + a.eps);
  }
  const float tg = a.gate_mode == MOE_GATE_TOKEN ? a.gate[t] * rstd : rstd;
  s[0] = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = threadIdx.x + kThreads * i;
    if (c < nch) {
      f32x8 n = o[i] * tg;
      if (a.post_gain) n *= load8<true>(a.post_gain, 8 * c);
      if (a.gate_mode == MOE_GATE_CHANNEL) n *= load8<true>(a.gate, 8 * c);
      o[i] = load8<kF32>(residual, base + 8 * c) * a.res_scale + n;
      store8<kF32>(out, base + 8 * c, o[i]);
      s[0] += sum8(o[i], o[i]);
    }
  }
  if (!next_out) return;
  block_sum<1, kWaves>(s, red[1]);
  rstd = rsqrtf(s[0] / a.d + a.eps);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = threadIdx.x + kThreads * i;
    if (c < nch) {
      f32x8 n = o[i] * rstd;
      if (next_gain) n *= load8<true>(next_gain, 8 * c);
      store8<false>(next_out, base + 8 * c, n);
    }
  }
}

template <bool kF32, bool kDyF32, int KM, int NC>
__global__ __launch_bounds__(kThreads) void combine_residual_bwd_kernel(
    BlockOutArgs a, const void* dout, void* __restrict__ dy, float* __restrict__ dtopk_w,
    void* __restrict__ dadd, void* dresidual, float* __restrict__ dgate_t,
    float* __restrict__ partial) {
  constexpr int kSums = 2 + 2 * KM;
  __shared__ float red[2][kSums * kWaves];
  const int nch = a.d >> 3;
  const bool post = a.post_gain != nullptr, gch = a.gate_mode == MOE_GATE_CHANNEL;
  f32x8 acc[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) acc[i] = 0.0f;
  int turn = 0;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
    const size_t base = (size_t)t * a.d;
    Pairs<KM> pr;
    pr.load(a, t);
    f32x8 o[NC], u[NC], r[NC];
    float s[kSums];
#pragma unroll
    for (int i = 0; i < kSums; ++i) s[i] = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = threadIdx.x + kThreads * i;
      if (c < nch) {
        f32x8 y[KM > 0 ? KM : 1];
        o[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < KM; ++j) {
          y[j] = 0.0f;
          if (pr.slot[j] >= 0) y[j] = load8<true>(a.y, (size_t)pr.slot[j] * a.d + 8 * c);
          o[i] += pr.w[j] * y[j];
        }
        if (a.add) o[i] += load8<kF32>(a.add, base + 8 * c);
        r[i] = load8<kF32>(dout, base + 8 * c);
        if (dresidual) store8<kF32>(dresidual, base + 8 * c, r[i] * a.res_scale);
        u[i] = r[i];
        if (gch) u[i] *= load8<true>(a.gate, 8 * c);
        if (post) u[i] *= load8<true>(a.post_gain, 8 * c);
        s[0] += sum8(o[i], o[i]);
        s[1] += sum8(u[i], o[i]);
#pragma unroll
        for (int j = 0; j < KM; ++j) {
          s[2 + j] += sum8(u[i], y[j]);
          s[2 + KM + j] += sum8(o[i], y[j]);
        }
      }
    }
    block_sum<kSums, kWaves>(s, red[turn]);
    const float tg = a.gate_mode == MOE_GATE_TOKEN ? a.gate[t] : 1.0f;
    const float rstd = post ? rsqrtf(s[0] / a.d + a.eps) : 1.0f;
    const float b = post ? s[1] / a.d * rstd * rstd : 0.0f;
    if (dgate_t && threadIdx.x == 0) dgate_t[t] = s[1] * rstd;
#pragma unroll
    for (int j = 0; j < KM; ++j)
      if (dtopk_w && j < a.k && (int)threadIdx.x == j)
        dtopk_w[(size_t)t * a.k + j] = tg * rstd * (s[2 + j] - b * s[2 + KM + j]);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = threadIdx.x + kThreads * i;
      if (c < nch) {
        const f32x8 g = (u[i] - o[i] * b) * (tg * rstd);
        if (dadd) store8<kF32>(dadd, base + 8 * c, g);
        if (dy) {
#pragma unroll
          for (int j = 0; j < KM; ++j)
            if (pr.slot[j] >= 0)
              store8<kDyF32>(dy, (size_t)pr.slot[j] * a.d + 8 * c, g * pr.w[j]);
        }
        acc[i] += r[i] * (o[i] * (tg * rstd));
      }
    }
  }
  if (!partial) return;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = threadIdx.x + kThreads * i;
    if (c < nch) store8<true>(partial, (size_t)blockIdx.x * a.d + 8 * c, acc[i]);
  }
}

// Calls f with the number of pairs a token's kernel is built for (0, 8 or
// 16) and the chunks a thread holds, as types.
template <typename F>
void by_shape(int k, int d, F&& f) {
  auto nc = [&](auto km) {
    switch ((d / 8 + kThreads - 1) / kThreads) {
      case 1: return f(km, std::integral_constant<int, 1>{});
      case 2: return f(km, std::integral_constant<int, 2>{});
      case 3: return f(km, std::integral_constant<int, 3>{});
      default: return f(km, std::integral_constant<int, 4>{});
    }
  };
  if (k == 0)
    nc(std::integral_constant<int, 0>{});
  else if (k <= 8)
    nc(std::integral_constant<int, 8>{});
  else
    nc(std::integral_constant<int, 16>{});
}

}  // namespace

hipError_t launch_combine_residual(const BlockOutArgs& a, const void* residual,
                                   const float* next_gain, void* out, void* next_out,
                                   hipStream_t s) {
  by_shape(a.k, a.d, [&](auto km, auto nc) {
    constexpr int KM = decltype(km)::value, NC = decltype(nc)::value;
    auto kern = a.f32 ? combine_residual_kernel<true, KM, NC>
                      : combine_residual_kernel<false, KM, NC>;
    hipLaunchKernelGGL(kern, dim3(a.T), dim3(kThreads), 0, s, a, residual, next_gain, out,
                       next_out);
  });
  return hipGetLastError();
}

size_t combine_residual_bwd_ws_bytes(int T, int d) {
  return (size_t)(T < kBwdBlocks ? T : kBwdBlocks) * d * sizeof(float);
}

hipError_t launch_combine_residual_bwd(const BlockOutArgs& a, const void* dout, void* dy,
                                       int dy_f32, float* dtopk_w, void* dadd, void* dresidual,
                                       float* dpost_gain, float* dgate, void* ws,
                                       hipStream_t s) {
  const int nb = a.T < kBwdBlocks ? a.T : kBwdBlocks;
  const bool gch = a.gate_mode == MOE_GATE_CHANNEL;
  float* dgate_t = a.gate_mode == MOE_GATE_TOKEN ? dgate : nullptr;
  float* dgate_c = gch ? dgate : nullptr;
  const bool colsum = dpost_gain || dgate_c;
  float* partial = colsum ? (float*)ws : nullptr;
  if (nb) {
    by_shape(a.k, a.d, [&](auto km, auto nc) {
      constexpr int KM = decltype(km)::value, NC = decltype(nc)::value;
      with_bools(a.f32, dy_f32, [&](auto f, auto yf) {
        hipLaunchKernelGGL((combine_residual_bwd_kernel<decltype(f)::value, decltype(yf)::value,
                                                        KM, NC>),
                           dim3(nb), dim3(kThreads), 0, s, a, dout, dy, dtopk_w, dadd, dresidual,
                           dgate_t, partial);
      });
    });
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !colsum) return e;
  return launch_colsum(partial, nb, a.d, dpost_gain, gch ? a.gate : nullptr, dgate_c,
                       a.post_gain, s);
}

}  // namespace moe
