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
// row of o in registers; all sums are fp32 in a fixed order.  Forward, 4096
// tokens of 2048 channels, top-8, with an fp32 residual, a shared output and
// the next norm (384 MB): 77 us, 5.0 TB/s; one token of 4096: 4.9 us.  Backward,
// 4093 tokens of 4096, top-8 (872 MB): 188 us, 4.6 TB/s.  A large copy reaches
// 4.9 TB/s.
#include "../../include/moe_wq.h"
#include "launch.hpp"
#include "rowops.hpp"

namespace moe {
namespace {
using namespace row;

// Blocks of the backward pass: each takes every kBwdBlocks-th row and keeps
// its share of the column sums in registers.
constexpr int kBwdBlocks = 512;

template <bool kF32, int KM, int NC, int kThreads>
__global__ __launch_bounds__(kThreads) void combine_residual_kernel(
    BlockOutArgs a, const void* residual, const float* __restrict__ next_gain, void* out,
    void* __restrict__ next_out) {
  constexpr int kWaves = kThreads / kWave;
  // few rows (wide blocks): what does not depend on the routing is asked for
  // before it, in registers that a full batch needs for occupancy
  constexpr bool kAhead = kThreads == 512;
  __shared__ float red[2][kWaves];
  const int t = blockIdx.x, nch = a.d >> 3;
  const size_t base = (size_t)t * a.d;
  f32x8 res[NC], fac[NC], nxt[NC];
  auto ask = [&](int i) {
    const int c = threadIdx.x + kThreads * i;
    fac[i] = 1.0f;
    nxt[i] = 1.0f;
    if (c >= nch) return;
    res[i] = load8<kF32>(residual, base + 8 * c);
    if (a.post_gain) fac[i] = load8<true>(a.post_gain, 8 * c);
    if (a.gate_mode == MOE_GATE_CHANNEL) fac[i] *= load8<true>(a.gate, 8 * c);
    if (kAhead && next_gain) nxt[i] = load8<true>(next_gain, 8 * c);
  };
  Pairs<KM> pr;
  pr.load(a.pair_pos, a.topk_w, a.T * a.k, a.k, t);
  if (kAhead) {
#pragma unroll
    for (int i = 0; i < NC; ++i) ask(i);
  }
  f32x8 o[NC];
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = threadIdx.x + kThreads * i;
    o[i] = 0.0f;
    if (c < nch) {
      constexpr int kBatch = KM < 8 ? (KM ? KM : 1) : 8;  // rows asked for together
      Raw8<true> y[kBatch];
#pragma unroll
      for (int j0 = 0; j0 < KM; j0 += kBatch) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (j0 + j < a.k) y[j].load(a.y, (size_t)pr.slot[j0 + j] * a.d + 8 * c);
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (j0 + j < a.k) o[i] += pr.w[j0 + j] * y[j].get(pr.mask[j0 + j]);
      }
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
    if (!kAhead) ask(i);
    if (c < nch) {
      o[i] = res[i] * a.res_scale + o[i] * tg * fac[i];
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
      if (!kAhead && next_gain) nxt[i] = load8<true>(next_gain, 8 * c);
      store8<false>(next_out, base + 8 * c, o[i] * rstd * nxt[i]);
    }
  }
}

template <bool kF32, bool kDyF32, int KM, int NC, int kThreads>
__global__ __launch_bounds__(kThreads) void combine_residual_bwd_kernel(
    BlockOutArgs a, const void* dout, void* __restrict__ dy, float* __restrict__ dtopk_w,
    void* __restrict__ dadd, void* dresidual, float* __restrict__ dgate_t,
    float* __restrict__ partial) {
  constexpr int kSums = 2 + 2 * KM, kWaves = kThreads / kWave;
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
    pr.load(a.pair_pos, a.topk_w, a.T * a.k, a.k, t);
    f32x8 o[NC], u[NC], r[NC];
    float s[kSums];
#pragma unroll
    for (int i = 0; i < kSums; ++i) s[i] = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = threadIdx.x + kThreads * i;
      if (c < nch) {
        // the rows of up to 8 pairs stay in registers between o and the sums
        // that need it; more are read four at a time, and again for the sums
        constexpr int kBatch = KM > 8 ? 4 : KM ? KM : 1;
        f32x8 y[kBatch];
        auto rows = [&](int j0) {
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            y[j] = 0.0f;
            if (j0 + j < a.k) y[j] = load8<true>(a.y, (size_t)pr.slot[j0 + j] * a.d + 8 * c);
          }
#pragma unroll
          for (int j = 0; j < kBatch; ++j)
            if (!pr.mask[j0 + j]) y[j] = 0.0f;
          if (KM > kBatch) __builtin_amdgcn_sched_barrier(0);
        };
        o[i] = 0.0f;
        r[i] = load8<kF32>(dout, base + 8 * c);
#pragma unroll
        for (int j0 = 0; j0 < KM; j0 += kBatch) {
          rows(j0);
#pragma unroll
          for (int j = 0; j < kBatch; ++j) o[i] += pr.w[j0 + j] * y[j];
        }
        if (a.add) o[i] += load8<kF32>(a.add, base + 8 * c);
        if (dresidual) store8<kF32>(dresidual, base + 8 * c, r[i] * a.res_scale);
        u[i] = r[i];
        if (gch) u[i] *= load8<true>(a.gate, 8 * c);
        if (post) u[i] *= load8<true>(a.post_gain, 8 * c);
        s[0] += sum8(o[i], o[i]);
        s[1] += sum8(u[i], o[i]);
#pragma unroll
        for (int j0 = 0; j0 < KM; j0 += kBatch) {
          if (KM > kBatch) rows(j0);
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            s[2 + j0 + j] += sum8(u[i], y[j]);
            s[2 + KM + j0 + j] += sum8(o[i], y[j]);
          }
        }
      }
      // one chunk's rows in registers at a time: occupancy hides more than
      // asking for the next chunk's early would
      __builtin_amdgcn_sched_barrier(0);
    }
    block_sum<kSums, kWaves>(s, red[turn]);
    const float tg = a.gate_mode == MOE_GATE_TOKEN ? a.gate[t] : 1.0f;
    const float rstd = post ? rsqrtf(s[0] / a.d + a.eps) : 1.0f;
    const float b = post ? s[1] / a.d * rstd * rstd : 0.0f;
    if (dgate_t && threadIdx.x == 0) dgate_t[t] = s[1] * rstd;
#pragma unroll
    for (int j = 0; j < KM; ++j)
      if (dtopk_w && j < a.k && (int)threadIdx.x == j)
        dtopk_w[(size_t)t * a.k + j] =
            !pr.mask[j] ? 0.0f
                        : tg * rstd * (post ? s[2 + j] - b * s[2 + KM + j] : s[2 + j]);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = threadIdx.x + kThreads * i;
      if (c < nch) {
        f32x8 g = u[i];
        if (post) g -= o[i] * b;
        g *= tg * rstd;
        if (dadd) store8<kF32>(dadd, base + 8 * c, g);
        if (dy) {
#pragma unroll
          for (int j = 0; j < KM; ++j)
            if (pr.mask[j])
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

}  // namespace

hipError_t launch_combine_residual(const BlockOutArgs& a, const void* residual,
                                   const float* next_gain, void* out, void* next_out,
                                   hipStream_t s) {
  with_pairs(a.k, [&](auto km) {
    with_shape(a.T, a.d, [&](auto th, auto nc) {
      constexpr int KM = decltype(km)::value, TH = decltype(th)::value, NC = decltype(nc)::value;
      auto kern = a.f32 ? combine_residual_kernel<true, KM, NC, TH>
                        : combine_residual_kernel<false, KM, NC, TH>;
      hipLaunchKernelGGL(kern, dim3(a.T), dim3(TH), 0, s, a, residual, next_gain, out, next_out);
    });
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
    with_pairs(a.k, [&](auto km) {
      with_shape(a.T, a.d, [&](auto th, auto nc) {
        constexpr int KM = decltype(km)::value, TH = decltype(th)::value, NC = decltype(nc)::value;
        with_bools(a.f32, dy_f32, [&](auto f, auto yf) {
          hipLaunchKernelGGL((combine_residual_bwd_kernel<decltype(f)::value, decltype(yf)::value,
                                                          KM, NC, TH>),
                             dim3(nb), dim3(TH), 0, s, a, dout, dy, dtopk_w, dadd, dresidual,
                             dgate_t, partial);
        });
      });
    });
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !colsum) return e;
  return launch_colsum(partial, nb, a.d, dpost_gain, gch ? a.gate : nullptr, dgate_c,
                       a.post_gain, s);
}

}  // namespace moe
