// Product of few rows (up to 16 tokens) with a weight matrix: C[t][n] = sum_k
// x[t][k] w[n][k], bound by the weights' bytes and by latency.  A block takes 16
// weight rows and its waves share k, 128 bytes of each row in turn.  Weights are
// loaded straight into registers as fragments of the 16 x 16 matrix
// instruction (lane l: row l % 16, bytes 16 (l / 16) of each 64), two groups of
// kU units ahead; the tokens' rows lie in LDS, chunk c of 16 bytes of row t at
// c ^ (t & 15) (no bank conflicts), a piece of k at a time where they are long.
// The waves' sums are joined once, through LDS, in wave order.
//
// Buffer loads do the bounds: weight rows past the end and bytes past k are out
// of range, read as zeros and cost no traffic.
//
// Pair form: 8 gate and 8 up rows a block, so that the join has both of a
// feature.
// Quantising form (int8 weights, bf16 tokens): each wave turns whole rows into
// codes on their way to LDS, while the weights are in flight.
//
// Bytes: one token of 4096 values through 14336 features (both products of the
// gated block) 69 us, 5.1 TB/s, the rate of a large copy; smaller calls are bound
// by the latency of a launch and of the first loads, and by the tokens' way to
// LDS, which 16 long tokens take as long for as the weights: 2048 through 1024
// features 8.6 us for one token and 10.6 for 16, 4096 through 2048 15.0 and 18.2.
// Eight waves a block share k, so that 16 weight rows a block still keep enough
// loads in flight; the first group of weights is asked for ahead of the tokens
// (16 tokens, 2048 through 1024: 1.1 us less than behind them).
#pragma once
#include "i8.hpp"
#include "mm_core.hpp"

namespace moe {
namespace mm {

struct DirectArgs {
  const char* x;
  const char* w;
  long long xstride, wstride;  // bytes between rows
  int T, N;    // N: features (of each matrix in the pair form: up rows follow N gate rows)
  int kbytes;  // bytes of k in a weight row
  int piece;   // bytes of k of a token in LDS, a multiple of 256
};

constexpr int kDirectWaves = 8;
constexpr int kDirectLds = 64 << 10;      // two blocks a CU
constexpr int kDirectLdsOne = 144 << 10;  // a block alone on its CU

template <typename Mma, int kU, bool kPair, bool kQuant, typename Epi>
__global__ __launch_bounds__(kDirectWaves* kWave, 4) void direct_kernel(const DirectArgs p,
                                                                       Epi epi) {
  typedef typename Mma::Acc Quad;
  constexpr int W = kDirectWaves;
  extern __shared__ __align__(1024) char lds[];  // tokens [T][piece]; then sums [W][64]
  __shared__ float sx[16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * (kPair ? 8 : 16), T = p.T;

  const int wrow = kPair ? r & 7 : r;
  uint32_t woff = (uint32_t)((kPair && r >= 8 ? p.N + wrow : wrow) * p.wstride) + 16 * q;
  if (n0 + wrow >= p.N) woff = kOutOfRange;
  const __amdgpu_buffer_rsrc_t wr = rsrc_of(p.w + (size_t)n0 * p.wstride);
  // The lane's token in LDS (rows past the last repeat it); its chunk i of 16
  // bytes lies at i ^ sw.
  const int token = min(r, T - 1), sw = token & 15;
  const char* const xrow = lds + token * p.piece;

  struct Unit {
    u32x4 w[2];
  };
  Quad acc = {0, 0, 0, 0};
  float inv_scale = 0.0f;

  for (int k0 = 0; k0 < p.kbytes; k0 += p.piece) {
    const int bytes = min(p.piece, p.kbytes - k0), units = (bytes + 127) >> 7;
    if (k0) __syncthreads();  // every wave has read the last piece
    auto load = [&](Unit (&u)[kU], int i) {  // (units past the last are out of range)
#pragma unroll
      for (int j = 0; j < kU; ++j)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int b = 128 * (wave + W * (i + j)) + 64 * s;
          const uint32_t o = b + 16 * q < bytes ? woff + k0 + b : kOutOfRange;
          u[j].w[s] =
              __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(wr, (int)o, 0, 0));
        }
    };
    Unit a[kU], b[kU];
    if constexpr (!kQuant) {
      load(a, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
    // tokens to LDS: asked for ahead of the weights
    if constexpr (!kQuant) {
      const int per = p.piece >> 4, n = T * per;  // chunks
      const __amdgpu_buffer_rsrc_t xr = rsrc_of(p.x + k0);
      for (int i = wave * kWave; i < n; i += W * kWave) {
        const int t = (i + lane) / per, c = (i + lane) - t * per, at = 16 * (c ^ (t & 15));
        const uint32_t o = t < T && at < bytes ? (uint32_t)(t * p.xstride) + at : kOutOfRange;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, (Lds)(lds + 16 * i), 16, (int)o, 0, 0, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (kQuant) {
      // a row is one wave's; all of it is read once for its largest value
      const int nch = p.kbytes >> 3;
      const __amdgpu_buffer_rsrc_t xr = rsrc_of(p.x);
      constexpr int kHold = 8;  // chunks of 8 values a lane holds
      u32x4 v[kHold];
      const int t = wave;
      if (t < T) {
#pragma unroll
        for (int h = 0; h < kHold; ++h) {
          const int c = 64 * h + lane;
          v[h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                     xr, (int)(c < nch ? (uint32_t)(t * p.xstride) + 16 * c : kOutOfRange), 0, 0));
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      load(a, 0);
      load(b, kU);
      __builtin_amdgcn_sched_barrier(0);
      if (t < T) {
        if (k0 == 0) {
          uint32_t m = 0;
#pragma unroll
          for (int h = 0; h < kHold; ++h) m = max(m, top8(bf16x8_to_f32(v[h])));
          for (int c = 64 * kHold + lane; c < nch; c += 64)
            m = max(m, top8(bf16x8_to_f32(*(const u32x4*)(p.x + t * p.xstride + 16 * c))));
#pragma unroll
          for (int o = 32; o > 0; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, kWave));
          const Scaling s(m);
          inv_scale = s.inv;
          if (lane == 0) sx[t] = s.scale;
        }
        // codes of values 8 c .. 8 c + 7 of the piece
        auto put = [&](int c, u32x4 x) {
          const int at = 8 * c - k0;
          if (at >= 0 && at < bytes)
            *(u32x2*)(lds + t * p.piece + 16 * ((at >> 4) ^ (t & 15)) + (at & 8)) =
                codes8(bf16x8_to_f32(x), inv_scale);
        };
#pragma unroll
        for (int h = 0; h < kHold; ++h) put(64 * h + lane, v[h]);
        for (int c = 64 * kHold + lane; c < nch; c += 64)
          put(c, *(const u32x4*)(p.x + t * p.xstride + 16 * c));
      }
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0); the weights stay in flight
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
    } else {
      load(b, kU);
      __builtin_amdgcn_sched_barrier(0);
      wait_stage<2 * kU>();  // the tokens are in; the weights stay in flight
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
    }
    const int mine = units > wave ? (units - wave + W - 1) / W : 0;  // units wave + W i
    auto use = [&](const Unit& u, int i) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int ch = 8 * (wave + W * i) + 4 * s + q;
        acc = Mma::mma(u.w[s], *(const u32x4*)(xrow + 16 * (ch ^ sw)), acc);
      }
    };
    for (int i = 0; i < mine; i += 2 * kU) {
#pragma unroll
      for (int j = 0; j < kU; ++j)
        if (i + j < mine) use(a[j], i + j);
      if (i + 2 * kU < mine) load(a, i + 2 * kU);
#pragma unroll
      for (int j = 0; j < kU; ++j)
        if (i + kU + j < mine) use(b[j], i + kU + j);
      if (i + 3 * kU < mine) load(b, i + 3 * kU);
    }
  }

  // join
  asm volatile("" : "+v"(acc));
  __syncthreads();  // the sums take the tokens' place
  Quad* red = (Quad*)lds;
  red[wave * 64 + lane] = acc;
  __syncthreads();
  auto sum = [&](int o) {
    Quad v = red[o];
#pragma unroll
    for (int w = 1; w < W; ++w) v += red[w * 64 + o];
    return v;
  };
  if constexpr (kQuant) epi.sx = sx;
  // four rows of a token a thread (pair form: of the gate tile and the up tile)
  for (int o = threadIdx.x; o < (kPair ? 32 : 64); o += W * kWave) {
    const int m = o & 15, n = n0 + 4 * (o >> 4);
    if (m >= T || n >= p.N) continue;
    if constexpr (kPair)
      epi(m, n, sum(o), sum(32 + o));
    else
      epi(m, n, sum(o));
  }
}

inline long long direct_blocks(long long N, bool pair) {
  return (N + (pair ? 7 : 15)) / (pair ? 8 : 16);
}
// (a launch has fewer than 2^32 threads, 32 a feature here: N of 2^27 goes to a tile)
inline bool direct_applies(long long T, long long N, long long row_bytes, bool pair) {
  return T <= 16 && (pair ? N + 8 : 16) * row_bytes < (1LL << 31) - (1 << 20) &&
         direct_blocks(N, pair) * (kDirectWaves * kWave) < 1LL << 32;
}
constexpr int kQuantRows = kDirectWaves;  // tokens that the quantising form takes

// x [T][..] (kQuant: bf16 rows, quantised by row) times w.
template <typename Mma, bool kPair, bool kQuant, typename Epi>
inline hipError_t launch_direct(DirectArgs p, const Epi& epi, hipStream_t s) {
  const int units = (p.kbytes + 127) >> 7;
  const int blocks = (int)direct_blocks(p.N, kPair);
  const int most = blocks <= 256 ? kDirectLdsOne : kDirectLds;
  p.piece = std::min((p.kbytes + 255) & ~255, most / p.T & ~255);
  // (the last load into LDS may reach past the tokens)
  const size_t lds = std::max((size_t)p.T * p.piece + 1024, (size_t)kDirectWaves * 1024);
  auto go = [&](auto u) {
    hipLaunchKernelGGL((direct_kernel<Mma, decltype(u)::value, kPair, kQuant, Epi>), dim3(blocks),
                       dim3(kDirectWaves * kWave), lds, s, p, epi);
  };
  using std::integral_constant;
  if (units <= 16)
    go(integral_constant<int, 1>{});
  else if (kQuant || units <= 32)
    go(integral_constant<int, 2>{});
  else
    go(integral_constant<int, kQuant ? 2 : 4>{});
  return hipGetLastError();
}

}  // namespace mm
}  // namespace moe
