// Gated feed-forward block with bf16 weights (a shared expert beside the routed
// ones) and its gradient.  Wgu [2f][d]: gate rows, then up rows; Wd [d][f].
//   g = x Wg^T, u = x Wu^T, h = silu(g) u, out = h Wd^T
// forward: one product over both projections, whose tiles hold a gate and the
// up feature beside it in one lane, so that activation and product are formed in
// registers; h goes to memory once, as bf16 (as the experts' does), for the
// second product.
// gradient, for dout, with s = 1 / (1 + e^-g) and g, u kept as bf16 or computed
// again:
//   dh = dout Wd
//   du = dh g s,  dg = dh u s (1 + g (1 - s)),  h = g s u       (its epilogue)
//   dx = [dg du] Wgu,  dWgu = [dg du]^T x,  dWd = dout^T h
// dg, du and h are rounded to bf16, the matrix cores' operand type, and so is an fp32
// dout, which is an operand too: results are 2.4e-3 (bf16's own rounding is 1.7e-3)
// from 64 bits.  g and u of an 8-bit checkpoint are formed from its codes and the
// scales (mm_core.hpp, kScaled), so that its rows are rounded to bf16 for dWgu alone,
// which is 2.9e-3 from 64 bits: there the scale changes along the sum, from token to
// token, and a second product with what the rounding leaves would be a quarter more
// operations.  (Rounded for all of them: 3.0e-3, 3.4e-3 and 3.3e-3 for dx, dWgu and
// dWd.  Scaling sums costs 1 to 5 %: 4093 tokens of 2048 through 1024 164 -> 170 us.)
// All sums are fp32 in a fixed order, and g and u that are computed again stay fp32.
//
// Bound by the matrix cores for prompts and training, by the weights' bytes and the
// launches' latency for few tokens.  bf16: 2501 tokens of 4096 through 2048 features
// 116 us (1.09 PFLOP/s), 4096 tokens 159 us (1.30); the gradient of 4096 tokens 370
// us (1.1; from an fp32 dout, into fp32 gradients of the weights 395), of which the product with the activation's gradient takes a quarter: its
// epilogue moves 84 MB that no other block's products hide.  Pre-activations
// computed again: 131 tokens of 2048 through 1024 29 us in three launches (five,
// product by product: 44 us), 4093 tokens from a checkpoint 167 to 175 us.
#include "moe_wq.h"
#include "mm_launch.hpp"

namespace moe {
namespace {
using namespace mm;

// h = silu(g) u, and the pre-activations where they are kept: bf16 for a caller,
// fp32 within a gradient (either null: not wanted).
struct GatedStore {
  uint16_t* h;
  void* gate_up;
  int gu_f32;
  int f;
  template <typename V>
  __device__ __forceinline__ void operator()(int m, int n, V g, V u) const {
    if (h) {
      V v;
#pragma unroll
      for (int r = 0; r < (int)(sizeof(V) / 4); ++r) v[r] = silu_f32(g[r]) * u[r];
      store_as(h, 0, (size_t)m * f + n, v);
    }
    if (gate_up) {
      const size_t at = (size_t)m * (2 * f) + n;
      store_as(gate_up, gu_f32, at, g);
      store_as(gate_up, gu_f32, at + f, u);
    }
  }
};

struct Store {
  void* out;
  long long N;
  int f32;
  template <typename V>
  __device__ __forceinline__ void operator()(int m, int n, V v) const {
    store_as(out, f32, (size_t)m * N + n, v);
  }
};

// dh -> dg, du and h of eight features.
__device__ __forceinline__ void gated_bwd(f32x8 dh, f32x8 g, f32x8 u, uint16_t* dgu, uint16_t* h,
                                          int m, int n, int f) {
  const size_t at = (size_t)m * (2 * f) + n;
  f32x8 dg, du, hv;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-g[r])), a = g[r] * s;
    du[r] = dh[r] * a;
    dg[r] = dh[r] * u[r] * (s + a * (1.0f - s));
    hv[r] = a * u[r];
  }
  store_as(dgu, 0, at, dg);
  store_as(dgu, 0, at + f, du);
  store_as(h, 0, (size_t)m * f + n, hv);
}

template <bool kGuF32>
struct GatedBwdStore {
  const void* gate_up;
  uint16_t* dgu;
  uint16_t* h;
  int f;
  struct Ahead {
    static constexpr int kRegs = kGuF32 ? 16 : 8;
    row::Raw8<kGuF32> g, u;
  };
  struct Columns {};
  __device__ __forceinline__ Columns columns(int) const { return {}; }
  __device__ __forceinline__ Ahead ahead(int m, int n) const {
    const size_t at = (size_t)m * (2 * f) + n;
    Ahead a;
    a.g.load(gate_up, at);
    a.u.load(gate_up, at + f);
    return a;
  }
  __device__ __forceinline__ void operator()(int m, int n, f32x8 dh, Columns,
                                             const Ahead& kept) const {
    gated_bwd(dh, kept.g.get(), kept.u.get(), dgu, h, m, n, f);
  }
};

// g and u of a block's tile in registers, for dh of the same tile.
template <int kR>
struct Kept {
  f32x8 g[kR], u[kR];
};
template <int kR>
struct KeepStore {
  static constexpr int kRounds = kR;
  Kept<kR>& kept;
  __device__ __forceinline__ void operator()(int, int, f32x8 g, f32x8 u, int round) const {
    kept.g[round] = g;
    kept.u[round] = u;
  }
};
template <int kR>
struct KeptBwdStore {
  static constexpr int kRounds = kR;
  const Kept<kR>& kept;
  uint16_t* dgu;
  uint16_t* h;
  int f;
  __device__ __forceinline__ void operator()(int m, int n, f32x8 dh, int round) const {
    gated_bwd(dh, kept.g[round], kept.u[round], dgu, h, m, n, f);
  }
};

// Gate, up and dh of a tile, one after the other in one block, so that the
// pre-activations that are computed again stay in registers.
template <typename ShG, typename ShH, bool kScaled>
__global__ __launch_bounds__(ShG::kThreads, ShG::kThreads / 256) void recompute_kernel(
    const Problem gu, const Problem dh, uint16_t* __restrict__ dgu, uint16_t* __restrict__ h,
    int f) {
  static_assert(ShG::BM == ShH::BM && ShG::BN == 2 * ShH::BN && ShG::WM == ShH::WM &&
                    ShG::WN == ShH::WN, "a thread's rows and columns are the same");
  constexpr int kWidth = ShH::BN / ShH::WN, kPass = 512 / kWidth < 16 ? 512 / kWidth : 16;
  constexpr int kR = ShG::BM / ShG::WM / 16 * ((16 + kPass - 1) / kPass);
  extern __shared__ __align__(1024) char lds[];
  Kept<kR> kept;
  product_block<Bf16, ShG, false, false, true, kScaled>(gu, KeepStore<kR>{kept}, lds, blockIdx.x,
                                                        0);
  __syncthreads();  // every wave's rows are turned around
  product_block<Bf16, ShH, false, true, false, false>(dh, KeptBwdStore<kR>{kept, dgu, h, f}, lds,
                                                      blockIdx.x, 0);
}

// dh -> dg, du and h where dh and the pre-activations come from one launch; eight
// values a thread.
__global__ __launch_bounds__(256) void gated_bwd_kernel(const float* __restrict__ dh, int T,
                                                        const GatedBwdStore<true> epi) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const int per = epi.f / 8;
  if (i >= (long long)T * per) return;
  const int m = (int)(i / per), n = 8 * (int)(i % per);
  epi(m, n, load_f32<f32x8>(dh, 8 * (size_t)i), {}, epi.ahead(m, n));
}

// fp32 rows to bf16, eight values a thread.
__global__ __launch_bounds__(256) void to_bf16_kernel(const float* __restrict__ x,
                                                      long long chunks,
                                                      uint16_t* __restrict__ out) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= chunks) return;
  store_as(out, 0, 8 * (size_t)i, load_f32<f32x8>(x, 8 * (size_t)i));
}

size_t round_up(size_t n) { return (n + 255) & ~(size_t)255; }
int stages_of(int k) { return (int)up(2LL * k, kStageBytes); }

Operand rows(const void* p, int stride, int n) {
  return {(const char*)p, nullptr, 2LL * stride, n};
}

// The gate and up rows of Wgu, in pairs.
Operand pairs(const uint16_t* w, int d, int f) {
  return {(const char*)w, (const char*)(w + (size_t)f * d), 2LL * d, f};
}

}  // namespace

size_t gated_ffn_ws_bytes(int T, int d, int f) {
  return round_up(2 * (size_t)T * f);
}

hipError_t launch_gated_ffn(const uint16_t* x, const uint16_t* w_gate_up, const uint16_t* w_down,
                            int T, int d, int f, void* out, int out_f32, uint16_t* gate_up,
                            void* ws, hipStream_t s) {
  uint16_t* h = (uint16_t*)ws;
  const hipError_t e = launch_product<Bf16, kInner, true>(
      rows(x, d, T), pairs(w_gate_up, d, f), T, f, d, 2, GatedStore{h, gate_up, 0, f}, nullptr, s);
  if (e != hipSuccess) return e;
  return launch_product<Bf16, kInner, false>(rows(h, f, T), rows(w_down, f, d), T, d, f, 2,
                                             Store{out, d, out_f32}, nullptr, s);
}

namespace {

template <int kTile>
using Tile = std::integral_constant<int, kTile>;

// The gradient's launches of several products.  dx and both weights' gradients:
const JointTiles kGradients[] = {
    {7, 6, 0.2f, "joint 32x64 64x64"},  {6, 5, 0.2f, "joint 64x64 64x128"},
    {5, 6, 0.2f, "joint 64x128 64x64"}, {5, 5, 0.2f, "joint 64x128 64x128"},
    {4, 4, 0.2f, "joint 128x128 k2"},   {2, 2, 0.2f, "joint 128x256"},
    {0, 0, 0.2f, "joint 256x256"},      {8, 11, 0.5f, "joint 32x64 k4 128x128"}};
int plan_gradients(int T, int d, int f, bool dx, bool dw_gate_up, bool dw_down) {
  const JointItem items[] = {{kOuterB, dx ? T : 0, d, stages_of(2 * f)},
                             {kOuterBoth, dw_gate_up ? 2LL * f : 0, d, stages_of(T)},
                             {kOuterBoth, dw_down ? d : 0, f, stages_of(T)}};
  float us;
  return plan_joint(kGradients, items, 0.0f, &us);
}
// ... and the pre-activations computed again beside dh, which then goes to memory
// and through a kernel of its own (20 bytes a value at 4.5 TB/s).
constexpr int kJointChoices = 4;
const JointTiles kRecompute[kJointChoices] = {{7, 7, 0.2f, "joint 32x64"},
                                              {6, 6, 0.2f, "joint 64x64"},
                                              {5, 5, 0.2f, "joint 64x128"},
                                              {8, 8, 0.5f, "joint 32x64 k4"}};
// ... or gate, up and dh of a tile in one block (recompute_kernel), which adds the
// two sums' times up but leaves g, u and dh in registers.
struct FusedTiles {
  int bm, bn;  // bn: of gate and up
  float fixed, block, one[2], each[2];
  const char* name;
};
const FusedTiles kFused[] = {{128, 128, 2.7f, 1.9f, {0.63f, 0.37f}, {0.51f, 0.36f}, "fused 128x128"},
                             {64, 128, 3.2f, 0.6f, {0.40f, 0.27f}, {0.39f, 0.25f}, "fused 64x128"}};

// -1: one by one; of kRecompute; behind them of kFused.  Over 60 random sizes (30 to
// 8192 tokens) 0.2 % above the fastest and 4 % less of the gradient's time than
// without the fused kernels: 7114 tokens of 256 through 1824 133 us one by one, 102
// fused; 131 of 2048 through 1024 29 us jointly, 44 fused.
int plan_recompute(int T, int d, int f) {
  const JointItem items[] = {{kInner, T, 2LL * f, stages_of(d)}, {kOuterB, T, f, stages_of(d)}};
  float us;
  int best = plan_joint(kRecompute, items, 20.0f / 4.5e6f * T * f, &us);
  // (one by one g and u go to memory and back, half of it beside the products)
  if (best < 0) us += 8.0f / 4.5e6f * T * f;
  for (int c = 0; c < 2; ++c) {
    const FusedTiles& t = kFused[c];
    const float n = (float)up(up(T, t.bm) * up(2LL * f, t.bn), 256);
    float fused = t.fixed + t.block * n;
    for (int p = 0; p < 2; ++p) fused += stages_of(d) * std::max(t.one[p], t.each[p] * n);
    if (fused < us) {
      us = fused;
      best = kJointChoices + c;
    }
  }
  return best;
}

// Bytes of split sums of the weights' gradients.
size_t sums_bytes(int d, int f, int stages) {
  return std::max(partial_bytes(2LL * f, d, stages), partial_bytes(d, f, stages));
}

// Workspace of the gradient, in bytes from its start; again: plan_recompute's.
struct BwdSpace {
  size_t dgu, h, gate_up, x, whole, unit, dout, dh, part;
  BwdSpace(int T, int d, int f, int do_f32, int x_i8, int kept, int again) {
    size_t at = 0;
    auto take = [&](bool wanted, size_t values, size_t size = 2) {
      const size_t p = at;
      if (wanted) at += round_up(size * values);
      return p;
    };
    dgu = take(true, (size_t)T * 2 * f);
    h = take(true, (size_t)T * f);
    // fp32: not rounded on the way
    gate_up = take(!kept && again < kJointChoices, (size_t)T * 2 * f, 4);
    x = take(x_i8, (size_t)T * d);
    whole = take(x_i8 && !kept, (size_t)T * d);
    unit = take(x_i8 && !kept, (size_t)T * up(d, 128), 4);
    dout = take(do_f32, (size_t)T * d);
    dh = take(!kept && again >= 0 && again < kJointChoices, (size_t)T * f, 4);
    part = at;  // (the last)
  }
};

}  // namespace

const char* gated_ffn_kernel(int product, int T, int d, int f, bool all) {
  if (all && product <= MOE_GATED_DH) {
    const int c = plan_recompute(T, d, f);
    if (product != MOE_GATED_DOWN && c >= 0)
      return c < kJointChoices ? kRecompute[c].name : kFused[c - kJointChoices].name;
  } else if (all) {
    const int c = plan_gradients(T, d, f, true, true, true);
    if (c >= 0) return kGradients[c].name;
  }
  switch (product) {
    case MOE_GATED_GATE_UP: return product_name(kInner, false, T, f, d, 2LL * d, true);
    case MOE_GATED_DOWN: return product_name(kInner, false, T, d, f, 2LL * f, false);
    case MOE_GATED_DH: return product_name(kOuterB, false, T, f, d, 0, false);
    case MOE_GATED_DX: return product_name(kOuterB, false, T, d, 2LL * f, 0, false);
    case MOE_GATED_DW_GATE_UP: return product_name(kOuterBoth, false, 2LL * f, d, T, 0, false);
    case MOE_GATED_DW_DOWN: return product_name(kOuterBoth, false, d, f, T, 0, false);
  }
  return "";
}

size_t gated_ffn_bwd_ws_bytes(int T, int d, int f, int do_f32, int x_i8, int kept) {
  const int again = kept || T == 0 ? -1 : plan_recompute(T, d, f);
  return BwdSpace(T, d, f, do_f32, x_i8, kept, again).part + sums_bytes(d, f, stages_of(T));
}

size_t gated_ffn_bwd_ws_most(int T, int d, int f, int do_f32, int x_i8, int kept) {
  size_t most = 0, sums = 0;
  auto bytes = [&](int t, int again) { return BwdSpace(t, d, f, do_f32, x_i8, kept, again).part; };
  // Every tile's rows are a multiple of 32, so over 32 tokens only the costs of what
  // goes to memory grow: the choice goes from a joint launch, which takes the most, to
  // one by one and to a fused kernel, which takes nothing more.
  for (int t = T, step = 1; t > 0 && bytes(t, 0) > most; t -= step) {
    const int first = (t - 1) / 32 * 32 + 1, again = kept ? -1 : plan_recompute(t, d, f);
    most = std::max(most, bytes(t, again));
    if (t == T || t % 32 == 0) {
      const int least = kept ? -1 : plan_recompute(first, d, f);
      step = bytes(t, least) > bytes(t, again) ? 1 : t - first + 1;
    }
  }
  const size_t one = 4 * (size_t)(2 * f) * d;  // a split's sums, at most
  // (so many splits at most of n stages, and of fewer)
  for (int n = stages_of(T); splits_most(n) > 1 && splits_most(n) * one > sums; --n)
    sums = std::max(sums, sums_bytes(d, f, n));
  return most + sums;
}

hipError_t launch_gated_ffn_bwd(const GatedBwdArgs& a, void* ws, hipStream_t s) {
  const int T = a.T, d = a.d, f = a.f;
  const int again = a.gate_up || T == 0 ? -1 : plan_recompute(T, d, f);
  const BwdSpace at(T, d, f, a.do_f32, a.x_scales != nullptr, a.gate_up != nullptr, again);
  auto place = [&](size_t p) { return (uint16_t*)((char*)ws + p); };
  uint16_t *dgu = place(at.dgu), *h = place(at.h);
  void* part = place(at.part);
  const uint16_t* x = (const uint16_t*)a.x;
  const uint16_t* dout = (const uint16_t*)a.dout;
  hipError_t e = hipSuccess;
  if (T > 0) {
    if (a.do_f32) {
      const long long chunks = (long long)T * (d / 8);
      hipLaunchKernelGGL(to_bf16_kernel, dim3((uint32_t)up(chunks, 256)), dim3(256), 0, s,
                         (const float*)a.dout, chunks, place(at.dout));
      if ((e = hipGetLastError()) != hipSuccess) return e;
      dout = place(at.dout);
    }
    Operand tokens = rows(x, d, T);  // of gate and up
    if (a.x_scales && (!a.gate_up || a.dw_gate_up)) {
      uint16_t *whole = a.gate_up ? nullptr : place(at.whole),
               *restored = a.dw_gate_up ? place(at.x) : nullptr;
      float* unit = (float*)place(at.unit);
      e = launch_unpack_i8((const int8_t*)a.x, a.x_scales, T, d, whole, unit, restored, s);
      if (e != hipSuccess) return e;
      tokens = {(const char*)whole, nullptr, 2LL * d, T, unit};
      x = restored;
    }
    // the choice's call of a kernel whose tokens are an 8-bit checkpoint's, or not
    auto by_tokens = [&](auto call) {
      return a.x_scales ? call(std::true_type{}) : call(std::false_type{});
    };
    const Operand m = rows(dout, d, T), w = rows(a.w_down, f, f);
    if (again >= kJointChoices) {
      auto go = [&](auto shape_g, auto shape_h) {
        typedef decltype(shape_g) G;
        typedef decltype(shape_h) H;
        const Problem gu =
            part_of<G, kInner, true>(tokens, pairs(a.w_gate_up, d, f), T, f, d, 0).p;
        const Problem dh = part_of<H, kOuterB, false>(m, w, T, f, d, 0).p;
        return by_tokens([&](auto scaled) {
          hipLaunchKernelGGL((recompute_kernel<G, H, decltype(scaled)::value>),
                             dim3(gu.nm * gu.nn), dim3(G::kThreads), std::max(G::kLds, H::kLds), s,
                             gu, dh, dgu, h, f);
          return hipGetLastError();
        });
      };
      if (again == kJointChoices)  // (as kFused has them)
        e = go(Shape<128, 128, 2, 2, 2, 1, 1>{}, Shape<128, 64, 2, 2, 2, 1, 1>{});
      else
        e = go(Shape<64, 128, 2, 2, 3>{}, Shape<64, 64, 2, 2, 3>{});
    } else if (again >= 0) {
      auto go = [&](auto tile) {
        typedef typename TileShape<decltype(tile)::value>::Type Sh;
        const auto dh = part_of<Sh, kOuterB, false>(m, w, T, f, d, Store{place(at.dh), f, 1});
        auto none = dh;
        none.blocks = 0;
        return by_tokens([&](auto scaled) {
          const auto gu = part_of<Sh, kInner, true, decltype(scaled)::value>(
              tokens, pairs(a.w_gate_up, d, f), T, f, d,
              GatedStore{nullptr, place(at.gate_up), 1, f});
          return launch_joint(gu, dh, none, s);
        });
      };
      switch (again) {  // (as kRecompute has them)
        case 0: e = go(Tile<7>{}); break;
        case 1: e = go(Tile<6>{}); break;
        case 2: e = go(Tile<5>{}); break;
        case 3: e = go(Tile<8>{}); break;
      }
      if (e != hipSuccess) return e;
      hipLaunchKernelGGL(gated_bwd_kernel, dim3((uint32_t)up((long long)T * (f / 8), 256)),
                         dim3(256), 0, s, (const float*)place(at.dh), T,
                         GatedBwdStore<true>{place(at.gate_up), dgu, h, f});
      e = hipGetLastError();
    } else if (a.gate_up) {
      e = launch_product<Bf16, kOuterB, false>(
          m, w, T, f, d, 2, GatedBwdStore<false>{a.gate_up, dgu, h, f}, nullptr, s);
    } else {
      e = by_tokens([&](auto scaled) {
        return launch_product<Bf16, kInner, true, decltype(scaled)::value>(
            tokens, pairs(a.w_gate_up, d, f), T, f, d, 2,
            GatedStore{nullptr, place(at.gate_up), 1, f}, nullptr, s);
      });
      if (e != hipSuccess) return e;
      e = launch_product<Bf16, kOuterB, false>(
          m, w, T, f, d, 2, GatedBwdStore<true>{place(at.gate_up), dgu, h, f}, nullptr, s);
    }
    if (e != hipSuccess) return e;
    const int joint = plan_gradients(T, d, f, a.dx, a.dw_gate_up, a.dw_down);
    if (joint >= 0) {
      auto go = [&](auto tile_x, auto tile_w) {
        typedef typename TileShape<decltype(tile_x)::value>::Type ShX;
        typedef typename TileShape<decltype(tile_w)::value>::Type ShW;
        auto dx = part_of<ShX, kOuterB, false>(rows(dgu, 2 * f, T), rows(a.w_gate_up, d, d), T, d,
                                               2 * f, Store{a.dx, d, 0});
        auto wu = part_of<ShW, kOuterBoth, false>(rows(dgu, 2 * f, 2 * f), rows(x, d, d), 2 * f, d,
                                                  T, Store{a.dw_gate_up, d, a.dw_f32});
        auto wd = part_of<ShW, kOuterBoth, false>(rows(dout, d, d), rows(h, f, f), d, f, T,
                                                  Store{a.dw_down, f, a.dw_f32});
        if (!a.dx) dx.blocks = 0;
        if (!a.dw_gate_up) wu.blocks = 0;
        if (!a.dw_down) wd.blocks = 0;
        return launch_joint(dx, wu, wd, s);
      };
      switch (joint) {  // (as kGradients has them)
        case 0: return go(Tile<7>{}, Tile<6>{});
        case 1: return go(Tile<6>{}, Tile<5>{});
        case 2: return go(Tile<5>{}, Tile<6>{});
        case 3: return go(Tile<5>{}, Tile<5>{});
        case 4: return go(Tile<4>{}, Tile<4>{});
        case 5: return go(Tile<2>{}, Tile<2>{});
        case 6: return go(Tile<0>{}, Tile<0>{});
        case 7: return go(Tile<8>{}, Tile<11>{});
      }
    }
    if (a.dx) {
      e = launch_product<Bf16, kOuterB, false>(rows(dgu, 2 * f, T), rows(a.w_gate_up, d, d), T,
                                               d, 2 * f, 2, Store{a.dx, d, 0}, nullptr, s);
      if (e != hipSuccess) return e;
    }
  }
  if (a.dw_gate_up) {
    e = launch_product<Bf16, kOuterBoth, false>(rows(dgu, 2 * f, 2 * f), rows(x, d, d), 2 * f, d, T,
                                                2, Store{a.dw_gate_up, d, a.dw_f32}, part, s);
    if (e != hipSuccess) return e;
  }
  if (a.dw_down)
    e = launch_product<Bf16, kOuterBoth, false>(rows(dout, d, d), rows(h, f, f), d, f, T, 2,
                                                Store{a.dw_down, f, a.dw_f32}, part, s);
  return e;
}

}  // namespace moe
