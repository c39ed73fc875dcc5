// Host side of the matrix products: the kernel and the split of k by the
// product's size, launch, and the join of split sums.
#pragma once
#include <algorithm>

#include "launch.hpp"
#include "mm_direct.hpp"

namespace moe {
namespace mm {

// Which operands have k across their rows: none, B (x W with W [k][n]), both (a
// sum over tokens).
enum Layout { kInner, kOuterB, kOuterBoth };

template <Layout kL, int bm, int bn, int wm, int wn, int stages, int groups = 1>
using ShapeOf = std::conditional_t<kL == kOuterBoth && (bm == 192 || bm == 32), void,
                                   Shape<bm, bn, wm, wn, stages, groups>>;

// The tiled kernels, and what a product takes: 3 us and, for each 128 bytes (or
// 64 rows) of k, the larger of `one` (latency of a stage: a block alone on a CU)
// and `each` for every block a CU gets.  us, fitted to 130 products of 24 to
// 4096 rows, 1000 to 12288 columns and k 1000 to 4096 on the whole chip.
struct TileCost {
  int bm, bn;
  float one[3], each[3];  // by Layout; 0: not built for it
  const char* name;
};
constexpr int kTileKernels = 9;
const TileCost kTileCosts[kTileKernels] = {
    {256, 256, {1.35f, 1.75f, 1.75f}, {1.60f, 1.75f, 1.75f}, "tile 256x256"},
    {192, 256, {1.15f, 1.45f, 0}, {1.30f, 1.45f, 0}, "tile 192x256"},
    {128, 128, {0.62f, 0.97f, 0.97f}, {0.50f, 0.52f, 0.55f}, "tile 128x128"},
    {128, 128, {0.60f, 0.76f, 0.76f}, {0.60f, 0.76f, 0.76f}, "tile 128x128 k2"},
    {64, 128, {0.43f, 0.80f, 0}, {0.33f, 0.43f, 0}, "tile 64x128"},
    {64, 64, {0.36f, 0.69f, 0.69f}, {0.21f, 0.30f, 0.30f}, "tile 64x64"},
    {64, 64, {0, 0.37f, 0.37f}, {0, 0.52f, 0.52f}, "tile 64x64 k4"},
    {32, 64, {0.24f, 0.33f, 0}, {0.165f, 0.31f, 0}, "tile 32x64"},
    {32, 32, {0.15f, 0, 0}, {0.115f, 0, 0}, "tile 32x32 k2"},
};

inline long long up(long long a, long long b) { return (a + b - 1) / b; }

struct Plan {
  int tile;    // of kTileCosts
  int splits;  // blocks that share a tile's k (both operands outer: k is long)
  int per;     // stages a block
};

// M rows and N columns (of B, so 2 f of the pair form), `stages` of k.
inline Plan plan_product(Layout l, long long M, long long N, int stages) {
  constexpr int kCUs = 256;
  Plan best = {0, 1, stages};
  float least = 1e30f;
  for (int t = 0; t < kTileKernels; ++t) {
    const TileCost& c = kTileCosts[t];
    if (c.one[l] == 0) continue;
    const long long tiles = up(M, c.bm) * up(N, c.bn);
    for (int k = 1; k <= (l == kOuterBoth ? 16 : 1); k *= 2) {
      if (k > 1 && stages / k < 8) break;
      const int per = std::max((int)up(stages, k), 1), n = std::max((int)up(stages, per), 1);
      const float us = per * std::max(c.one[l], c.each[l] * up(tiles * n, kCUs)) +
                       // a second launch, and the sums written and read (4 TB/s)
                       (n > 1 ? 4.0f + 2.0e-6f * n * M * N : 0.0f);
      if (us < least) {
        least = us;
        best = {t, n, per};
      }
    }
  }
  return best;
}

// Workspace of a product over tokens (both operands outer).
inline size_t partial_bytes(long long M, long long N, int stages) {
  const Plan p = plan_product(kOuterBoth, M, N, stages);
  return p.splits > 1 ? (size_t)p.splits * M * N * 4 : 0;
}

// A split's sums.
struct StorePartial {
  float* ws;
  long long M, N;
  __device__ __forceinline__ void operator()(int m, int n, f32x4 v) const {
    *(f32x4*)(ws + ((size_t)blockIdx.y * M + m) * N + n) = v;
  }
};

// The splits' sums in their order, and the epilogue; four columns a thread.
template <typename Epi>
__global__ __launch_bounds__(256) void join_kernel(const float* __restrict__ ws, long long M,
                                                   long long N, int splits, const Epi epi) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x, nq = N / 4;
  if (i >= M * nq) return;
  const int m = (int)(i / nq), n = 4 * (int)(i % nq);
  const float* p = ws + (size_t)m * N + n;
  f32x4 v = *(const f32x4*)p;
  for (int s = 1; s < splits; ++s) v += *(const f32x4*)(p + (size_t)s * M * N);
  epi(m, n, v);
}

template <typename Mma, typename Sh, Layout kL, bool kPair, typename Epi>
inline void launch_shape(Problem p, const Plan& plan, const Epi& epi, hipStream_t s) {
  if constexpr (!std::is_void_v<Sh>) {
    p.nm = (int)up(p.M, Sh::BM);
    p.nn = (int)up(kPair ? 2LL * p.N : p.N, Sh::BN);
    p.per_group = (int)up(plan.per, Sh::G);
    hipLaunchKernelGGL((product_kernel<Mma, Sh, kL == kOuterBoth, kL != kInner, kPair, Epi>),
                       dim3(p.nm * p.nn, plan.splits), dim3(Sh::kThreads), Sh::kLds, s, p, epi);
  }
}

template <typename Mma, Layout kL, bool kPair, typename Epi>
inline void launch_tiles(const Problem& p, const Plan& plan, const Epi& epi, hipStream_t s) {
  auto go = [&](auto* shape) {
    launch_shape<Mma, std::remove_pointer_t<decltype(shape)>, kL, kPair>(p, plan, epi, s);
  };
  constexpr bool kOuter = kL != kInner, kSlim = kL != kOuterBoth;
  switch (plan.tile) {
    case 0: return go((ShapeOf<kL, 256, 256, 2, 4, 2>*)nullptr);
    case 1: return go((ShapeOf<kL, 192, 256, 2, 4, 2>*)nullptr);
    case 2: return go((ShapeOf<kL, 128, 128, 2, 2, 2>*)nullptr);
    case 3: return go((ShapeOf<kL, 128, 128, 2, 2, 2, 2>*)nullptr);
    case 4:
      if constexpr (kSlim) return go((ShapeOf<kL, 64, 128, 1, 4, 3>*)nullptr);
      return;
    case 5: return go((ShapeOf<kL, 64, 64, 2, 2, 3>*)nullptr);
    case 6:
      if constexpr (kOuter) return go((ShapeOf<kL, 64, 64, 2, 2, 2, 4>*)nullptr);
      return;
    case 7:
      if constexpr (kOuter)
        return go((ShapeOf<kL, 32, 64, 2, 2, 3, 4>*)nullptr);
      else
        return go((ShapeOf<kL, 32, 64, 2, 2, 4>*)nullptr);
    case 8:
      if constexpr (!kOuter) return go((ShapeOf<kL, 32, 32, 2, 1, 4, 2>*)nullptr);
      return;
  }
}

// C = A B^T with the epilogue; k values a row.  ws: partial_bytes of it (both
// operands outer).
template <typename Mma, Layout kL, bool kPair, typename Epi>
inline hipError_t launch_product(const Operand& a, const Operand& b, int M, int N, int k,
                                 int elem_bytes, const Epi& epi, void* ws, hipStream_t s) {
  Problem p{};
  p.a = a;
  p.b = b;
  p.M = M;
  p.N = N;
  p.kbytes = k * elem_bytes;
  p.krows = k;
  p.stages = (int)up((long long)k * elem_bytes, kStageBytes);
  if constexpr (kL == kInner) {
    if (direct_applies(M, N, b.stride, kPair))
      return launch_direct<Mma, kPair, false>({a.p, b.p, a.stride, b.stride, M, N, p.kbytes, 0},
                                              epi, s);
  }
  const Plan plan = plan_product(kL, M, kPair ? 2LL * N : N, p.stages);
  if constexpr (kL == kOuterBoth) {
    if (plan.splits > 1) {
      launch_tiles<Mma, kL, kPair>(p, plan, StorePartial{(float*)ws, M, N}, s);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      hipLaunchKernelGGL((join_kernel<Epi>), dim3((uint32_t)up((long long)M * (N / 4), 256)),
                         dim3(256), 0, s, (const float*)ws, (long long)M, (long long)N,
                         plan.splits, epi);
      return hipGetLastError();
    }
  }
  launch_tiles<Mma, kL, kPair>(p, plan, epi, s);
  return hipGetLastError();
}

}  // namespace mm
}  // namespace moe
