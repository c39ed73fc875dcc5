// Host side of the matrix products: the kernel and the split of k by the
// product's size, launch, and the join of split sums.
#pragma once
#include <algorithm>
#include <utility>

#include "launch.hpp"
#include "mm_direct.hpp"

namespace moe {
namespace mm {

// Which operands have k across their rows: none, B (x W with W [k][n]), both (a
// sum over tokens).
enum Layout { kInner, kOuterB, kOuterBoth };

// The tiled kernels: what a product takes on the whole chip, in us, is
//   fixed + block * n + stages * max(one, each * n)
// for n blocks a CU and stages of 128 bytes (or 64 rows) of k; one: the latency
// of a stage where a block is alone on its CU, each: its share of a full CU.
// Fitted by kind of product to 140 to 180 random sizes each (1 to 8192 rows, 64
// to 50304 columns, k 8 to 8192); on 70 others of each kind the choice took 0.2 to
// 0.7 % longer than the fastest tile on average, 12 % at most
// (profiles/product_choice.txt).
struct TileCost {
  int bm, bn;
  struct {
    float fixed, block, one, each;  // all 0: not built
  } of[4];  // inner bf16, inner int8, outer B, both outer
  const char* name;  // behind the prefix of one whose k is split over blocks
};
constexpr int kSplitPrefix = 6;  // "split "
constexpr int kTileKernels = 11;  // and one behind them for launches of several products
const TileCost kTileCosts[kTileKernels + 1] = {
    {256, 256,
     {{0.0f, 7.0f, 1.48f, 1.43f}, {0.0f, 8.5f, 1.17f, 1.22f}, {0.0f, 6.9f, 0.20f, 1.22f},
      {0.0f, 9.0f, 0.46f, 1.18f}},
     "split tile 256x256"},
    {192, 256,
     {{0.0f, 6.5f, 1.21f, 1.17f}, {0.0f, 7.1f, 0.32f, 1.08f}, {0.0f, 6.1f, 0.23f, 0.94f}, {}},
     "split tile 192x256"},
    {128, 256,
     {{}, {0.0f, 5.7f, 0.89f, 0.90f}, {0.0f, 5.0f, 0.03f, 0.73f}, {0.0f, 6.3f, 0.79f, 0.80f}},
     "split tile 128x256"},
    {128, 128,
     {{2.6f, 1.5f, 0.63f, 0.51f}, {0.9f, 3.5f, 0.56f, 0.53f}, {}, {2.3f, 2.8f, 0.59f, 0.51f}},
     "split tile 128x128"},
    {128, 128,
     {{1.6f, 4.0f, 0.27f, 0.56f}, {0.0f, 5.6f, 0.49f, 0.52f}, {0.0f, 5.4f, 0.44f, 0.46f},
      {0.0f, 6.6f, 0.45f, 0.47f}},
     "split tile 128x128 k2"},
    {64, 128,
     {{3.2f, 0.78f, 0.38f, 0.37f}, {2.3f, 1.7f, 0.08f, 0.38f}, {2.7f, 0.94f, 0.37f, 0.36f},
      {2.7f, 1.8f, 0.43f, 0.38f}},
     "split tile 64x128"},
    {64, 64,
     {{3.2f, 0.36f, 0.26f, 0.24f}, {2.9f, 0.70f, 0.25f, 0.25f}, {3.1f, 0.21f, 0.29f, 0.26f},
      {2.8f, 0.89f, 0.36f, 0.27f}},
     "split tile 64x64"},
    {32, 64,
     {{3.1f, 0.34f, 0.19f, 0.17f}, {3.1f, 0.47f, 0.15f, 0.17f}, {2.8f, 0.46f, 0.26f, 0.20f}, {}},
     "split tile 32x64"},
    {32, 64,
     {{1.7f, 2.8f, 0.02f, 0.17f}, {}, {0.8f, 3.7f, 0.17f, 0.18f}, {}},
     "split tile 32x64 k4"},
    {32, 32, {{2.6f, 0.85f, 0.12f, 0.10f}, {2.8f, 0.91f, 0.10f, 0.09f}, {}, {}}, "split tile 32x32 k2"},
    {160, 256,
     {{0.0f, 5.9f, 1.09f, 1.05f}, {0.0f, 6.6f, 0.95f, 0.96f}, {0.0f, 5.7f, 0.80f, 0.80f}, {}},
     "split tile 160x256"},
    {128, 128, {{}, {}, {}, {1.5f, 3.1f, 0.75f, 0.61f}}, "split tile 128x128 w16"},
};

inline long long up(long long a, long long b) { return (a + b - 1) / b; }

struct Plan {
  int tile;    // of kTileCosts
  int splits;  // blocks that share a tile's k (both operands outer: k is long)
  int per;     // stages a block
  float us;    // what it takes
};

// Blocks that may share so many stages of k: 16, of eight stages each or more.
inline int splits_most(int stages) { return std::min(16, std::max(1, stages / 8)); }

// M rows and N columns (of B, so 2 f of the pair form), `stages` of k.  scaled: A's
// rows have units: tiles of 32 rows are left out (a joint launch is faster where they
// would be chosen).
inline Plan plan_product(Layout l, bool i8, long long M, long long N, int stages,
                         bool scaled = false) {
  constexpr int kCUs = 256;
  const int kind = l == kInner ? i8 : l == kOuterB ? 2 : 3;
  Plan best = {0, 1, stages, 1e30f};
  for (int t = 0; t < kTileKernels; ++t) {
    const auto& c = kTileCosts[t].of[kind];
    if (c.one == 0 || (scaled && kTileCosts[t].bm == 32)) continue;
    const long long tiles = up(M, kTileCosts[t].bm) * up(N, kTileCosts[t].bn);
    for (int k = 1; k <= (l == kOuterBoth ? splits_most(stages) : 1); k *= 2) {
      const int per = std::max((int)up(stages, k), 1), splits = std::max((int)up(stages, per), 1);
      const float n = (float)up(tiles * splits, kCUs);
      const float us = c.fixed + c.block * n + per * std::max(c.one, c.each * n) +
                       // a second launch, and the sums written and read (4 TB/s)
                       (splits > 1 ? 4.0f + 2.0e-6f * splits * M * N : 0.0f);
      if (us < best.us) best = {t, splits, per, us};
    }
  }
  return best;
}

// The kernel that a product runs: "direct", a tile's name, "split ..".
inline const char* product_name(Layout l, bool i8, long long M, long long N, long long k,
                                long long b_stride, bool pair) {
  if (l == kInner && direct_applies(M, N, b_stride, pair)) return "direct";
  const Plan p = plan_product(l, i8, M, pair ? 2 * N : N, (int)up(k * (i8 ? 1 : 2), kStageBytes));
  return kTileCosts[p.tile].name + (p.splits > 1 ? 0 : kSplitPrefix);
}

// Workspace of a product over tokens (both operands outer).
inline size_t partial_bytes(long long M, long long N, int stages) {
  const Plan p = plan_product(kOuterBoth, false, M, N, stages);
  return p.splits > 1 ? (size_t)p.splits * M * N * 4 : 0;
}

// A split's sums.
struct StorePartial {
  float* ws;
  long long M, N;
  template <typename V>
  __device__ __forceinline__ void operator()(int m, int n, V v) const {
    store_as(ws, 1, ((size_t)blockIdx.y * M + m) * N + n, v);
  }
};

// The splits' sums in their order, and the epilogue; eight columns a thread.
template <typename Epi>
__global__ __launch_bounds__(256) void join_kernel(const float* __restrict__ ws, long long M,
                                                   long long N, int splits, const Epi epi) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x, per = N / 8;
  if (i >= M * per) return;
  const int m = (int)(i / per), n = 8 * (int)(i % per);
  const size_t at = (size_t)m * N + n;
  f32x8 v = row::load8<true>(ws, at);
  for (int s = 1; s < splits; ++s) v += row::load8<true>(ws, at + (size_t)s * M * N);
  epi(m, n, v);
}

template <typename Mma, Layout kL, bool kPair, bool kScaled, typename Epi, int... kShape>
inline void launch_shape(Problem p, const Plan& plan, const Epi& epi, hipStream_t s,
                         std::integer_sequence<int, kShape...>) {
  typedef Shape<kShape...> Sh;
  p.nm = (int)up(p.M, Sh::BM);
  p.nn = (int)up(kPair ? 2LL * p.N : p.N, Sh::BN);
  p.per_group = (int)up(plan.per, Sh::G);
  hipLaunchKernelGGL((product_kernel<Mma, Sh, kL == kOuterBoth, kL != kInner, kPair, kScaled, Epi>),
                     dim3(p.nm * p.nn, plan.splits), dim3(Sh::kThreads), Sh::kLds, s, p, epi);
}

template <typename Mma, Layout kL, bool kPair, bool kScaled, typename Epi>
inline void launch_tiles(const Problem& p, const Plan& plan, const Epi& epi, hipStream_t s) {
  auto go = [&](auto shape) { launch_shape<Mma, kL, kPair, kScaled>(p, plan, epi, s, shape); };
  using std::integer_sequence;
  constexpr bool kIn = kL == kInner, kB = kL == kOuterB, kBoth = kL == kOuterBoth;
  switch (plan.tile) {  // (as kTileCosts has them)
    case 0: return go(integer_sequence<int, 256, 256, 2, 4, 2, 1, 1>{});
    case 1:
      if constexpr (!kBoth) go(integer_sequence<int, 192, 256, 2, 4, 2, 1, 1>{});
      return;
    case 2:
      if constexpr (!kIn || std::is_same_v<Mma, I8>)
        go(integer_sequence<int, 128, 256, 2, 4, 2, 1, 1>{});
      return;
    case 3:
      if constexpr (!kB) go(integer_sequence<int, 128, 128, 2, 2, 2, 1, 1>{});
      return;
    case 4: return go(integer_sequence<int, 128, 128, 2, 2, 2, 2, 1>{});
    case 5: return go(integer_sequence<int, 64, 128, 1, 4, 3>{});
    case 6: return go(integer_sequence<int, 64, 64, 2, 2, 3>{});
    case 7:
      if constexpr (!kBoth && !kScaled) go(integer_sequence<int, 32, 64, 2, 2, 4>{});
      return;
    case 8:
      if constexpr (kB || (kIn && !kScaled && std::is_same_v<Mma, Bf16>))
        go(integer_sequence<int, 32, 64, 2, 2, 3, 4>{});
      return;
    case 9:
      if constexpr (kIn && !kScaled) go(integer_sequence<int, 32, 32, 2, 1, 4, 2>{});
      return;
    case 10:
      if constexpr (!kBoth) go(integer_sequence<int, 160, 256, 2, 4, 2, 1, 1>{});
      return;
  }
}

inline Problem problem_of(const Operand& a, const Operand& b, int M, int N, int k,
                          int elem_bytes) {
  Problem p{};
  p.a = a;
  p.b = b;
  p.M = M;
  p.N = N;
  p.kbytes = k * elem_bytes;
  p.krows = k;
  p.stages = (int)up((long long)k * elem_bytes, kStageBytes);
  return p;
}

// C = A B^T with the epilogue; k values a row.  ws: partial_bytes of it (both
// operands outer).
template <typename Mma, Layout kL, bool kPair, bool kScaled = false, typename Epi>
inline hipError_t launch_product(const Operand& a, const Operand& b, int M, int N, int k,
                                 int elem_bytes, const Epi& epi, void* ws, hipStream_t s) {
  const Problem p = problem_of(a, b, M, N, k, elem_bytes);
  if constexpr (kL == kInner && !kScaled) {
    if (direct_applies(M, N, b.stride, kPair))
      return launch_direct<Mma, kPair, false>({a.p, b.p, a.stride, b.stride, M, N, p.kbytes, 0},
                                              epi, s);
  }
  const Plan plan =
      plan_product(kL, std::is_same_v<Mma, I8>, M, kPair ? 2LL * N : N, p.stages, kScaled);
  if constexpr (kL == kOuterBoth) {
    if (plan.splits > 1) {
      launch_tiles<Mma, kL, kPair, kScaled>(p, plan, StorePartial{(float*)ws, M, N}, s);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      hipLaunchKernelGGL((join_kernel<Epi>), dim3((uint32_t)up((long long)M * (N / 8), 256)),
                         dim3(256), 0, s, (const float*)ws, (long long)M, (long long)N,
                         plan.splits, epi);
      return hipGetLastError();
    }
  }
  launch_tiles<Mma, kL, kPair, kScaled>(p, plan, epi, s);
  return hipGetLastError();
}

// ------------------------------------------------ several products a launch
// Products that do not wait for each other share a launch where that is faster:
// the blocks of one run where another leaves CUs idle, and a launch is saved.
// The first product has one tile, the others have another; both by cost:
//   max(longest, work) + overlap * min(longest, work)
// with the longest block's time alone on a CU, and all blocks' shares of a full
// CU over the 256 CUs; overlap 0.2, or 0.5 where a block has its CU to itself and
// is there for few blocks with a long k (the gradient of 1 token, d 896, f 1952 28.3 us
// with tiles of four waves, 25.1 with 16; 131, 2048, 1024: 29.9 and 31.0); one by one they take
// the sum of their plans.  Over 80 random sizes of a gradient (1 to 8192 tokens,
// 128 to 4096 values) the choice took 1.6 % longer than the best and 26 % less than
// one by one; 5000 tokens of 2560 through 2560 features 350 us together and 385 us
// one by one, 4096 of 4096 through 2048, which 256 blocks a product fill evenly, 382
// and 369 us (profiles/product_choice.txt).
struct JointTiles {
  int first, second;  // of kTileCosts
  float overlap;
  const char* name;
};
struct JointItem {
  Layout l;
  long long M, N;  // N: of the tile grid; M = 0: not wanted
  int stages;
};

// Which of the choices of tiles, or -1: one by one; *took: the time.  extra: us
// that a joint launch costs beside it.
template <int kChoices, int kItems>
inline int plan_joint(const JointTiles (&choices)[kChoices], const JointItem (&items)[kItems],
                      float extra, float* took) {
  float apart = 0.0f, best_us = 1e30f;
  int best = -1, wanted = 0;
  for (const JointItem& it : items) {
    if (!it.M) continue;
    ++wanted;
    apart += plan_product(it.l, false, it.M, it.N, it.stages).us;
  }
  *took = apart;
  if (wanted < 2) return -1;
  for (int c = 0; c < kChoices; ++c) {
    float longest = 0.0f, work = 0.0f, fixed = 0.0f;
    for (int i = 0; i < kItems; ++i) {
      const JointItem& it = items[i];
      if (!it.M) continue;
      const TileCost& t = kTileCosts[i ? choices[c].second : choices[c].first];
      const auto& us = t.of[it.l == kInner ? 0 : it.l == kOuterB ? 2 : 3];
      const float blocks = (float)(up(it.M, t.bm) * up(it.N, t.bn));
      fixed = std::max(fixed, us.fixed);
      longest = std::max(longest, us.block + it.stages * std::max(us.one, us.each));
      work += blocks * (us.block + it.stages * us.each) / 256;
    }
    const float us = fixed + extra + std::max(longest, work) +
                     choices[c].overlap * std::min(longest, work);
    if (us < best_us) {
      best_us = us;
      best = c;
    }
  }
  if (best_us >= apart) return -1;
  *took = best_us;
  return best;
}

// (as kTileCosts has them)
template <int kTile>
struct TileShape;
template <> struct TileShape<0> { typedef Shape<256, 256, 2, 4, 2, 1, 1> Type; };
template <> struct TileShape<2> { typedef Shape<128, 256, 2, 4, 2, 1, 1> Type; };
template <> struct TileShape<4> { typedef Shape<128, 128, 2, 2, 2, 2, 1> Type; };
template <> struct TileShape<5> { typedef Shape<64, 128, 1, 4, 3> Type; };
template <> struct TileShape<6> { typedef Shape<64, 64, 2, 2, 3> Type; };
template <> struct TileShape<7> { typedef Shape<32, 64, 2, 2, 4> Type; };
template <> struct TileShape<8> { typedef Shape<32, 64, 2, 2, 3, 4> Type; };
template <> struct TileShape<11> { typedef Shape<128, 128, 4, 4, 2> Type; };

// A product as a part of a launch.
template <typename Sh, Layout kL, bool kPair, bool kScaled = false, typename Epi>
inline auto part_of(const Operand& a, const Operand& b, int M, int N, int k, const Epi& epi) {
  Part<Sh, kL == kOuterBoth, kL != kInner, kPair, kScaled, Epi> part{
      problem_of(a, b, M, N, k, 2), epi, 0};
  Problem& p = part.p;
  p.nm = (int)up(M, Sh::BM);
  p.nn = (int)up(kPair ? 2LL * N : N, Sh::BN);
  p.per_group = p.stages;
  part.blocks = (p.nm * p.nn + 7) & ~7;
  return part;
}

// (a part with blocks = 0 is left out)
template <typename First, typename Second>
inline hipError_t launch_joint(const First& a, const Second& b, const Second& c, hipStream_t s) {
  constexpr int kLds = std::max(First::Sh::kLds, Second::Sh::kLds);
  hipLaunchKernelGGL((joint_kernel<First, Second>), dim3(a.blocks + b.blocks + c.blocks),
                     dim3(First::Sh::kThreads), kLds, s, a, b, c,
                     // the longest sums first
                     a.p.stages < b.p.stages && b.blocks ? a.blocks : 0);
  return hipGetLastError();
}

}  // namespace mm
}  // namespace moe
