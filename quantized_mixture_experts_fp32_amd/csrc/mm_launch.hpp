// Host side of the tiled matrix product (mm_core.hpp): tile shape and split of
// k by the product's size, launch, and the join of split sums.
#pragma once
#include <algorithm>

#include "launch.hpp"
#include "mm_core.hpp"

namespace moe {
namespace mm {

typedef Shape<256, 256, 2, 4, 2> Big;
typedef Shape<128, 128, 2, 2, 2> Mid;
typedef Shape<64, 128, 1, 4, 3> Low;

struct Plan {
  int shape;   // 0 Big, 1 Mid, 2 Low
  int splits;  // of k
  int per;     // stages a split
};

inline long long up(long long a, long long b) { return (a + b - 1) / b; }

// M rows and N columns (of B, so 2 f of the pair form), `stages` of k; low: the
// product has the shape of few rows.
inline Plan plan_product(long long M, long long N, int stages, bool low) {
  constexpr int kCUs = 256;
  Plan best = {1, 1, stages};
  double least = 1e30;
  const struct {
    int bm, bn, a_cu;
    double stage;  // us a stage, all places of a CU taken
  } kShapes[] = {{256, 256, 1, 1.95}, {128, 128, 2, 1.24}, {64, 128, 2, 0.75}};
  for (int s = 0; s < (low ? 3 : 2); ++s) {
    const long long tiles = up(M, kShapes[s].bm) * up(N, kShapes[s].bn);
    for (int k = 1; k <= 16 && (k == 1 || stages / k >= 4); k *= 2) {
      const int per = (int)up(stages, k), n = per ? (int)up(stages, per) : 1;
      const double rounds = (double)up(tiles * n, kCUs * kShapes[s].a_cu);
      const double us = rounds * kShapes[s].stage * std::max(per, 1) +
                        (n > 1 ? 4.0 + 8.0e-6 * n * M * N / 4.0 : 0.0);
      if (us < least) {
        least = us;
        best = {s, n, per};
      }
    }
  }
  return best;
}

inline size_t partial_bytes(long long M, long long N, int stages, bool low) {
  const Plan p = plan_product(M, N, stages, low);
  return p.splits > 1 ? (size_t)p.splits * M * N * 4 : 0;
}

// A split's sums, as the instruction has them.
template <typename Acc>
struct StorePartial {
  float* ws;
  long long M, N;  // N: all columns (both of the pair form)
  __device__ __forceinline__ void operator()(int m, int n, Acc v) const {
    *(Acc*)(ws + ((size_t)blockIdx.y * M + m) * N + n) = v;
  }
  __device__ __forceinline__ void operator()(int m, int n, Acc a, Acc b) const {
    (*this)(m, n, a);
    (*this)(m, n + (int)(N / 2), b);
  }
};

// The splits' sums in their order, and the epilogue; four columns a thread.
template <typename Acc, bool kPair, typename Epi>
__global__ __launch_bounds__(256) void join_kernel(const float* __restrict__ ws, long long M,
                                                   long long N, int splits, const Epi epi) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long nq = (kPair ? N / 2 : N) / 4;
  if (i >= M * nq) return;
  const int m = (int)(i / nq), n = 4 * (int)(i % nq);
  const float* p = ws + (size_t)m * N + n;
  Acc a = *(const Acc*)p, b = a;
  if (kPair) b = *(const Acc*)(p + N / 2);
  for (int s = 1; s < splits; ++s) {
    p += M * N;
    a += *(const Acc*)p;
    if (kPair) b += *(const Acc*)(p + N / 2);
  }
  if constexpr (kPair)
    epi(m, n, a, b);
  else
    epi(m, n, a);
}

template <typename Mma, typename Sh, bool kAOuter, bool kBOuter, bool kPair, typename Epi>
inline void launch_shape(Problem p, const Plan& plan, const Epi& epi, hipStream_t s) {
  p.nm = (int)up(p.M, Sh::BM);
  p.nn = (int)up(kPair ? 2LL * p.N : p.N, Sh::BN);
  p.per_split = plan.per;
  hipLaunchKernelGGL((product_kernel<Mma, Sh, kAOuter, kBOuter, kPair, Epi>),
                     dim3(p.nm * p.nn, plan.splits), dim3(Sh::kThreads), Sh::kLds, s, p, epi);
}

// C = A B^T with the epilogue.  a, b: the operands; stages_of: k.  ws: at least
// partial_bytes of it.
template <typename Mma, bool kAOuter, bool kBOuter, bool kPair, typename Epi>
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
  constexpr bool kLow = !kAOuter;
  const long long cols = kPair ? 2LL * N : N;
  const Plan plan = plan_product(M, cols, p.stages, kLow);
  auto go = [&](const auto& e) {
    typedef std::decay_t<decltype(e)> E;
    if (plan.shape == 0) {
      launch_shape<Mma, Big, kAOuter, kBOuter, kPair, E>(p, plan, e, s);
    } else if (plan.shape == 1) {
      launch_shape<Mma, Mid, kAOuter, kBOuter, kPair, E>(p, plan, e, s);
    } else {
      if constexpr (kLow) launch_shape<Mma, Low, kAOuter, kBOuter, kPair, E>(p, plan, e, s);
    }
  };
  if (plan.splits == 1) {
    go(epi);
    return hipGetLastError();
  }
  typedef typename Mma::Acc Acc;
  go(StorePartial<Acc>{(float*)ws, M, cols});
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const long long quads = (long long)M * (N / 4);
  hipLaunchKernelGGL((join_kernel<Acc, kPair, Epi>), dim3((uint32_t)up(quads, 256)), dim3(256), 0,
                     s, (const float*)ws, (long long)M, cols, plan.splits, epi);
  return hipGetLastError();
}

}  // namespace mm
}  // namespace moe
