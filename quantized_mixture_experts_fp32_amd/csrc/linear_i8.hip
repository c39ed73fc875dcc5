// Linear map in 8-bit integers: codes of the activations (a scale for each
// token) times codes of the weights (a scale for each feature).
//   out[t][n] = (sum_k qx[t][k] qw[n][k] * sw[n]) * sx[t] + bias[n]
// The sum is exact in int32 (K below 2^17); its products with sw and then sx and
// the bias are fp32, rounded once on store.  In this order no step leaves fp32's
// normal range before the result does (a sum is 0 or at least 1, and a scale of
// the quantiser at least 2^-126; sw below 2^97).
//
// A library of its own (libmoe_wq_i8.so), which libmoe_wq.so is linked to: its
// matrix instruction, 16 x 16 x 64, multiplies twice as fast as the one of 16 x
// 16 x 32, the widest that the check of libmoe_wq.so's waits knows (2501 x 4096 x
// 4096: 65 -> 45 us); its own waits have a check of their own.
//
// 2501 x 4096 -> 4096 from codes 43 us (1.9 POP/s), 4096 tokens 61 us (2.2), 8192^3
// 420 us (2.6); from bf16 tokens and their quantising 54 us.  One token of 2048 ->
// 2048 4.4 us, a launch: its codes are formed on the way into LDS.  64 tokens of 4096
// -> 12288 24 us, 4.5 of them the quantising, bound by the loads that 192 blocks keep
// in flight (2.7 TB/s).
#include "mm_launch.hpp"

namespace moe {
namespace {
using namespace mm;

struct ScaleStore {
  const float* sx;
  const float* sw;
  const float* bias;  // or null
  void* out;
  long long N;
  int f32;
  struct Columns {
    f32x8 w, b;
  };
  struct Ahead {
    static constexpr int kRegs = 1;
    float s;
  };
  __device__ __forceinline__ Columns columns(int n) const {
    return {load_f32<f32x8>(sw, n), bias_at<f32x8>(n)};
  }
  __device__ __forceinline__ Ahead ahead(int m, int) const { return {sx[m]}; }
  __device__ __forceinline__ void operator()(int m, int n, i32x8 a, const Columns& c,
                                             const Ahead& r) const {
    put(m, n, a, r.s, c.w, c.b);
  }
  // (the kernel for few tokens: four columns, read in place)
  __device__ __forceinline__ void operator()(int m, int n, i32x4 a) const {
    put(m, n, a, sx[m], load_f32<f32x4>(sw, n), bias_at<f32x4>(n));
  }
  template <typename V>
  __device__ __forceinline__ V bias_at(int n) const {
    return bias ? load_f32<V>(bias, n) : V(0.0f);
  }
  template <typename I, typename V>
  __device__ __forceinline__ void put(int m, int n, I a, float s, V w, V b) const {
    V v;
#pragma unroll
    for (int r = 0; r < (int)(sizeof(I) / 4); ++r) v[r] = (float)a[r] * w[r] * s;
    if (bias) v += b;
    store_as(out, f32, (size_t)m * N + n, v);
  }
};

}  // namespace

hipError_t launch_product_i8(const void* x, const float* x_scales, int T, int N, int K,
                             const int8_t* codes, const float* scales, const float* bias,
                             void* out, int out_f32, hipStream_t s) {
  const ScaleStore epi = {x_scales, scales, bias, out, N, out_f32};
  if (!x_scales)
    return launch_direct<I8, false, true>(
        {(const char*)x, (const char*)codes, 2LL * K, K, T, N, K, 0}, epi, s);
  const Operand a = {(const char*)x, nullptr, K, T}, b = {(const char*)codes, nullptr, K, N};
  return launch_product<I8, kInner, false>(a, b, T, N, K, 1, epi, nullptr, s);
}

const char* product_i8_name(int T, int N, int K) {
  return product_name(kInner, true, T, N, K, K, false);
}

bool product_i8_quantizes(int T, int N, int K) {
  return T <= kQuantRows && direct_applies(T, N, K, false);
}

}  // namespace moe
