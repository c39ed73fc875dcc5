// Linear map in 8-bit integers: codes of the activations (a scale for each
// token) times codes of the weights (a scale for each feature).
//   out[t][n] = sx[t] sw[n] sum_k qx[t][k] qw[n][k] + bias[n]
// The sum is exact in int32 (K below 2^17); the scales' product, its product
// with the sum and the bias are fp32, rounded once on store.
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
  template <typename I>
  __device__ __forceinline__ void operator()(int m, int n, I a) const {
    typedef std::conditional_t<sizeof(I) == 32, f32x8, f32x4> V;
    const float s = sx[m];
    const V w = load_as<V>(sw, 1, n);
    V v;
#pragma unroll
    for (int r = 0; r < (int)(sizeof(I) / 4); ++r) v[r] = (float)a[r] * (s * w[r]);
    if (bias) v += load_as<V>(bias, 1, n);
    store_as(out, f32, (size_t)m * N + n, v);
  }
};

size_t round_up(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

size_t linear_i8_ws_bytes(int T, int N, int K, int x_bf16) {
  if (!x_bf16 || (T <= kQuantRows && direct_applies(T, N, K, false))) return 0;
  return round_up((size_t)T * K) + round_up(4 * (size_t)T);
}

hipError_t launch_linear_i8(const void* x, const float* x_scales, int T, int N, int K,
                            const int8_t* codes, const float* scales, const float* bias, void* out,
                            int out_f32, void* ws, hipStream_t s) {
  if (!x_scales && T <= kQuantRows && direct_applies(T, N, K, false))
    return launch_direct<I8, false, true>(
        {(const char*)x, (const char*)codes, 2LL * K, K, T, N, K, 0},
        ScaleStore{nullptr, scales, bias, out, N, out_f32}, s);
  if (!x_scales) {
    int8_t* q = (int8_t*)ws;
    float* sx = (float*)((char*)ws + round_up((size_t)T * K));
    const hipError_t e = launch_quantize_i8(x, 0, T, K, 1, q, sx, s);
    if (e != hipSuccess) return e;
    x = q;
    x_scales = sx;
  }
  const Operand a = {(const char*)x, nullptr, K, T}, b = {(const char*)codes, nullptr, K, N};
  return launch_product<I8, kInner, false>(
      a, b, T, N, K, 1, ScaleStore{x_scales, scales, bias, out, N, out_f32}, nullptr, s);
}

}  // namespace moe
