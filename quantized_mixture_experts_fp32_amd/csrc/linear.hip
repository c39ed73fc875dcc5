// Linear map with int4 weights: y = x W'^T (+ bias) for dense projections,
// with the codes and group scales of the experts (W' = s q, group 128).
//
// Arithmetic.  A code word becomes eight bf16 values 192 + 8 q (w4_top); every
// 128-group's MFMA sum is corrected by -192 * sum(x over the group), which
// leaves 8 sum(q x) in fp32, and the fp16 scale / 8 (exact) weights it into the
// running fp32 total.  Weights are never rounded; the result is rounded once,
// on store.
//
// Layout.  Lane (row r, quarter kq) of a wave reads bytes [16 kq, 16 kq + 16)
// of row r of a 16-row tile's group: one 16-byte load per lane takes the
// whole 1 KiB block.  The activations of token c sit in lanes (c, kq).  The
// scale of row 4 q + i is loaded by lane i of each quad of lane row q and
// reaches the quad by a lane permutation of the multiply's operand.
//
// Kernels.  Few tokens are bound by the codes' bytes, large batches by the
// matrix cores; between them the conversion of codes (a VALU step per code and
// token pass) and the activations, which every block reads whole, take as long
// as either.  Measured (launches captured in a graph, weights rotated past the
// Infinity Cache where they fit):
//   tokens x K x N        us     bound
//   1 x 2048 x 2048       3.2    launch
//   1 x 4096 x 4096       4.4    launch and one round trip to HBM
//   1 x 8192 x 8192       9.4    3.7 TB/s of codes
//   4 x 4096 x 50304     22.6    4.7 TB/s (a large copy: 4.9)
//   16 x 4096 x 12288     8.0    3.3 TB/s
//   64 x 4096 x 12288    13.2    codes converted twice, activations 256 KB a CU
//   512 x 4096 x 4096    27      638 TFLOP/s
//   2501 x 4096 x 4096  104      806 TFLOP/s
//   4096 x 4096 x 4096  141      977 TFLOP/s (a library bf16 product: 1225)
#include <math.h>

#include <algorithm>

#include "kcommon.hpp"
#include "launch.hpp"

namespace moe {
namespace {

constexpr uint32_t kOffset = 0x43404340u;     // 192.0 twice, the conversion offset
constexpr uint32_t kNegOffset = 0xC340C340u;  // -192.0 twice
constexpr int kMaxTiles = 256;                // row tiles of a block
constexpr int kMaxTotals = 32;                // the same when K takes several chunks
constexpr int kCUs = 256;

// Lane 4 q + i's value to all four lanes of quad q.
template <int i>
__device__ __forceinline__ uint32_t quad_lane(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x55 * i, 0xF, 0xF, true);
}

// Four features of a token, with the bias (null: none) added.
template <bool kF32>
__device__ __forceinline__ void store_out(void* out, const float* bias, int t, int N, int n,
                                          f32x4 v) {
  if (bias) v += *(const f32x4*)(bias + n);
  if (kF32) {
    *(f32x4*)((float*)out + (size_t)t * N + n) = v;
  } else {
    uint2 pk;
    pk.x = f32_to_bf16_rne(v[0]) | (f32_to_bf16_rne(v[1]) << 16);
    pk.y = f32_to_bf16_rne(v[2]) | (f32_to_bf16_rne(v[3]) << 16);
    *(uint2*)((uint16_t*)out + (size_t)t * N + n) = pk;
  }
}

// Activations of one 128-group as MFMA fragments: lane (col, kq) gets the 32
// values 32 kq .. of token col.  Read like that, neighbouring lanes would sit
// in different rows, which the L1 serves at a third of its rate (9.7 against
// 30 TB/s over the chip, all in L2); so a wave reads whole 256-byte row
// pieces, four tokens an instruction, and turns them around in 4 KiB of LDS of
// its own (chunk c of token t at position c ^ t: no bank conflicts).
struct XPiece {
  u32x4 v[4];
  // Byte offsets of lane's chunk in four full rows, and in the four rows that
  // the last token ends (those past it repeat it; their columns are not
  // stored).
  struct Lane {
    uint32_t full, last;
    __device__ __forceinline__ Lane(int T, int K, int lane) {
      full = (uint32_t)(lane >> 4) * K * 2 + 16 * (lane & 15);
      last = (uint32_t)min(lane >> 4, (T - 1) & 3) * K * 2 + 16 * (lane & 15);
    }
  };
  // rows t0 + 4 i + lane / 16 of the 16 from t0 on, chunk lane % 16
  // (mask 0: one word of the first chunk instead, a load for nothing)
  __device__ __forceinline__ void load(const uint16_t* x, int t0, int T, int K, int g, Lane& l,
                                       uint32_t mask = ~0u) {
    asm volatile("" : "+v"(l.full), "+v"(l.last));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = min(t0 + 4 * i, (T - 1) & ~3);
      const char* b = (const char*)(x + (size_t)t * K + 128 * g);
      v[i] = *(const u32x4*)(b + ((t + 4 <= T ? l.full : l.last) & mask));
    }
  }
  __device__ __forceinline__ void turn(u32x4* buf, int lane, bf16x8 (&f)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 4 * i + (lane >> 4);
      buf[t * 16 + ((lane & 15) ^ t)] = v[i];
    }
    const int col = lane & 15, kq = lane >> 4;
#pragma unroll
    for (int m = 0; m < 4; ++m) f[m] = as_bf16x8(buf[col * 16 + ((4 * kq + m) ^ col)]);
  }
};

// Streaming kernel (few tokens, HBM-bound).  A block holds the activations of
// 16 NT tokens for a chunk of up to 16 NG groups of K in registers, wave w
// those of groups w, w + 16, .., and walks row tiles: per tile a wave loads
// and multiplies only codes, D tiles ahead, and the waves' totals are joined
// through LDS in wave order.  A longer K takes several chunks, whose totals
// are kept in LDS between them.  Token passes (of 16 NT) of the same tiles run
// next to each other on one XCD, which then reads the codes once from HBM.
// Every load of the main tile loop is unconditional (a wave past the last group
// reads it again, with scale 0): a load under a branch would make the compiler
// wait for all loads in flight.
template <int W, int NT, int NG, int D, bool kOutF32>
__global__ __launch_bounds__(W * kWave) void linear_w4_stream(
    const uint16_t* __restrict__ x, const uint8_t* __restrict__ codes,
    const uint16_t* __restrict__ scales, const float* __restrict__ bias, int T, int N, int K,
    int npass, int nchunk, int gpc, void* __restrict__ out) {
  extern __shared__ f32x4 lds[];
  constexpr int kRed = W * 64 * (NT > 2 ? 2 * NT : 4);
  f32x4* red = lds;                         // x pieces [W][256], then totals [2][W][NT][64]
  f32x4* bias_lds = lds + kRed;             // [kMaxTiles][4]
  f32x4* total = bias_lds + kMaxTiles * 4;  // [tiles][NT][64] (several chunks)
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, kq = lane >> 4, G = K >> 7;
  uint32_t lane_code = 64 * col + 16 * kq, lane_scale = (4 * kq + (col & 3)) * G * 2;
  XPiece::Lane xlane(T, K, lane);
  const int id = blockIdx.x, nslot = gridDim.x / npass;
  const int slot = ((id >> 3) / npass) * 8 + (id & 7), t0 = ((id >> 3) % npass) * 16 * NT;
  const int ntile = N >> 4;
  if (slot >= ntile) return;
  const int nmine = (ntile - slot + nslot - 1) / nslot;
  if (bias) {
    for (int i = tid; i < nmine * 4; i += (W * kWave))
      bias_lds[i] = *(const f32x4*)(bias + ((slot + nslot * (i >> 2)) << 4) + 4 * (i & 3));
  }

  for (int ch = 0; ch < nchunk; ++ch) {
    const int g0 = ch * gpc + wave, gend = min(G, (ch + 1) * gpc);
    auto load = [&](int i, u32x4 (&q)[NG], _Float16 (&sc)[NG]) {
      const int n0 = (slot + nslot * i) << 4;
      const uint8_t* cd = codes + (size_t)n0 * (K >> 1);
      const uint16_t* sr = scales + (size_t)n0 * G;
      asm volatile("" : "+v"(lane_code), "+v"(lane_scale));
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        const int g = min(g0 + W * j, gend - 1);
        q[j] = *(const u32x4*)(cd + (size_t)1024 * g + lane_code);
        sc[j] = *(const _Float16*)((const char*)(sr + g) + lane_scale);
      }
    };
    u32x4 q[D][NG];
    _Float16 sc[D][NG];
#pragma unroll
    for (int u = 0; u < D; ++u) {
      if (u < nmine) load(u, q[u], sc[u]);
      __builtin_amdgcn_sched_barrier(0);
    }
    bf16x8 xf[NT][NG][4];
    float seed[NT][NG];
#pragma unroll
    for (int c = 0; c < NT; ++c) {
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        XPiece px;
        px.load(x, t0 + 16 * c, T, K, min(g0 + W * j, gend - 1), xlane);
        px.turn((u32x4*)red + 256 * wave, lane, xf[c][j]);
        f32x4 p = {0.0f, 0.0f, 0.0f, 0.0f};
        u32x4 neg;
        neg = kNegOffset;
#pragma unroll
        for (int m = 0; m < 4; ++m) p = mfma16(as_bf16x8(neg), xf[c][j][m], p);
        seed[c][j] = p[0];  // -192 * sum of token col's group: the same in every row
      }
    }

    // one tile from a buffer, which then receives the tile D ahead
    auto step = [&](int i, u32x4 (&q)[NG], _Float16 (&sc)[NG], auto ahead) {
      f32x4 acc[NT];
#pragma unroll
      for (int c = 0; c < NT; ++c) acc[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        const float f = g0 + W * j < gend ? 0.125f : 0.0f;
        const uint32_t sb = __float_as_uint(f * (float)sc[j]);
        const float s[4] = {__uint_as_float(quad_lane<0>(sb)), __uint_as_float(quad_lane<1>(sb)),
                            __uint_as_float(quad_lane<2>(sb)), __uint_as_float(quad_lane<3>(sb))};
        f32x4 p[NT];
#pragma unroll
        for (int c = 0; c < NT; ++c) p[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const bf16x8 w = w4_top(q[j][m], kOffset);
#pragma unroll
          for (int c = 0; c < NT; ++c) p[c] = mfma16(w, xf[c][j][m], p[c]);
        }
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[c][r] = fmaf(s[r], p[c][r] + seed[c][j], acc[c][r]);
        if (NT * NG > 2) __builtin_amdgcn_sched_barrier(0);
      }
      // The totals are formed before the branch: read behind it, the last MFMA's
      // result came too early (the compiler's wait states did not cover the
      // path around the loads).
#pragma unroll
      for (int c = 0; c < NT; ++c) asm volatile("" : "+v"(acc[c]));
      if (decltype(ahead)::value || i + D < nmine) load(i + D, q, sc);
      f32x4* rd = red + (i & 1) * (W * NT * 64);
#pragma unroll
      for (int c = 0; c < NT; ++c) rd[(wave * NT + c) * 64 + lane] = acc[c];
      // one barrier a tile: buffer i & 1 is written again only past the
      // barrier of tile i + 1, which its readers reach after reading
      __syncthreads();
      if (tid < NT * 64) {
        f32x4 v = rd[tid];
#pragma unroll 3
        for (int w = 1; w < W; ++w) v += rd[w * NT * 64 + tid];
        if (nchunk > 1) {  // thread tid alone keeps entry (i, tid)
          if (ch > 0) v += total[i * NT * 64 + tid];
          if (ch + 1 < nchunk) total[i * NT * 64 + tid] = v;
        }
        const int t = t0 + 16 * (tid >> 6) + col;
        if (ch + 1 == nchunk && t < T) {
          const int n = ((slot + nslot * i) << 4) + 4 * kq;
          if (bias) v += bias_lds[4 * i + kq];
          store_out<kOutF32>(out, nullptr, t, N, n, v);
        }
      }
    };
    __syncthreads();  // the waves' x pieces and the totals share LDS
    int i0 = 0;
    for (; i0 + 2 * D <= nmine; i0 += D) {
#pragma unroll
      for (int u = 0; u < D; ++u) step(i0 + u, q[u], sc[u], std::true_type{});
    }
#pragma unroll
    for (int u = 0; u < 2 * D - 1; ++u)
      if (i0 + u < nmine) step(i0 + u, q[u % D], sc[u % D], std::false_type{});
    __syncthreads();  // the next chunk starts on buffer 0 again
  }
}

// Tile kernel.  A block computes 16 RT features of 16 NT tokens; its W waves
// take the 128-groups of K in turn (wave w those of w, w + W, ..) and stream
// codes and activations into registers, one group ahead; the waves' totals
// are joined once, through LDS in wave order.  (The loop is kept small: with
// more groups in flight its code grows, and at 3 to 10 us a call fetching it
// costs more than the deeper queue gives.)
template <int W, int NT, int RT, bool kOutF32>
__global__ __launch_bounds__(W * kWave) void linear_w4_tile(
    const uint16_t* __restrict__ x, const uint8_t* __restrict__ codes,
    const uint16_t* __restrict__ scales, const float* __restrict__ bias, int T, int N, int K,
    int ntb, void* __restrict__ out) {
  extern __shared__ f32x4 lds[];  // x pieces [W][256], then totals [W][RT * NT][64]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, kq = lane >> 4, G = K >> 7, ntile = N >> 4;
  // the token blocks of one row block run next to each other on one XCD
  const int id = blockIdx.x;
  const int rb = ((id >> 3) / ntb) * 8 + (id & 7), t0 = ((id >> 3) % ntb) * 16 * NT;
  if (rb * RT >= ntile) return;
  uint32_t lane_code = 64 * col + 16 * kq, lane_scale = (4 * kq + (col & 3)) * G * 2;
  const uint8_t* cb[RT];
  const uint16_t* sb[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {  // tiles past the last one repeat it, unstored
    const int n0 = min(rb * RT + r, ntile - 1) << 4;
    cb[r] = codes + (size_t)n0 * (K >> 1);
    sb[r] = scales + (size_t)n0 * G;
  }
  XPiece px[NT];
  XPiece::Lane xlane(T, K, lane);
  struct Codes {
    u32x4 q[RT];
    _Float16 sc[RT];
  };
  // Loads past the wave's last group read one word for nothing: a load under
  // a branch would make the compiler wait for all loads in flight.
  auto load_codes = [&](int g, Codes& f) {
    const uint32_t mask = g < G ? ~0u : 0u;
    const int gc = min(g, G - 1);
    asm volatile("" : "+v"(lane_code), "+v"(lane_scale));
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      f.q[r] = *(const u32x4*)(cb[r] + (size_t)1024 * gc + (lane_code & mask));
      f.sc[r] = *(const _Float16*)((const char*)(sb[r] + gc) + (lane_scale & mask));
    }
  };
  auto load_x = [&](int g) {
#pragma unroll
    for (int c = 0; c < NT; ++c)
      px[c].load(x, t0 + 16 * c, T, K, min(g, G - 1), xlane, g < G ? ~0u : 0u);
  };
  f32x4 acc[RT][NT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int c = 0; c < NT; ++c) acc[r][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  // Group g from f and px.  Loads return in order, so the activations of the
  // next group are asked for before the codes of the one after it: waiting
  // for the former leaves the latter, which come from HBM, in flight.
  auto step = [&](int g, Codes& f) {
    bf16x8 xf[NT][4];
#pragma unroll
    for (int c = 0; c < NT; ++c) px[c].turn((u32x4*)lds + 256 * wave, lane, xf[c]);
    load_x(g + W);
    __builtin_amdgcn_sched_barrier(0);
    f32x4 seed[NT];  // -192 * sum of token col's group, in every row
    u32x4 neg;
    neg = kNegOffset;
#pragma unroll
    for (int c = 0; c < NT; ++c) {
      seed[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int m = 0; m < 4; ++m) seed[c] = mfma16(as_bf16x8(neg), xf[c][m], seed[c]);
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const uint32_t sv = __float_as_uint(0.125f * (float)f.sc[r]);
      const float s[4] = {__uint_as_float(quad_lane<0>(sv)), __uint_as_float(quad_lane<1>(sv)),
                          __uint_as_float(quad_lane<2>(sv)), __uint_as_float(quad_lane<3>(sv))};
      f32x4 p[NT];
#pragma unroll
      for (int c = 0; c < NT; ++c) p[c] = seed[c];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const bf16x8 w = w4_top(f.q[r][m], kOffset);
#pragma unroll
        for (int c = 0; c < NT; ++c) p[c] = mfma16(w, xf[c][m], p[c]);
      }
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[r][c][i] = fmaf(s[i], p[c][i], acc[r][c][i]);
    }
    __builtin_amdgcn_sched_barrier(0);
    load_codes(g + 2 * W, f);
    __builtin_amdgcn_sched_barrier(0);
  };
  if (wave < G) {
    Codes a, b;
    load_codes(wave, a);
    __builtin_amdgcn_sched_barrier(0);
    load_x(wave);
    __builtin_amdgcn_sched_barrier(0);
    load_codes(wave + W, b);
    __builtin_amdgcn_sched_barrier(0);
    int g = wave;
    for (; g + W < G; g += 2 * W) {
      step(g, a);
      step(g + W, b);
    }
    if (g < G) step(g, a);
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int c = 0; c < NT; ++c) lds[(wave * RT * NT + r * NT + c) * 64 + lane] = acc[r][c];
  __syncthreads();
  for (int o = tid; o < RT * NT * 64; o += W * kWave) {
    f32x4 v = lds[o];
#pragma unroll
    for (int w = 1; w < W; ++w) v += lds[w * RT * NT * 64 + o];
    const int t = t0 + 16 * ((o >> 6) % NT) + col, n = ((rb * RT + o / (NT * 64)) << 4) + 4 * kq;
    if (n < N && t < T) store_out<kOutF32>(out, bias, t, N, n, v);
  }
}

template <int W, int NT, int RT>
hipError_t tile_as(const uint16_t* x, const uint8_t* codes, const uint16_t* scales,
                   const float* bias, int T, int N, int K, void* out, int out_f32,
                   hipStream_t s) {
  const int ntb = (T + 16 * NT - 1) / (16 * NT), nrb = ((N >> 4) + RT - 1) / RT;
  auto kern = out_f32 ? linear_w4_tile<W, NT, RT, true> : linear_w4_tile<W, NT, RT, false>;
  hipLaunchKernelGGL(kern, dim3(((nrb + 7) & ~7) * ntb), dim3(W * kWave),
                     sizeof(f32x4) * 64 * W * std::max(RT * NT, 4), s, x, codes, scales, bias, T,
                     N, K, ntb, out);
  return hipGetLastError();
}

template <int W, int NT, int NG, int D>
hipError_t stream_as(const uint16_t* x, const uint8_t* codes, const uint16_t* scales,
                     const float* bias, int T, int N, int K, void* out, int out_f32,
                     hipStream_t s) {
  const int G = K >> 7, ntile = N >> 4, npass = (T + 16 * NT - 1) / (16 * NT);
  const int nchunk = (G + W * NG - 1) / (W * NG), gpc = (G + nchunk - 1) / nchunk;
  // one block a CU over all passes, more where LDS would not hold its tiles
  const int most = nchunk > 1 ? kMaxTotals : kMaxTiles;
  int nslot = std::max((kCUs + npass - 1) / npass, (ntile + most - 1) / most);
  nslot = (std::min(nslot, ntile) + 7) & ~7;
  const size_t lds = sizeof(f32x4) * (W * 64 * (NT > 2 ? 2 * NT : 4) + 4 * kMaxTiles +
                                      (nchunk > 1 ? 64 * NT * kMaxTotals : 0));
  // a block with one tile has nothing to load ahead
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3(nslot * npass), dim3((W * kWave)), lds, s, x, codes, scales, bias,
                       T, N, K, npass, nchunk, gpc, out);
  };
  if (ntile <= nslot)
    out_f32 ? go(linear_w4_stream<W, NT, NG, 1, true>) : go(linear_w4_stream<W, NT, NG, 1, false>);
  else
    out_f32 ? go(linear_w4_stream<W, NT, NG, D, true>) : go(linear_w4_stream<W, NT, NG, D, false>);
  return hipGetLastError();
}

}  // namespace

// Tokens per tile of the GEMM kernel (blocks of 256 features, two a CU) where
// it is the faster one, otherwise 0.  Its time goes by blocks a CU; measured
// at K = 4096 (us, one block a CU and two): tiles of 64 tokens 50 and 81, of 96
// 68 and 112, of 128 83 and 140, plus about 4 for the group sums.  The kernels
// below take 2.9e-9 us per token, feature and input (3.2e-9 for K <= 2048,
// 4.6e-9 for K <= 1024).  E.g. N = 4096: 1024 tokens 49 us streamed, 52 us in
// tiles of 64; 2501 tokens 104 us in tiles of 96, 116 us in tiles of 128.
static int gemm_tile(int T, int N, int K) {
  if (T <= 64) return 0;
  static const struct {
    int tokens;
    float one, two;
  } kTiles[] = {{128, 83.0f, 140.0f}, {96, 68.0f, 112.0f}, {64, 50.0f, 81.0f}};
  const float per = K <= 1024 ? 4.6e-9f : K <= 2048 ? 3.2e-9f : 2.9e-9f;
  float best = per * (float)((T + 31) / 32 * 32) * N * K;
  int tokens = 0;
  for (const auto& t : kTiles) {
    const float blocks = (float)((T + t.tokens - 1) / t.tokens) * ((N + 255) / 256);
    const float per_cu = ceilf(blocks / kCUs);
    const float us = (per_cu <= 1.0f ? t.one : 0.5f * per_cu * t.two) * (K / 4096.0f) + 4.0f;
    if (us < best) {
      best = us;
      tokens = t.tokens;
    }
  }
  return tokens;
}

size_t linear_w4_ws_bytes(int T, int N, int K) {
  return gemm_tile(T, N, K) ? linear_w4_gemm_ws_bytes(T, K) : 0;
}

hipError_t launch_linear_w4(const uint16_t* x, const uint8_t* codes, const uint16_t* scales,
                            const float* bias, int T, int N, int K, void* out, int out_f32,
                            void* ws, hipStream_t s) {
  if (const int tokens = gemm_tile(T, N, K))
    return launch_linear_w4_gemm(x, codes, scales, bias, T, N, K, tokens, out, out_f32, ws, s);
  auto as = [&](auto f) { return f(x, codes, scales, bias, T, N, K, out, out_f32, s); };
  const int G = K >> 7, ntile = N >> 4;
  if (T <= 16) {
    // Tile kernel while every row tile is taken at once, by a block of one to
    // three tiles a CU (K <= 1024: by two of four waves, 50304 features of 4
    // tokens 8.7 us, streamed 12.6); with more, the streaming kernel, which
    // reads x once a block (K = 4096, N = 50304: 22.5 us, tiled 26).
    if (ntile <= kCUs) return G >= 96 ? as(tile_as<16, 1, 1>) : as(tile_as<8, 1, 1>);
    if (G <= 8) return as(tile_as<4, 1, 2>);
    if (ntile <= 2 * kCUs) return as(tile_as<8, 1, 2>);
    if (ntile <= 5 * kCUs) return as(tile_as<8, 1, 3>);
    return G <= 16 ? as(stream_as<16, 1, 1, 2>) : as(stream_as<16, 1, 2, 2>);
  }
  // 32 tokens a block or pass.  Tile kernel up to 8 row tiles a CU (and for a
  // K that would leave streaming waves idle), with as many tiles a block as
  // leave one or two blocks a CU; beyond, the streaming kernel.  At K = 4096:
  // 64 tokens, N = 50304: 42 us streamed, 52 us tiled; 512 tokens, N = 4096: 27
  // and 29 us; 128 tokens: 11.2 and 10.4 us; 64 tokens, N = 12288: 13.2 us with
  // six tiles, 15.7 us with four.
  const int units = (int)std::min<long long>(
      ((long long)ntile * ((T + 31) / 32) + kCUs - 1) / kCUs, 1 << 30);
  if (units <= 2) return as(tile_as<8, 2, 2>);
  if (units == 5 || units == 6) return as(tile_as<4, 2, 6>);
  if (units <= 8 || G <= 8) return as(tile_as<4, 2, 4>);
  return G <= 16 ? as(stream_as<16, 2, 1, 2>) : as(stream_as<16, 2, 2, 1>);
}

}  // namespace moe
