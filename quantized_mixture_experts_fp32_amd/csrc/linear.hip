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
// matrix cores; between them the issue of instructions counts: the conversion
// of codes (a VALU step per code and token block), the activations, which every
// block reads whole, and the MFMAs run one after the other in a wave.  Measured
// (launches captured in a graph, weights rotated past the Infinity Cache where
// they fit):
//   tokens x K x N        us     bound
//   1 x 2048 x 2048       3.2    launch
//   1 x 4096 x 4096       4.4    launch and one round trip to HBM
//   1 x 8192 x 8192       8.9    3.9 TB/s of codes
//   4 x 4096 x 50304     22.5    4.7 TB/s (a large copy: 4.9)
//   16 x 4096 x 12288     7.4    3.6 TB/s
//   64 x 4096 x 12288    11.7    issue: one wave a SIMD, which issues in 57 % of
//                                its cycles, waits for the slot in 15 % and for
//                                memory, LDS and results in 29 %
//                                (profiles/counters_linear_w4_batch.txt);
//                                without any memory traffic 0.8 us less
//   64 x 4096 x 50304    40      issue: without any memory traffic 35
//   512 x 4096 x 4096    23.8    721 TFLOP/s
//   2501 x 4096 x 4096  105      798 TFLOP/s
//   4096 x 4096 x 4096  143      959 TFLOP/s (a library bf16 product: 1225)
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
  __device__ __forceinline__ void load(const uint16_t* x, int t0, int T, int K, int g, Lane& l) {
    asm volatile("" : "+v"(l.full), "+v"(l.last));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = min(t0 + 4 * i, (T - 1) & ~3);
      const char* b = (const char*)(x + (size_t)t * K + 128 * g);
      v[i] = *(const u32x4*)(b + (t + 4 <= T ? l.full : l.last));
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

// Calls f with the integral constants 0 .. N - 1.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<N, I + 1>(f);
  }
}

// Lane n of every row of 16 lanes to all lanes of the row.
template <int n>
__device__ __forceinline__ uint32_t row_lane(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x150 + n, 0xF, 0xF, true);
}

// Tile kernel.  A block computes 16 RT features of 16 NT tokens; its W waves
// take the 128-groups of K in turn (wave w those of w, w + W, ..), and the
// waves' totals are joined once, through LDS in wave order.  Of its group a
// wave holds the codes in registers and the activations in 4 NT KiB of LDS of
// its own, both asked for one group ahead.  The activations go to LDS directly
// (no registers, and no stores to issue: 64 tokens x 4096 x 12288 11.6 us,
// through registers 13.2), in whole 256-byte row pieces, chunk c of token t at
// position c ^ t: no bank conflicts.  One scale load serves four row tiles,
// lane 4 r + i of a row of 16 lanes holding row 4 kq + i of tile r.
//
// The compiler does not follow direct loads into LDS, so the waits are written
// out: all of a group's loads are waited for before its pieces are read, and
// the reads before the next group's loads may overwrite them.  Only this wave
// touches its pieces.
template <int W, int NT, int RT, bool kOutF32>
__global__ __launch_bounds__(W * kWave) void linear_w4_tile(
    const uint16_t* __restrict__ x, const uint8_t* __restrict__ codes,
    const uint16_t* __restrict__ scales, const float* __restrict__ bias, int T, int N, int K,
    int ntb, void* __restrict__ out) {
  extern __shared__ f32x4 lds[];  // x pieces [W][NT][256], then totals [W][RT * NT][64]
  constexpr int RS = (RT + 3) / 4;  // scale loads, of four row tiles each
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, kq = lane >> 4, G = K >> 7, ntile = N >> 4;
  // The token blocks of one row block run next to each other on one XCD, which
  // then reads the codes once; the row blocks past a multiple of the eight XCDs
  // are dealt over all of them (700 tokens x 4096 x 1024: 12.4 us, on the first
  // XCDs 19.6).
  const int id = blockIdx.x, nrb = (ntile + RT - 1) / RT, rest = nrb & 7;
  const int first = (nrb - rest) * ntb;  // blocks of the row blocks that come in eights
  const bool even = id < first;
  const int rb = even ? ((id >> 3) / ntb) * 8 + (id & 7) : nrb - rest + (id - first) % rest;
  const int t0 = (even ? (id >> 3) % ntb : (id - first) / rest) * 16 * NT;
  uint32_t lane_code = 64 * col + 16 * kq, lane_scale[RS];
  const uint8_t* cb[RT];
  const uint16_t* sb = scales + (size_t)(rb * RT) * 16 * G;
#pragma unroll
  for (int r = 0; r < RT; ++r) {  // tiles past the last one repeat it, unstored
    const int n0 = min(rb * RT + r, ntile - 1) << 4;
    cb[r] = codes + (size_t)n0 * (K >> 1);
  }
#pragma unroll
  for (int r = 0; r < RS; ++r) {
    const int tile = min(min(4 * r + (col >> 2), RT - 1), ntile - 1 - rb * RT);
    lane_scale[r] = (16 * tile + 4 * kq + (col & 3)) * G * 2;
  }
  u32x4* xl = (u32x4*)lds + wave * (NT * 256);
  const char* xb = (const char*)(x + (size_t)t0 * K);
  uint32_t xoff[NT][4];
#pragma unroll
  for (int c = 0; c < NT; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 4 * i + (lane >> 4);
      xoff[c][i] = (uint32_t)min(16 * c + t, T - 1 - t0) * K * 2 + 16 * ((lane & 15) ^ t);
    }
  struct Codes {
    u32x4 q[RT];
    _Float16 sc[RS];
  };
  // Loads past the wave's last group read one word for nothing: a load under
  // a branch would make the compiler wait for all loads in flight.
  auto load_codes = [&](int g, Codes& f) {
    const uint32_t mask = g < G ? ~0u : 0u;
    const int gc = min(g, G - 1);
    asm volatile("" : "+v"(lane_code));
#pragma unroll
    for (int r = 0; r < RT; ++r)
      f.q[r] = *(const u32x4*)(cb[r] + (size_t)1024 * gc + (lane_code & mask));
#pragma unroll
    for (int r = 0; r < RS; ++r) {
      asm volatile("" : "+v"(lane_scale[r]));
      f.sc[r] = *(const _Float16*)((const char*)(sb + gc) + (lane_scale[r] & mask));
    }
  };
  auto load_x = [&](int g) {
    const uint32_t mask = g < G ? ~0u : 0u;
    const char* b = xb + (size_t)256 * min(g, G - 1);
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t o = xoff[c][i] & mask;
        asm volatile("" : "+v"(o));
        __builtin_amdgcn_global_load_lds(
            b + o, (__attribute__((address_space(3))) void*)(xl + c * 256 + i * 64), 16, 0, 0);
      }
  };
  f32x4 acc[RT][NT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int c = 0; c < NT; ++c) acc[r][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto step = [&](int g, Codes& f, Codes& next) {
    bf16x8 xf[NT][4];
    // group g's pieces and codes, issued one group ago, have landed ..
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
      for (int m = 0; m < 4; ++m)
        xf[c][m] = as_bf16x8(xl[c * 256 + col * 16 + ((4 * kq + m) ^ col)]);
    // .. and are in registers before the next group's overwrite them
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    load_x(g + W);
    load_codes(g + W, next);
    __builtin_amdgcn_sched_barrier(0);
    f32x4 seed[NT];  // -192 * sum of token col's group, in every row
    u32x4 neg;
    neg = kNegOffset;
#pragma unroll
    for (int c = 0; c < NT; ++c) seed[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int c = 0; c < NT; ++c) seed[c] = mfma16(as_bf16x8(neg), xf[c][m], seed[c]);
    uint32_t sv[RS];
#pragma unroll
    for (int r = 0; r < RS; ++r) sv[r] = __float_as_uint(0.125f * (float)f.sc[r]);
    static_for<RT>([&](auto rc) {
      constexpr int r = decltype(rc)::value, b = 4 * (r & 3);
      const float s[4] = {__uint_as_float(row_lane<b>(sv[r >> 2])),
                          __uint_as_float(row_lane<b + 1>(sv[r >> 2])),
                          __uint_as_float(row_lane<b + 2>(sv[r >> 2])),
                          __uint_as_float(row_lane<b + 3>(sv[r >> 2]))};
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
    });
    __builtin_amdgcn_sched_barrier(0);
  };
  if (wave < G) {
    Codes a, b;
    load_x(wave);
    load_codes(wave, a);
    int g = wave;
    for (; g + W < G; g += 2 * W) {
      step(g, a, b);
      step(g + W, b, a);
    }
    if (g < G) step(g, a, b);
    // the loads for nothing past the last group still write this wave's pieces
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0F70);
    asm volatile("" ::: "memory");
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
  hipLaunchKernelGGL(kern, dim3(nrb * ntb), dim3(W * kWave),
                     sizeof(f32x4) * 64 * W * std::max(RT * NT, 4 * NT), s, x, codes, scales,
                     bias, T, N, K, ntb, out);
  return hipGetLastError();
}

// Blocks of the streaming kernel per token pass: one a CU over all passes, more
// where LDS would not hold a block's tiles; a multiple of 8 for the XCDs.
int stream_slots(int ntile, int npass, int nchunk) {
  const int most = nchunk > 1 ? kMaxTotals : kMaxTiles;
  const int n = std::max(std::max(kCUs / npass & ~7, 8), (ntile + most - 1) / most);
  return (std::min(n, ntile) + 7) & ~7;
}

template <int W, int NT, int NG, int D>
hipError_t stream_as(const uint16_t* x, const uint8_t* codes, const uint16_t* scales,
                     const float* bias, int T, int N, int K, void* out, int out_f32,
                     hipStream_t s) {
  const int G = K >> 7, ntile = N >> 4, npass = (T + 16 * NT - 1) / (16 * NT);
  const int nchunk = (G + W * NG - 1) / (W * NG), gpc = (G + nchunk - 1) / nchunk;
  const int nslot = stream_slots(ntile, npass, nchunk);
  const size_t lds = sizeof(f32x4) * (W * 64 * (NT > 2 ? 2 * NT : 4) + 4 * kMaxTiles +
                                      (nchunk > 1 ? 64 * NT * kMaxTotals : 0));
  auto kern =
      out_f32 ? linear_w4_stream<W, NT, NG, D, true> : linear_w4_stream<W, NT, NG, D, false>;
  hipLaunchKernelGGL(kern, dim3(nslot * npass), dim3(W * kWave), lds, s, x, codes, scales, bias, T,
                     N, K, npass, nchunk, gpc, out);
  return hipGetLastError();
}

typedef hipError_t (*RunFn)(const uint16_t*, const uint8_t*, const uint16_t*, const float*, int,
                            int, int, void*, int, hipStream_t);

// A tile kernel and its time, which goes by blocks a CU: at K = 4096 (32
// groups) `fixed` + `per` for each block a CU, and 0.065 us per MB of codes.
// Fitted to 480 shapes of 1 to 512 tokens, K 512 to 14336, N 512 to 50304 (a
// tenth off on most).  On 120 random shapes of 1 to 4096 tokens the choice took
// 1.3 % longer than the fastest kernel on average, 29 % at most
// (profiles/linear_choice.txt).  For up to 1024 inputs (8 groups) four waves do.
struct Tile {
  int tokens, rows, min_groups, max_groups;
  float fixed, per;
  RunFn run;
  const char* name;
};
const Tile kTiles[] = {
    {16, 1, 1, 1 << 30, 2.3f, 1.85f, tile_as<8, 1, 1>, "tile 16x16 w8"},
    {16, 2, 1, 8, 2.4f, 2.6f, tile_as<4, 1, 2>, "tile 16x32 w4"},
    {16, 2, 9, 1 << 30, 2.4f, 2.5f, tile_as<8, 1, 2>, "tile 16x32 w8"},
    {16, 3, 9, 1 << 30, 2.7f, 3.15f, tile_as<8, 1, 3>, "tile 16x48 w8"},
    {32, 2, 1, 1 << 30, 2.8f, 3.75f, tile_as<4, 2, 2>, "tile 32x32 w4"},
    {32, 3, 1, 1 << 30, 3.1f, 4.55f, tile_as<4, 2, 3>, "tile 32x48 w4"},
    {32, 4, 1, 1 << 30, 3.0f, 5.9f, tile_as<4, 2, 4>, "tile 32x64 w4"},
    {32, 6, 1, 1 << 30, 3.4f, 7.65f, tile_as<4, 2, 6>, "tile 32x96 w4"},
    {48, 4, 1, 1 << 30, 3.6f, 7.5f, tile_as<4, 3, 4>, "tile 48x64 w4"},
    {64, 4, 1, 1 << 30, 4.4f, 9.3f, tile_as<4, 4, 4>, "tile 64x64 w4"},
};

// The streaming kernel for T tokens and K inputs.
struct Stream {
  RunFn run;
  const char* name;
};
Stream stream_for(int T, int K) {
  if (T <= 16) return {stream_as<16, 1, 2, 2>, "stream 16"};
  if (K <= 16 * 128) return {stream_as<16, 2, 1, 2>, "stream 32 short"};
  return {stream_as<16, 2, 2, 1>, "stream 32"};
}

struct Choice {
  const Tile* tile;  // a tile kernel, or
  int gemm_tokens;   // the GEMM in tiles of so many tokens, or (0) streaming
};

Choice choose(int T, int N, int K) {
  const int G = K >> 7, ntile = N >> 4;
  auto up = [](long long a, long long b) { return (a + b - 1) / b; };
  Choice c = {nullptr, 0};
  float best = 1e30f;
  // The token blocks of a row block run next to each other, and past some 640
  // tokens their activations do not stay in an XCD's L2: at K = 4096 1.17 times
  // the time at 1024 tokens, 1.41 at 1536, 1.85 at 2501.  (By T alone; for the
  // six of the 120 shapes with more than 640 tokens and K up to 1024 the choice
  // took 0.5 % longer than the fastest.)
  const float crowd = 1.0f + std::max(T - 640, 0) / 2200.0f;
  for (const Tile& t : kTiles) {
    if (G < t.min_groups || G > t.max_groups) continue;
    const float per_cu = (float)up(up(T, t.tokens) * up(ntile, t.rows), kCUs);
    const float us = t.fixed + t.per * crowd * per_cu * G / 32 + 0.0325e-6f * N * K;
    if (us < best) {
      best = us;
      c.tile = &t;
    }
  }
  // Streaming: the prologue, which goes by K, and a block's row tiles.  It
  // reads the activations once a block: 4 tokens x 4096 x 50304 22.5 us
  // (tiled 23.1), 16 tokens 23.2 (27.9), 64 tokens 41 (48.9).
  // (For few tokens and up to 2048 inputs the tile kernel is the faster one.)
  if (G > (T <= 16 ? 16 : 8)) {
    const int npass = (int)up(T, T <= 16 ? 16 : 32);
    const int nslot = stream_slots(ntile, npass, (int)up(G, G <= 16 ? 16 : 32));
    const float tiles = crowd * up(ntile, nslot) * up((long long)nslot * npass, kCUs);
    const float us = T <= 16 ? 1.2f + 0.165f * G + tiles * (0.45f + 0.025f * G)
                             : 5.0f + 0.165f * G + tiles * (0.18f + 0.033f * G);
    if (us < best) {
      best = us;
      c.tile = nullptr;
    }
  }
  // GEMM (blocks of 256 features, two a CU): at K = 4096, one block a CU and
  // two, tiles of 64 tokens 50 and 81 us, of 96 68 and 112, of 128 83 and 140,
  // plus about 4 for the group sums.  E.g. N = 4096: 1024 tokens 49 us as
  // 64-token tiles of the tile kernel, 52 us here; 2501 tokens 105 us in tiles
  // of 96, 117 us in tiles of 128.
  if (T > 64) {
    static const struct {
      int tokens;
      float one, two;
    } kGemm[] = {{128, 83.0f, 140.0f}, {96, 68.0f, 112.0f}, {64, 50.0f, 81.0f}};
    for (const auto& t : kGemm) {
      const float per_cu = (float)up(up(T, t.tokens) * up(N, 256), kCUs);
      const float us = (per_cu <= 1.0f ? t.one : 0.5f * per_cu * t.two) * (K / 4096.0f) + 4.0f;
      if (us < best) {
        best = us;
        c.tile = nullptr;
        c.gemm_tokens = t.tokens;
      }
    }
  }
  return c;
}

}  // namespace

const char* linear_w4_kernel(int T, int N, int K) {
  const Choice c = choose(T, N, K);
  if (c.gemm_tokens)
    return c.gemm_tokens == 64 ? "gemm 64" : c.gemm_tokens == 96 ? "gemm 96" : "gemm 128";
  return c.tile ? c.tile->name : stream_for(T, K).name;
}

size_t linear_w4_ws_bytes(int T, int N, int K) {
  return choose(T, N, K).gemm_tokens ? linear_w4_gemm_ws_bytes(T, K) : 0;
}

hipError_t launch_linear_w4(const uint16_t* x, const uint8_t* codes, const uint16_t* scales,
                            const float* bias, int T, int N, int K, void* out, int out_f32,
                            void* ws, hipStream_t s) {
  const Choice c = choose(T, N, K);
  if (c.gemm_tokens)
    return launch_linear_w4_gemm(x, codes, scales, bias, T, N, K, c.gemm_tokens, out, out_f32, ws,
                                 s);
  const RunFn run = c.tile ? c.tile->run : stream_for(T, K).run;
  return run(x, codes, scales, bias, T, N, K, out, out_f32, s);
}

}  // namespace moe
