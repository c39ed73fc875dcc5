// Tiled matrix product for gfx950: C[m][n] = sum_k A(m, k) B(n, k), bf16 or
// int8 operands, 32-bit sums.  One body serves the forward and both gradient
// products of a map: either operand may be stored with k running along a row
// (K-inner) or along the columns (K-outer, bf16 only).
//
// A block computes a BM x BN tile; its waves take TM x TN of it in 16 x 16
// matrix instructions.  B's rows are the instruction's rows, so a lane holds
// four consecutive n of one m.
//
// Operands go to LDS directly, 128 bytes of k (K-inner) or 64 rows of k
// (K-outer) a stage, S stages in a ring.  Buffer loads do the bounds: rows past
// the end, and k past the end of a K-outer operand, read zeros; a K-inner
// operand's last stage sends chunks past K out of range.
//
//   K-inner: row r takes 128 bytes, 16-byte chunk c at c ^ ((r >> 1) & 7): the
//     16 rows a fragment reads fall on all 64 banks.
//   K-outer: row k takes 2 BM bytes, 32-byte granule g at g ^ f(k), f(k) =
//     k & 3 | (k >> 1) & 4; fragments come through the LDS transpose read, which
//     turns four rows of 16 values into four values for each of 16 lanes.
#pragma once
#include "kcommon.hpp"

namespace moe {
namespace mm {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int16_t i16x4 __attribute__((ext_vector_type(4)));
typedef int16_t i16x8 __attribute__((ext_vector_type(8)));

constexpr int kStageBytes = 128;  // bytes of k a stage, K-inner
constexpr int kStageK = 64;       // rows of k a stage, K-outer
constexpr uint32_t kOutOfRange = 0x80000000u;

// One operand of a product.
struct Operand {
  const char* p;
  const char* p2;      // second matrix, interleaved by 16 rows (pair form), or null
  long long stride;    // bytes between rows
  int rows;            // rows of the product (m or n), per matrix
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const char* p, long long bytes) {
  const long long n = bytes < 0 ? 0 : bytes > 0x7FFFFFFF ? 0x7FFFFFFF : bytes;
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)n, 0x00020000);
}

template <int vm>  // all but vm of this wave's vector loads are done, its LDS reads too
__device__ __forceinline__ void wait_stage() {
  __builtin_amdgcn_s_waitcnt((vm & 15) | ((vm >> 4) << 14) | 0x70);
}

// Loader of one operand's stages.  kRows: rows (K-inner) or columns (K-outer)
// of the tile; kPair: rows of two matrices, interleaved by 16.
template <bool kOuter, bool kPair, int kRows, int kWaves>
struct Loader {
  static constexpr int kLoads = kRows / 8 / kWaves;  // a wave's loads a stage
  static_assert(kRows % (8 * kWaves) == 0, "whole loads a wave");
  uint32_t off[kLoads];
  const char* base;
  const char* base2;
  long long left, left2, step;  // bytes to the end of the matrix; bytes a stage
  int kleft;                    // bytes of k to the end of a row (K-inner)
  int w;

  // tile: first row (K-inner, of each matrix) or column (K-outer)
  __device__ __forceinline__ void init(const Operand& o, int row0, int kbytes, int stage0,
                                       int stages_k, int wave, int lane) {
    w = wave;
    if (kOuter) {
      constexpr int kChunks = kRows / 8;  // 16-byte chunks a row
      const long long at = (long long)stage0 * kStageK * o.stride + 2LL * row0;
      base = o.p + at;
      left = (long long)stages_k * o.stride - at;  // stages_k: rows of k
      step = kStageK * o.stride;
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int i = (wave * kLoads + j) * 64 + lane;
        const int k = i / kChunks, pos = i % kChunks;
        const int g = (pos >> 1) ^ (((k & 3) | ((k >> 1) & 4)) & (kChunks / 2 - 1));
        off[j] = (uint32_t)(k * o.stride) + 32 * g + 16 * (pos & 1);
      }
    } else {
      const long long at = (long long)row0 * o.stride;
      const long long k0 = (long long)stage0 * kStageBytes;
      base = o.p + at + k0;
      left = (long long)o.rows * o.stride - at - k0;
      if (kPair) {
        base2 = o.p2 + at + k0;
        left2 = left;
      }
      step = kStageBytes;
      kleft = kbytes - (int)k0;
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int r = (wave * kLoads + j) * 8 + (lane >> 3);
        const int row = kPair ? (r >> 5) * 16 + (r & 15) : r;
        off[j] = (uint32_t)(row * o.stride) + 16 * ((lane & 7) ^ ((r >> 1) & 7));
      }
    }
  }

  // asks for the next stage into lds (the tile's first byte)
  __device__ __forceinline__ void load(char* lds, int lane) {
    const __amdgpu_buffer_rsrc_t r0 = rsrc_of(base, left);
    __amdgpu_buffer_rsrc_t r1 = r0;
    if (kPair) r1 = rsrc_of(base2, left);
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int i = w * kLoads + j;
      uint32_t o = off[j];
      if (!kOuter && kleft < kStageBytes) {
        const int r = i * 8 + (lane >> 3);
        if (16 * ((lane & 7) ^ ((r >> 1) & 7)) >= kleft) o = kOutOfRange;
      }
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          kPair && ((i >> 1) & 1) ? r1 : r0, (__attribute__((address_space(3))) void*)(lds + i * 1024),
          16, (int)o, 0, 0, 0);
    }
    base += step;
    left -= step;
    if (kPair) base2 += step;
    kleft -= kStageBytes;
  }
};

// Fragments of a stage: 16 rows from the tile's row 16 t on, k step ks (64
// bytes of k).
template <bool kOuter, int kRows, int kTiles>
struct Reader {
  uint32_t at[kOuter ? kTiles : 2];
  __device__ __forceinline__ void init(int row0, int lane) {  // the wave's first row
    const int i = lane & 15, q = lane >> 4;
    if (kOuter) {
      constexpr int kGran = kRows / 16;
      const int k = 8 * q + (i >> 2), f = ((k & 3) | ((k >> 1) & 4)) & (kGran - 1);
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
        at[t] = k * (2 * kRows) + (((row0 / 16 + t) ^ f) << 5) + 8 * (i & 3);
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s)
        at[s] = (row0 + i) * kStageBytes + (((4 * s + q) ^ ((i >> 1) & 7)) << 4);
    }
  }
  __device__ __forceinline__ u32x4 get(const char* lds, int t, int ks) const {
    if (kOuter) {
      typedef __attribute__((address_space(3))) i16x4* P;
      const char* b = lds + at[t] + ks * 32 * (2 * kRows);
      const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(b));
      const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(b + 4 * (2 * kRows)));
      const i16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      return __builtin_bit_cast(u32x4, v);
    }
    return *(const u32x4*)(lds + at[ks] + t * (16 * kStageBytes));
  }
};

// The matrix instruction on 64 bytes of k.
struct Bf16 {
  typedef f32x4 Acc;
  static __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    return mfma16(as_bf16x8(a), as_bf16x8(b), c);
  }
};
struct I8 {
  typedef i32x4 Acc;
  // two instructions of 32 bytes of k: both operands give them in the same order
  static __device__ __forceinline__ i32x4 mma(u32x4 a, u32x4 b, i32x4 c) {
    const u64x2 x = __builtin_bit_cast(u64x2, a), y = __builtin_bit_cast(u64x2, b);
    c = __builtin_amdgcn_mfma_i32_16x16x32_i8((long)x[0], (long)y[0], c, 0, 0, 0);
    return __builtin_amdgcn_mfma_i32_16x16x32_i8((long)x[1], (long)y[1], c, 0, 0, 0);
  }
};

// Four consecutive values as fp32 or bf16 (round to nearest even).
__device__ __forceinline__ void store4(void* p, int f32, size_t i, f32x4 v) {
  if (f32) {
    *(f32x4*)((float*)p + i) = v;
  } else {
    u32x2 w;
    w[0] = f32_to_bf16_rne(v[0]) | (f32_to_bf16_rne(v[1]) << 16);
    w[1] = f32_to_bf16_rne(v[2]) | (f32_to_bf16_rne(v[3]) << 16);
    *(u32x2*)((uint16_t*)p + i) = w;
  }
}

// Tile and wave counts of a configuration.
template <int bm, int bn, int wm, int wn, int stages>
struct Shape {
  static constexpr int BM = bm, BN = bn, WM = wm, WN = wn, S = stages;
  static constexpr int kWaves = wm * wn, kThreads = 64 * kWaves;
  static constexpr int kLds = (bm + bn) * kStageBytes * stages;
};

struct Problem {
  Operand a, b;
  int M, N;       // N: of the tile grid (pair form: 2 features a column pair)
  int kbytes;     // bytes of k in a row (K-inner)
  int krows;      // values of k: rows of a K-outer operand
  int stages;     // stages of k in all
  int per_split;  // stages of k a split
  int nm, nn;     // tiles
};

// Block -> tile.  Consecutive blocks go to the eight XCDs in turn; each XCD
// gets a run of neighbouring tiles (bands of 8 tile rows), so that its L2 serves
// the shared rows.
__device__ __forceinline__ void tile_of(int id, int nm, int nn, int& tm, int& tn) {
  const int n = nm * nn, per = n >> 3, rest = n & 7, x = id & 7;
  int i = (id >> 3) + x * per + min(x, rest);
  constexpr int kBand = 8;
  const int band = i / (kBand * nn), first = band * kBand, rows = min(kBand, nm - first);
  i -= first * nn;
  tm = first + i % rows;
  tn = i / rows;
}

// Epi: operator()(m, n, Acc) for four consecutive n, or in the pair form
// operator()(m, n, Acc first, Acc second).
template <typename Mma, typename Sh, bool kAOuter, bool kBOuter, bool kPair, typename Epi>
__global__ __launch_bounds__(Sh::kThreads, Sh::kWaves == 8 ? 2 : 1) void product_kernel(
    const Problem p, const Epi epi) {
  extern __shared__ __align__(1024) char lds[];
  constexpr int TM = Sh::BM / Sh::WM, TN = Sh::BN / Sh::WN, MI = TM / 16, NI = TN / 16;
  constexpr int kA = Sh::BM * kStageBytes, kStage = kA + Sh::BN * kStageBytes;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / Sh::WN, wn = wave % Sh::WN;
  int tm, tn;
  tile_of(blockIdx.x, p.nm, p.nn, tm, tn);
  const int m0 = tm * Sh::BM, n0 = tn * Sh::BN;
  const int stage0 = blockIdx.y * p.per_split;
  const int count = min(p.per_split, p.stages - stage0);

  Loader<kAOuter, false, Sh::BM, Sh::kWaves> la;
  Loader<kBOuter, kPair, Sh::BN, Sh::kWaves> lb;
  la.init(p.a, m0, p.kbytes, stage0, p.krows, wave, lane);
  lb.init(p.b, kPair ? n0 / 2 : n0, p.kbytes, stage0, p.krows, wave, lane);
  Reader<kAOuter, Sh::BM, MI> ra;
  Reader<kBOuter, Sh::BN, NI> rb;
  ra.init(wm * TM, lane);
  rb.init(wn * TN, lane);

  typename Mma::Acc acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = typename Mma::Acc{0, 0, 0, 0};

  constexpr int kLoads = decltype(la)::kLoads + decltype(lb)::kLoads;
  int put = 0, get = 0;
  auto ask = [&]() {  // past the last stage the loads are out of range
    char* s = lds + put * kStage;
    la.load(s, lane);
    lb.load(s + kA, lane);
    put = put + 1 == Sh::S ? 0 : put + 1;
  };
#pragma unroll
  for (int s = 0; s < Sh::S - 1; ++s) ask();
  for (int kt = 0; kt < count; ++kt) {
    // this wave's loads of the stage are through, and its reads of the stage
    // that the next loads overwrite; behind the barrier, every wave's
    wait_stage<(Sh::S - 2) * kLoads>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    ask();
    __builtin_amdgcn_sched_barrier(0);
    const char* s = lds + get * kStage;
    get = get + 1 == Sh::S ? 0 : get + 1;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      u32x4 fa[MI], fb[NI];
#pragma unroll
      for (int j = 0; j < NI; ++j) fb[j] = rb.get(s + kA, j, ks);
#pragma unroll
      for (int i = 0; i < MI; ++i) fa[i] = ra.get(s, i, ks);
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = Mma::mma(fb[j], fa[i], acc[i][j]);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  // The loads past the end land before the block's LDS is given back, and the
  // sums are formed before the branches below.
  wait_stage<0>();
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) asm volatile("" : "+v"(acc[i][j]));
  const int col = lane & 15, q = lane >> 4;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int m = m0 + wm * TM + 16 * i + col;
    if (m >= p.M) continue;
    if constexpr (kPair) {
#pragma unroll
      for (int j = 0; j < NI; j += 2) {
        const int n = (n0 + wn * TN) / 2 + 8 * j + 4 * q;
        if (n < p.N) epi(m, n, acc[i][j], acc[i][j + 1]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const int n = n0 + wn * TN + 16 * j + 4 * q;
        if (n < p.N) epi(m, n, acc[i][j]);
      }
    }
  }
}

}  // namespace mm
}  // namespace moe
