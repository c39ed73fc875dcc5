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
//   K-outer: row k takes 2 BM bytes.  A lane reads F = TM / 16 neighbouring
//     values of eight rows of k and pairs them up in registers, so that it holds
//     eight k of F fragments: fragment t is the tile's rows F r + t, r < 16 (the
//     LDS transpose read gives rows 16 t + r, but at a quarter of the rate:
//     8192^3 with both operands outer 888 us, this way 828 us).  Sixteen-byte chunk c
//     lies at c ^ s(k), which keeps the four octets of k on different banks.
//
// kScaled: A (K-inner) holds whole numbers of a unit in [1, 2) for each 128 values of
// a row, two stages.  Sums are in the unit of their last stage: a ratio of two units
// takes them from one to the next, and they are multiplied by the last one at the
// end.  So rows restored from 8-bit codes are not rounded to bf16 on their way here.
// Each row of sums is multiplied behind the matrix instructions of the row before: the
// gradient of 2048 tokens of 2048 through 1024 114.6 us, all of them between two stages
// 121, without units 112.
//
// Bound by the matrix cores where a launch fills the chip and k is long: bf16, the
// gated block's two products of 8192 tokens of 8192 values through 4096 features
// 1172 us, 1.41 PFLOP/s (the library's product 8192^3 713 us, 1.54, on the same
// card; its instructions alone 575 us); int8 8192^3 420 us, 2.6 POP/s (the
// library's 491).  Short k is bound by what a block does before and after its
// stages, 4 to 8 us of a 256 x 256 tile.  Tried without gain: deeper rings, a
// raised wave priority, 32 x 32 instructions (slower).
#pragma once
#include <type_traits>

#include "rowops.hpp"

namespace moe {
namespace mm {

using row::f32x8;
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));

constexpr int kStageBytes = 128;  // bytes of k a stage, K-inner
constexpr int kStageK = 64;       // rows of k a stage, K-outer
constexpr uint32_t kOutOfRange = 0x80000000u;

// One operand of a product.
struct Operand {
  const char* p;
  const char* p2;      // second matrix, interleaved by 16 rows (pair form), or null
  long long stride;    // bytes between rows
  int rows;            // rows of the product (m or n), per matrix
  const float* unit = nullptr;  // (kScaled) of each two stages of a row, [..][rows]
};

typedef __attribute__((address_space(3))) void* Lds;

// Offsets are below 2^31 where they are in range.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const char* p) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, 0x7FFFFFFF, 0x00020000);
}

template <int vm>  // all but vm of this wave's vector loads are done, its LDS reads too
__device__ __forceinline__ void wait_stage() {
  __builtin_amdgcn_s_waitcnt((vm & 15) | ((vm >> 4) << 14) | 0x70);
}

// Where row k of a K-outer stage has its chunks: a read takes 16, 32 or 64 lanes
// at a time (8, 4 or 2 values each), so 1, 2 or 4 octets of k.
template <int kRows, int kF>
__device__ __forceinline__ int swizzle(int k) {
  return kF >= 8 ? 0 : (((k >> 3) & (8 / kF - 1)) * 2 * kF) & (kRows / 8 - 1);
}

// Rows of a K-inner tile that its waves load in whole instructions, eight rows
// each; those past the tile are out of range and cost no traffic.
constexpr int whole_loads(int rows, int waves) {
  return (rows + 8 * waves - 1) / (8 * waves) * (8 * waves);
}

// Loader of one operand's stages.  kRows: rows (K-inner) or columns (K-outer)
// of the tile; kPair: rows of two matrices, interleaved by 16.
// kGroups: the stages are dealt to so many loaders in turn.
// kF: fragments of a wave's rows.
template <bool kOuter, bool kPair, int kRows, int kF, int kWaves, int kGroups>
struct Loader {
  static constexpr int kPlaces = whole_loads(kRows, kWaves);  // rows in LDS
  static constexpr int kLoads = kPlaces / 8 / kWaves;         // a wave's loads a stage
  static_assert(!kOuter || kRows == kPlaces, "whole loads a wave");
  uint32_t off[kLoads];    // bytes from the stage's base
  const char* base;        // of the next stage
  const char* base2;       // of the second matrix (pair form)
  long long step;          // bytes from one of its stages to the next
  int full;                // whole stages of k from the next one on
  int rest;                // bytes (K-inner) or rows (K-outer) of k after them
  int w, lane;

  // load j's row (K-inner) or row of k (K-outer), and its chunk of 16 bytes there
  __device__ __forceinline__ int row_of(int j) const {
    return kOuter ? ((w * kLoads + j) * 64 + lane) / (kRows / 8) : (w * kLoads + j) * 8 + (lane >> 3);
  }
  __device__ __forceinline__ int chunk_of(int j) const {
    const int r = row_of(j);
    if (!kOuter) return (lane & 7) ^ ((r >> 1) & 7);
    const int pos = ((w * kLoads + j) * 64 + lane) % (kRows / 8);
    return pos ^ swizzle<kRows, kF>(r);
  }

  // row0: the tile's first row (K-inner, of each matrix) or column (K-outer);
  // k: bytes (K-inner) or rows (K-outer) of k in all
  __device__ __forceinline__ void init(const Operand& o, int row0, int k, int stage0, int wave,
                                       int ln) {
    constexpr int kStage = kOuter ? kStageK : kStageBytes;
    w = wave;
    lane = ln;
    step = kOuter ? kStageK * o.stride : kStageBytes;
    const long long at = (kOuter ? 2LL * row0 : row0 * o.stride) + stage0 * step;
    base = o.p + at;
    if (kPair) base2 = o.p2 + at;
    step *= kGroups;
    full = k / kStage - stage0;
    rest = k % kStage;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int r = row_of(j), c = chunk_of(j);
      const int row = kPair ? (r >> 5) * 16 + (r & 15) : r;
      off[j] = (uint32_t)(row * o.stride) + 16 * c;
      if (row0 + (kOuter ? 8 * c : row) >= o.rows || r >= kRows) off[j] = kOutOfRange;
    }
    if (full <= 0) last();
  }

  // the stage that k ends in: what is past its end is out of range, and in the
  // stages after it everything
  __device__ __forceinline__ void last() {
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      if (full < 0 || (kOuter ? row_of(j) : 16 * chunk_of(j)) >= rest) off[j] = kOutOfRange;
  }

  // load j of the next stage into lds (the tile's first byte)
  __device__ __forceinline__ void load(int j, char* lds) const {
    const int i = w * kLoads + j;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rsrc_of(kPair && ((i >> 1) & 1) ? base2 : base), (Lds)(lds + i * 1024), 16, (int)off[j], 0,
        0, 0);
  }
  __device__ __forceinline__ void next() {
    base += step;
    if (kPair) base2 += step;
    full -= kGroups;
    if (full <= 0) last();
  }
};

// A wave's fragments of a stage, k step ks (64 bytes, 32 rows of k): what is read
// of LDS, and fragment t from it.
template <bool kOuter, int kRows, int kF>
struct Reader {
  static constexpr int kReads = kOuter ? 8 : kF;
  typedef uint32_t Part __attribute__((ext_vector_type(kOuter ? (kF < 8 ? kF / 2 : 4) : 4)));
  struct Raw {
    Part v[kReads];
  };
  static_assert(!kOuter || kF == 2 || kF == 4 || kF == 8, "whole reads");
  uint32_t at[kOuter ? 1 : 2];
  __device__ __forceinline__ void init(int row0, int lane) {  // the wave's first row
    const int i = lane & 15, q = lane >> 4;
    if (kOuter) {
      const int b = 2 * row0 + 2 * kF * i;  // byte of a row; swizzled by chunks of 16
      at[0] = 8 * q * (2 * kRows) + (b ^ (16 * swizzle<kRows, kF>(8 * q)));
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s)
        at[s] = (row0 + i) * kStageBytes + (((4 * s + q) ^ ((i >> 1) & 7)) << 4);
    }
  }
  __device__ __forceinline__ void read(Raw& raw, const char* lds, int r, int ks) const {
    raw.v[r] = kOuter ? *(const Part*)(lds + at[0] + (32 * ks + r) * (2 * kRows))
                      : *(const Part*)(lds + at[kOuter ? 0 : ks] + r * (16 * kStageBytes));
  }
  // dword p (k = 2 p, 2 p + 1) of fragment t of an outer operand
  __device__ __forceinline__ uint32_t part(const Raw& raw, int t, int p) const {
    return __builtin_amdgcn_perm(raw.v[2 * p + 1][t >> 1], raw.v[2 * p][t >> 1],
                                 t & 1 ? 0x07060302u : 0x05040100u);
  }
  __device__ __forceinline__ u32x4 get(const Raw& raw, int t) const {
    if constexpr (kOuter)
      return u32x4{part(raw, t, 0), part(raw, t, 1), part(raw, t, 2), part(raw, t, 3)};
    else
      return raw.v[t];
  }
  // The wave's row that lane column c (of 16) of fragment t holds.
  static __device__ __forceinline__ int row(int t, int c) { return kOuter ? kF * c + t : 16 * t + c; }
};

// The matrix instruction on 64 bytes of k.
struct Bf16 {
  typedef float Value;
  typedef f32x4 Acc;
  typedef f32x8 Acc8;
  static __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    return mfma16(as_bf16x8(a), as_bf16x8(b), c);
  }
  static __device__ __forceinline__ f32x4 times(f32x4 c, float f) { return c * f; }
};
struct I8 {
  typedef int32_t Value;
  typedef i32x4 Acc;
  typedef i32x8 Acc8;
  static __device__ __forceinline__ Acc mma(u32x4 a, u32x4 b, Acc c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a),
                                                 __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ Acc times(Acc c, float) { return c; }  // (not called)
};

// Four or eight consecutive values (V: f32x4, f32x8) of an fp32 array, and to one that
// is fp32 or bf16 (round to nearest even).
template <typename V>
__device__ __forceinline__ V load_f32(const float* p, size_t i) {
  if constexpr (sizeof(V) == 32)
    return row::load8<true>(p, i);
  else
    return *(const V*)(p + i);
}
template <typename V>
__device__ __forceinline__ void store_as(void* p, int f32, size_t i, V v) {
  if (f32) {
    *(V*)((float*)p + i) = v;
  } else {
    // (two values an instruction; in integer arithmetic the conversion takes seven
    // each, 3 us of a 256 x 256 tile)
    typedef __bf16 Half __attribute__((ext_vector_type(sizeof(V) / 4)));
    *(Half*)((uint16_t*)p + i) = __builtin_convertvector(v, Half);
  }
}

// A configuration: tile, waves along m and n, stages in the rings, groups of
// waves that share the tile's k (each with rings of its own, joined in LDS), and
// stages that B's ring has more than A's.
template <int bm, int bn, int wm, int wn, int stages, int groups = 1, int more = 0>
struct Shape {
  static constexpr int BM = bm, BN = bn, WM = wm, WN = wn, S = stages, G = groups, SB = S + more;
  static constexpr int kWaves = wm * wn, kThreads = 64 * kWaves * groups;  // waves: of a group
  static constexpr int kA = whole_loads(bm, kWaves) * kStageBytes, kB = bn * kStageBytes;
  static constexpr int kRing = kA * S + kB * SB;
  static constexpr int kLds = groups * kRing;
};

struct Problem {
  Operand a, b;
  int M, N;       // N: of the tile grid (pair form: 2 features a column pair)
  int kbytes;     // bytes of k in a row (K-inner)
  int krows;      // values of k: rows of a K-outer operand
  int stages;     // stages of k in all
  int per_group;  // stages of k a group of waves
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

// What an epilogue reads from memory is asked for before the rows are turned
// around: Epi::Columns by columns(n), once, and Epi::Ahead by ahead(m, n), for a
// piece of a row; nothing where it has no such types.
template <typename Epi, typename = void>
struct ReadAhead {
  struct Type {};
  struct Columns {};
  static __device__ __forceinline__ Type get(const Epi&, int, int) { return {}; }
  static __device__ __forceinline__ Columns columns(const Epi&, int) { return {}; }
  static constexpr int kDepth = 0;
};
template <typename Epi>
struct ReadAhead<Epi, std::void_t<typename Epi::Ahead>> {
  typedef typename Epi::Ahead Type;
  typedef typename Epi::Columns Columns;
  static __device__ __forceinline__ Type get(const Epi& epi, int m, int n) {
    return epi.ahead(m, n);
  }
  static __device__ __forceinline__ Columns columns(const Epi& epi, int n) {
    return epi.columns(n);
  }
  static constexpr int kDepth = 64 / Type::kRegs;  // pieces in flight, in 64 registers
};

// Epilogues that keep values of a thread from one product of a block to the next
// take the round's number last (Epi::kRounds of them): a thread has the same rows
// and columns in every product of the same waves and tile.
template <typename Epi, typename = void>
struct ByRound : std::false_type {};
template <typename Epi>
struct ByRound<Epi, std::void_t<decltype(Epi::kRounds)>> : std::true_type {};

// Epi: operator()(m, n, v) for eight consecutive n (N is a multiple of 8; the
// direct kernel: four), or in the pair form operator()(m, n, first, second).
// With Epi::Ahead: operator()(m, n, v, columns(n), ahead(m, n)).
// id: the block's among the tiles' blocks; part: its share of k.
template <typename Mma, typename Sh, bool kAOuter, bool kBOuter, bool kPair, bool kScaled,
          typename Epi>
__device__ __forceinline__ void product_block(const Problem& p, const Epi& epi, char* lds, int id,
                                              int part) {
  constexpr int TM = Sh::BM / Sh::WM, TN = Sh::BN / Sh::WN, MI = TM / 16, NI = TN / 16;
  constexpr int kA = Sh::kA, kB = Sh::kB;
  const int lane = threadIdx.x & 63;
  const int any = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = any / Sh::kWaves, wave = any % Sh::kWaves;
  const int wm = wave / Sh::WN, wn = wave % Sh::WN;
  char* const ring = lds + group * Sh::kRing;
  int tm, tn;
  tile_of(id, p.nm, p.nn, tm, tn);
  const int m0 = tm * Sh::BM, n0 = tn * Sh::BN;
  // The groups take the block's stages in turn, so that together they read long
  // pieces of a row; past the end of k stages are zeros.
  const int block0 = part * Sh::G * p.per_group, stage0 = block0 + group;
  const int count = min(p.per_group, (p.stages - block0 + Sh::G - 1) / Sh::G);

  Loader<kAOuter, false, Sh::BM, MI, Sh::kWaves, Sh::G> la;
  Loader<kBOuter, kPair, Sh::BN, NI, Sh::kWaves, Sh::G> lb;
  la.init(p.a, m0, kAOuter ? p.krows : p.kbytes, stage0, wave, lane);
  lb.init(p.b, kPair ? n0 / 2 : n0, kBOuter ? p.krows : p.kbytes, stage0, wave, lane);
  Reader<kAOuter, Sh::BM, MI> ra;
  Reader<kBOuter, Sh::BN, NI> rb;
  ra.init(wm * TM, lane);
  rb.init(wn * TN, lane);

  typename Mma::Acc acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = typename Mma::Acc{0, 0, 0, 0};

  constexpr int kLA = decltype(la)::kLoads, kLoads = kLA + decltype(lb)::kLoads;
  // The rings' next places: to load into, and to read.
  struct Place {
    int put = 0, get = 0;
  } at_a, at_b;
  auto after = [](int i, int stages) { return i + 1 == stages ? 0 : i + 1; };
  char* const ring_b = ring + Sh::S * kA;
  auto ask = [&](int j) {  // (past the last stage the loads are out of range)
    if (j < kLA)
      la.load(j, ring + at_a.put * kA);
    else
      lb.load(j - kLA, ring_b + at_b.put * kB);
  };
  auto asked_a = [&]() {
    la.next();
    at_a.put = after(at_a.put, Sh::S);
  };
  auto asked_b = [&]() {
    lb.next();
    at_b.put = after(at_b.put, Sh::SB);
  };
  struct Frags {
    typename decltype(ra)::Raw a;
    typename decltype(rb)::Raw b;
  } f0, f1;
  constexpr int kReadsB = decltype(rb)::kReads, kReads = kReadsB + decltype(ra)::kReads;
  auto read = [&](Frags& f, int r, int ks) {
    if (r < kReadsB)
      rb.read(f.b, ring_b + at_b.get * kB, r, ks);
    else
      ra.read(f.a, ring + at_a.get * kA, r - kReadsB, ks);
  };
  // A lane has the units of rows lane, lane + 64 of the wave's.
  constexpr int kUnits = kScaled ? (TM + 63) / 64 : 1;
  struct Units {
    float v[kUnits];
  } unit, after_unit, later_unit;  // of the sums, of the next group, as asked for
  float factor[MI];                // from the first to the second, of a fragment's rows
  static_assert(!kScaled || !kAOuter, "rows of a K-inner operand, k not split");
  auto units_of = [&](int kt) {
    const int stage = min(stage0 + Sh::G * kt, p.stages - 1);
    Units u;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      int row = m0 + wm * TM + 64 * i + lane;
      asm volatile("" : "+v"(row));  // (not kept in a register)
      row = min(row, p.M - 1);
      u.v[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
          rsrc_of((const char*)p.a.unit), 4 * row, 4 * p.M * (stage >> 1), 0));
    }
    return u;
  };
  auto by_fragment = [&](const Units& u) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
      factor[i] = __shfl(u.v[16 * i / 64], (16 * i + (lane & 15)) & 63, kWave);
  };
  if constexpr (kScaled) {
    unit = after_unit = units_of(0);
    later_unit = units_of(1);
#pragma unroll
    for (int i = 0; i < MI; ++i) factor[i] = 1.0f;
  }
  // The products of one k step; between its rows the fragments of the next step
  // are asked for (in its first rows) and, `loads`, the next stage's loads: all
  // at once they would hold the wave up while the memory pipe takes them in.
  constexpr int kHalf = (MI + 1) / 2;
  // An outer operand's fragments are made one row of products ahead.
  u32x4 b[NI], a;
  // Rows of sums that go to another unit first do so behind the products of the row
  // before them.
  auto multiply = [&](const Frags& f, Frags& next, int ks, auto from, auto to, auto rescale) {
    constexpr int kFrom = decltype(from)::value, kMore = decltype(to)::value - kFrom;
    constexpr bool kRescale = decltype(rescale)::value;
    if constexpr (kRescale) {
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[0][j] = Mma::times(acc[0][j], factor[0]);
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      if (i < kHalf)
#pragma unroll
        for (int r = i * kReads / kHalf; r < (i + 1) * kReads / kHalf; ++r) read(next, r, ks);
#pragma unroll
      for (int j = i * kMore / MI; j < (i + 1) * kMore / MI; ++j) ask(kFrom + j);
      if (!kAOuter) a = ra.get(f.a, i);
      if (!kBOuter && i == 0)
#pragma unroll
        for (int j = 0; j < NI; ++j) b[j] = rb.get(f.b, j);
      u32x4 ahead;
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        acc[i][j] = Mma::mma(b[j], a, acc[i][j]);
        if constexpr (kRescale) {
          if (i + 1 < MI) acc[i + 1][j] = Mma::times(acc[i + 1][j], factor[i + 1]);
          if (MI < 8) __builtin_amdgcn_sched_barrier(0);  // (256 x 256 would spill)
        }
        if constexpr (kAOuter) {
#pragma unroll
          for (int q = j * 4 / NI; q < (j + 1) * 4 / NI; ++q)
            ahead[q] = i + 1 < MI ? ra.part(f.a, i + 1, q) : ra.part(next.a, 0, q);
          __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (kBOuter) {
          if (i + 1 == MI) b[j] = rb.get(next.b, j);
        }
      }
      if (kAOuter) a = ahead;
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  using std::integral_constant;
  constexpr bool kApart = Sh::SB > Sh::S;  // B's loads in the other half than A's
  constexpr integral_constant<int, 0> kFirst{};
  constexpr integral_constant<int, kLA> kBetween{};
  constexpr integral_constant<int, kLoads> kLast{};
#pragma unroll
  for (int s = 0; s < Sh::S; ++s) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) ask(j);
    asked_a();
    asked_b();
  }
  wait_stage<(Sh::S - 1) * kLoads>();
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int r = 0; r < kReads; ++r) read(f0, r, 0);
  a = ra.get(f0.a, 0);
#pragma unroll
  for (int j = 0; j < NI; ++j) b[j] = rb.get(f0.b, j);
  // One stage.  kScaled: the first or the last of its group, of this wave's stages.
  constexpr std::false_type kNo{};
  auto step = [&](int kt, auto first, auto last) __attribute__((always_inline)) {
    if constexpr (decltype(first)::value) unit = after_unit;
    if constexpr (kApart) {
      multiply(f0, f1, 1, kBetween, kLast, first);
      asked_b();
    } else {
      multiply(f0, f1, 1, kFirst, kFirst, first);
    }
    // this wave's loads of the next stage are through (behind them are S - 2
    // stages' loads, or B's loads of this half), and its reads of the one that
    // the next loads overwrite; behind the barrier, every wave's
    wait_stage<(Sh::S - 2) * kLoads + (kApart ? kLoads - kLA : 0)>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    at_a.get = after(at_a.get, Sh::S);
    at_b.get = after(at_b.get, Sh::SB);
    // (units are asked for between two stages' loads, so that no wait is longer)
    if constexpr (decltype(last)::value) {
      after_unit = later_unit;
      Units ratio;
#pragma unroll
      for (int i = 0; i < kUnits; ++i)
        ratio.v[i] = unit.v[i] * __builtin_amdgcn_rcpf(after_unit.v[i]);
      by_fragment(ratio);
    }
    if constexpr (decltype(first)::value && !kApart) later_unit = units_of(kt + 2);
    if constexpr (kScaled) __builtin_amdgcn_sched_barrier(0);
    if constexpr (kApart) {
      multiply(f1, f0, 0, kFirst, kBetween, kNo);
    } else {
      multiply(f1, f0, 0, kFirst, kLast, kNo);
      asked_b();
    }
    asked_a();
    if constexpr (decltype(first)::value && kApart) later_unit = units_of(kt + 2);
  };
  if constexpr (kScaled) {
    constexpr std::true_type kYes{};
    constexpr std::integral_constant<bool, (Sh::G > 1)> kEach{};  // (a group a stage)
    for (int kt = 0; kt < count; kt += 2) {
      step(kt, kYes, kEach);
      if (kt + 1 == count) break;
      step(kt + 1, kEach, kYes);
    }
  } else {
    for (int kt = 0; kt < count; ++kt) step(kt, kNo, kNo);
  }
  typedef typename Mma::Acc8 Acc8;
  constexpr int kRow = TN * 4 + 16, kWidth = kPair ? TN / 2 : TN;  // features of the wave
  constexpr int kLanes = kWidth / 8, kPass = 64 / kLanes < 16 ? 64 / kLanes : 16;  // rows at a time
  constexpr int kPasses = (16 + kPass - 1) / kPass, kRounds = MI * kPasses;
  const int row = lane / kLanes, at = 8 * (lane % kLanes);
  const int n = (kPair ? n0 / 2 : n0) + wn * kWidth + at;
  auto row_of = [&](int round) {
    return m0 + wm * TM +
           decltype(ra)::row(round / kPasses, round % kPasses * kPass + row);
  };
  // what the epilogue reads of the first rounds
  typedef ReadAhead<Epi> Early;
  constexpr int kDepth = Early::kDepth < kRounds ? Early::kDepth : kRounds;
  typename Early::Type early[kDepth ? kDepth : 1];
  auto fetch = [&](int round) {  // (rows and columns past the end read the last)
    early[round % (kDepth ? kDepth : 1)] =
        Early::get(epi, min(row_of(round), p.M - 1), min(n, p.N - 8));
  };
#pragma unroll
  for (int r = 0; r < kDepth; ++r) fetch(r);
  const typename Early::Columns columns = Early::columns(epi, min(n, p.N - 8));
  // The loads past the end land before the block's LDS is given back, and the
  // sums are formed before the branches below.
  wait_stage<0>();
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) asm volatile("" : "+v"(acc[i][j]));
  if constexpr (kScaled) {
    by_fragment(unit);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[i][j] = Mma::times(acc[i][j], factor[i]);
  }
  if constexpr (Sh::G > 1) {
    typedef typename Mma::Acc Quad;
    Quad* red = (Quad*)lds + wave * (MI * NI * 64) + lane;
    constexpr int kGroup = Sh::kWaves * MI * NI * 64;
    __syncthreads();  // the sums take the stages' place
    if (group > 0) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) red[(group - 1) * kGroup + (i * NI + j) * 64] = acc[i][j];
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 1; g < Sh::G; ++g)
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] += red[(g - 1) * kGroup + (i * NI + j) * 64];
  }
  // A lane's four values of 16 rows would go to memory in pieces of 32 bytes, so
  // each wave turns its rows around in LDS, 16 at a time, and writes 128 bytes of
  // a row together (64 with TN = 32).
  __syncthreads();  // the last stage has been read (or, of a group, the sums)
  char* const turn = lds + (Sh::G - 1) * (Sh::kWaves * MI * NI * 1024) + wave * (16 * kRow);
  const int col = lane & 15, q = lane >> 4;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    char* const to = turn + col * kRow;
    if constexpr (kBOuter) {  // NI neighbouring columns, one of each fragment
      typedef typename Mma::Value Row __attribute__((ext_vector_type(NI)));
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        Row v;
#pragma unroll
        for (int j = 0; j < NI; ++j) v[j] = acc[i][j][r];
        *(Row*)(to + 4 * NI * (4 * q + r)) = v;
      }
    } else {
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const int c = kPair ? (j & 1) * kWidth + 8 * (j & ~1) : 16 * j;  // the tile's columns
        *(typename Mma::Acc*)(to + 4 * (c + 4 * q)) = acc[i][j];
      }
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int r = 0; r < kPasses; ++r) {
      const int round = i * kPasses + r, at_row = r * kPass + row, m = row_of(round);
      if (at_row < 16 && m < p.M && n < p.N) {
        const char* v = turn + at_row * kRow + 4 * at;
        if constexpr (ByRound<Epi>::value && kPair)
          epi(m, n, *(const Acc8*)v, *(const Acc8*)(v + 4 * kWidth), round);
        else if constexpr (ByRound<Epi>::value)
          epi(m, n, *(const Acc8*)v, round);
        else if constexpr (kDepth > 0)
          epi(m, n, *(const Acc8*)v, columns, early[round % kDepth]);
        else if constexpr (kPair)
          epi(m, n, *(const Acc8*)v, *(const Acc8*)(v + 4 * kWidth));
        else
          epi(m, n, *(const Acc8*)v);
      }
      if (kDepth && round + kDepth < kRounds) fetch(round + kDepth);
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
  }
}

template <typename Mma, typename Sh, bool kAOuter, bool kBOuter, bool kPair, bool kScaled,
          typename Epi>
__global__ __launch_bounds__(Sh::kThreads, Sh::kThreads / 256) void product_kernel(
    const Problem p, const Epi epi) {
  extern __shared__ __align__(1024) char lds[];
  product_block<Mma, Sh, kAOuter, kBOuter, kPair, kScaled>(p, epi, lds, blockIdx.x, blockIdx.y);
}

// Products that do not wait for each other, in one launch: one of the first kind
// and up to two of the second, whose blocks follow.
template <typename Shape_, bool kAOuter, bool kBOuter, bool kPair, bool kScaled, typename Epi_>
struct Part {
  typedef Shape_ Sh;
  typedef Epi_ Epi;
  Problem p;
  Epi epi;
  int blocks;  // a multiple of 8, so that a tile's XCD is the one it has alone
  __device__ __forceinline__ void run(char* lds, int id) const {
    if (id < p.nm * p.nn)
      product_block<Bf16, Sh, kAOuter, kBOuter, kPair, kScaled>(p, epi, lds, id, 0);
  }
};

template <typename First, typename Second>
__global__ __launch_bounds__(First::Sh::kThreads, First::Sh::kThreads / 256) void joint_kernel(
    const First a, const Second b, const Second c, int shift) {
  static_assert(First::Sh::kThreads == Second::Sh::kThreads, "blocks of one size");
  extern __shared__ __align__(1024) char lds[];
  int id = blockIdx.x + shift;
  if (id >= (int)gridDim.x) id -= gridDim.x;
  const int after = id - a.blocks;
  if (after < 0)
    a.run(lds, id);
  else if (after < b.blocks)
    b.run(lds, after);
  else
    c.run(lds, after - b.blocks);
}

}  // namespace mm
}  // namespace moe
