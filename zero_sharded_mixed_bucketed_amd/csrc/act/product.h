// Products of 16-bit matrices on the matrix instructions, with the reduction axis k
// either fast (rows of neighbouring k) or slow (rows of neighbouring outputs) in
// each operand, and a caller's own epilogue:
//   c(m, n) = sum over k of a(m, k) b(n, k),  fp32 sums of exact products.
//
// A workgroup of four waves makes a TM x TN tile of c, 64 of k at a time, through two
// buffers of shared memory and one barrier a turn.  While the matrix unit works on
// one tile, the next one goes from registers to the other buffer and the one after
// it is loaded into those registers; the operands of a matrix step are read from
// shared memory during the step before it.
//   - k fast: a row's 64 k are eight 16-byte chunks, placed by chunk ^ (row / 2 % 8),
//     so that sixteen neighbouring rows of one chunk lie in different banks; a lane
//     reads its eight k with one load.
//   - k slow: rows of TILE columns as they come, in 64-byte granules permuted by k,
//     read with the transposing loads.
#ifndef ZERO_ACT_PRODUCT_H_
#define ZERO_ACT_PRODUCT_H_

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act/format.h"
#include "act/launch.h"

namespace zero {
namespace act {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef __bf16 bhalf8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kMulThreads = 256;  // four waves
constexpr int kMulFrag = 32;      // rows and columns of a matrix instruction
constexpr int kMulStep = 16;      // k of a matrix instruction
constexpr int kMulDepth = 64;     // k of a turn

// One operand in device memory.  extent: rows (k fast) or columns (k slow) that
// exist; of two stacked matrices (an epilogue of pairs) those of each.
struct Operand {
  const uint16_t* p;
  uint64_t stride, extent;
  bool padded;   // its fast axis is followed by zeros up to a whole chunk
};

// In a count: half of what it counts stands a second time, behind the others.  It comes
// with the count, in one load.
constexpr uint32_t kTwice = 1u << 31;

// The sizes of a product.  A count in device memory, where there is one, says how
// many rows of c (or, with count_k, how many k) there are past `first`, at most m
// (k): the host knows the most only.
struct Extents {
  uint64_t m, n, k;
  uint32_t splits;          // of k, each a range of whole turns
  uint32_t most, fill;      // see splits_of
  const uint32_t* count;
  uint64_t first;
  int count_k;
};

__device__ __forceinline__ uint64_t counted(const Extents& x, uint64_t most, bool* twice) {
  const uint32_t held = *x.count;
  const uint64_t c = held & ~kTwice;
  const uint64_t left = c > x.first ? c - x.first : 0;
  *twice = (held & kTwice) != 0;
  return left < most ? left : most;
}

// The splits of a product whose rows are counted on the device: as planned for the most
// rows, or with fewer tiles than that what fills the chip, `fill` workgroups, but not over
// `most`.  (1200 of 3001 tokens with a loss, 50001 words at 2050: dx 510 -> 290 us with its join.)
__host__ __device__ inline uint32_t splits_of(uint32_t splits, uint32_t most, uint32_t fill,
                                              uint32_t tiles) {
  if (most <= splits || tiles == 0) return splits;
  const uint32_t s = fill / tiles;
  return s <= splits ? splits : s < most ? s : most;
}

template <typename T>
__device__ __forceinline__ f32x16 mul(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (T::kType == kF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, a),
                                                  __builtin_bit_cast(half8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bhalf8, a),
                                                   __builtin_bit_cast(bhalf8, b), c, 0, 0, 0);
}

// Orders one wave's shared-memory accesses before and after this point.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// One operand's side of a workgroup: its loads, its shared tile and its fragments.
// PAIR != 0: the operand is two stacked matrices, and a tile holds PAIR rows of the
// first, the same rows of the second, the next PAIR rows of the first, and so on.
template <bool FAST, int TILE, int PAIR = 0>
struct Side {
  static_assert(FAST ? TILE % 32 == 0 : TILE >= 128 && !PAIR, "granules are permuted in fours");
  static constexpr int kPass = TILE / 32;                   // loads of a thread a turn
  static constexpr uint32_t kLanes = FAST ? kMulDepth / kChunk : TILE / kChunk;
  static constexpr uint32_t kStep = kMulThreads / kLanes;   // rows of memory a pass
  static constexpr uint32_t kElems = TILE * kMulDepth;
  static constexpr int kReads = FAST ? 1 : 2;               // shared loads a fragment

  const uint16_t* p;       // row (k fast) or row 0 (k slow) of the tile
  uint64_t stride, extent, first;
  uint32_t row, chunk;     // of this thread in a pass
  uint32_t off[FAST ? kPass : 1];

  __device__ __forceinline__ uint64_t row_of(uint32_t r) const {   // k fast
    if constexpr (PAIR != 0) {
      const uint64_t at = first + r / (2 * PAIR) * PAIR + r % PAIR;
      return (at < extent ? at : extent - 1) + (r / PAIR % 2 ? extent : 0);
    }
    const uint64_t at = first + r;
    return at < extent ? at : extent - 1;
  }

  // Rows and columns past the matrix's edge take the last row or column 0: they reach
  // only sums that are not kept.
  __device__ __forceinline__ void begin(const Operand& o, uint64_t at) {
    stride = o.stride;
    extent = o.extent;
    first = at;
    row = threadIdx.x / kLanes;
    chunk = threadIdx.x % kLanes * kChunk;
    if constexpr (FAST) {
      p = o.p + first * stride;
#pragma unroll
      for (int i = 0; i < kPass; ++i)
        off[i] = static_cast<uint32_t>(((row_of(i * kStep + row) - first) * stride + chunk) * 2);
    } else {
      p = o.p;
      off[0] = (row * static_cast<uint32_t>(stride) +
                static_cast<uint32_t>(first + chunk < extent ? first + chunk : 0)) * 2;
    }
  }

  // Without a check: turns that end before k `safe` (see safe_k).
  __device__ __forceinline__ u32x4 load(uint64_t k, int i) const {
    const uint8_t* at;
    if constexpr (FAST)
      at = reinterpret_cast<const uint8_t*>(p + k) + off[i];
    else
      at = reinterpret_cast<const uint8_t*>(p + (k + i * kStep) * stride) + off[0];
    return *reinterpret_cast<const u32x4_at2*>(at);
  }

  // With every check: 0 from k_hi on and past the columns' edge.
  __device__ __forceinline__ u32x4 load_checked(uint64_t k, uint64_t k_hi, int i) const {
    if constexpr (FAST) {
      if (k + chunk >= k_hi) return u32x4{0, 0, 0, 0};
      return load8(p + (row_of(i * kStep + row) - first) * stride, k + chunk, k_hi);
    } else {
      const uint64_t t = k + i * kStep + row;
      if (t >= k_hi || first + chunk >= extent) return u32x4{0, 0, 0, 0};
      return load8(p + t * stride, first + chunk, extent);
    }
  }

  __device__ __forceinline__ void stage(uint16_t* tile, int i, u32x4 w) const {
    const uint32_t r = i * kStep + row;
    uint16_t* at;
    if constexpr (FAST)
      at = tile + r * kMulDepth + (chunk ^ ((r / 2 % 8) * kChunk));
    else
      at = tile + r * TILE + ((((chunk >> 5) ^ (r & 3)) << 5) | (chunk & 31));
    *reinterpret_cast<u32x4*>(at) = w;
  }

  // Part q of kReads of a fragment: 32 rows from `at` on, 16 k from `step` * 16 on.
  // Lane l gets row l % 32 of eight k, from 8 (l / 32) on.
  static __device__ __forceinline__ void read(const uint16_t* tile, int step, uint32_t at, int q,
                                              u32x4& to) {
    const uint32_t lane = threadIdx.x % 64;
    if constexpr (FAST) {
      const uint32_t r = at + lane % 32, c = step * 2 + lane / 32;
      to = *reinterpret_cast<const u32x4*>(tile + r * kMulDepth + ((c ^ (r / 2 % 8)) * kChunk));
    } else {
      typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
      const uint32_t r = step * kMulStep + (lane / 32) * 8 + (lane % 16) / 4 + q * 4;
      const uint32_t c = at + (lane / 16 % 2) * 16 + lane % 4 * 4;
      const uint16_t* from = tile + r * TILE + ((((c >> 5) ^ (r & 3)) << 5) | (c & 31));
      const u32x2 v = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                     (lds_s16x4*)(__attribute__((address_space(3))) uint16_t*)from));
      to[2 * q] = v[0];
      to[2 * q + 1] = v[1];
    }
  }
};

// The k below which an operand's turns may be loaded without a check: whole chunks
// stay inside the matrix's memory, and offsets inside a tile within 32 bits.
inline uint64_t safe_k(const Operand& o, bool fast, uint64_t k, bool pairs = false) {
  constexpr uint64_t kFar = 1ull << 30;
  if (o.stride >= kFar / 512) return 0;
  if (fast) return ((pairs ? o.extent : 0) + 256) * o.stride < kFar * 2 - kMulDepth ? k : 0;
  const uint64_t over = (kChunk - o.extent % kChunk) % kChunk;
  if (over == 0) return k;
  const uint64_t back = k > 1 ? (over + o.stride - 1) / o.stride : k;
  return back < k ? k - back : 0;
}

// The tile and split of a workgroup.  Workgroups go to the eight dies in turn, each
// with an L2 of its own: die x takes the x-th eighth of the pieces, and pieces run
// down groups of eight tile rows, so that the 32 that a die has in hand together
// read 8 + 4 strips of the operands.
struct Spot {
  uint32_t split, m, n;
};

__device__ __forceinline__ Spot spot_of(uint32_t wg, uint32_t wgs, uint32_t tiles_m,
                                        uint32_t tiles_n) {
  constexpr uint32_t kDies = 8, kGroup = 8;
  const uint32_t die = wg % kDies, each = wgs / kDies, more = wgs % kDies;
  const uint32_t id = die * each + (die < more ? die : more) + wg / kDies;
  const uint32_t tiles = tiles_m * tiles_n;
  const uint32_t split = id / tiles, tile = id % tiles;
  const uint32_t group = tile / (kGroup * tiles_n), rest = tile % (kGroup * tiles_n);
  const uint32_t row0 = group * kGroup;
  const uint32_t rows = tiles_m - row0 < kGroup ? tiles_m - row0 : kGroup;
  return {split, row0 + rest % rows, rest / rows};
}

// A wave's sums, FM x FN fragments from row m0 and column n0 on, to an epilogue.  b's
// fragment is the matrix instructions' first operand, so the sums' rows are the lanes'
// (l % 32), and a lane has four neighbouring columns of a row at a time.  Through shared
// memory (`piece`, 32 rows of 64 columns), it gets eight; the 16-byte pieces are permuted
// by row, so that sixteen neighbouring rows of one lie in different banks.
//
// An epilogue E holds what it writes.  put<T>(split, m, n, rows, x) takes eight
// neighbouring sums x of row m, from column n on (a multiple of eight; rows from `rows`
// on and columns past the edge among them); with E::kPairs, put<T>(split, m, n, rows, x,
// y) those of the same columns of both stacked matrices.  All lanes of a wave call it
// together.  With E::kRows, columns(row, x, m, n, rows) sees each lane's sums x of row m
// first, half of the columns at a time, the others in lane ^ 32, with a Row of its own to
// keep, which finish(row, m, piece, rows) gets in the end, `piece` being which of the
// row's 32 FN columns these were.  stores() says whether there is anything to store.
// simple() says whether a whole
// tile needs none of put's checks: now<false>(split, m0, factor) then gives what stores it
// (now<true> with E::kAdds, if adds(): what it adds to is read ahead), factor what
// load_factor() gave at the kernel's begin; row_of(i, line, m) is the row at
// which it stores row m, line `line` of the wave's i-th 32.
template <typename T, bool WHOLE, int FM, int FN, typename E, typename P>
__device__ __forceinline__ void wave_store(const f32x16 (&acc)[FM][FN], float* piece, const E& e,
                                           const P& to, uint32_t split, uint64_t m0, uint64_t n0,
                                           uint64_t m_all) {
  constexpr int kWide = !E::kPairs && FN > 1 ? 2 : 1;       // fragments of c beside each other
  constexpr uint32_t kLanes = kWide * 4, kLines = 64 / kLanes, kPass = 32 / kLines;
  constexpr int kUnroll = WHOLE && !E::kPairs ? kPass : 1;
  constexpr int kTurns = E::kPairs ? FN / 2 : FN / kWide;
  constexpr int kHeld = E::kPairs ? 2 : kWide;              // fragments a turn
  constexpr bool kOld = WHOLE && P::kOld;
  const uint32_t lane = threadIdx.x % 64, c = lane % kLanes;
  const auto column = [&](int step) __attribute__((always_inline)) {
    return n0 + step % kTurns * (kWide * kMulFrag) + c * kChunk;
  };
  // What is added, read before the turn through shared memory where it fits.
  constexpr uint32_t kAhead = kPass / 2;
  [[maybe_unused]] typename P::Old old[kAhead];
  [[maybe_unused]] const auto fetch = [&](int step, uint32_t r0) __attribute__((always_inline)) {
    if constexpr (kOld) {
#pragma unroll
      for (uint32_t r = r0; r < r0 + kAhead; ++r)
        old[r % kAhead] = to.fetch(m0 + step / kTurns * kMulFrag + r * kLines + lane / kLanes,
                            column(step));
    }
  };
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    [[maybe_unused]] typename E::Row row;
#pragma unroll
    for (int h = 0; h < kTurns; ++h) {
      const int step = i * kTurns + h;
      fetch(step, 0);
#pragma unroll
      for (int j = 0; j < kHeld; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const f32x16& v = acc[i][E::kPairs ? h + kTurns * j : kWide * h + j];
          const uint32_t line = lane % 32, q = j * 8 + r * 2 + lane / 32;
          *reinterpret_cast<f32x4*>(piece + line * 64 + ((q ^ (line % 16)) * 4)) =
              f32x4{v[4 * r], v[4 * r + 1], v[4 * r + 2], v[4 * r + 3]};
        }
      wave_fence();
      if constexpr (E::kRows) {
        constexpr int kHalf = kWide * kMulFrag / 2;
        float x[kHalf];
#pragma unroll
        for (int t = 0; t < kHalf / 4; ++t) {
          const uint32_t line = lane % 32, q = lane / 32 * (kHalf / 4) + t;
          const f32x4 v = *reinterpret_cast<const f32x4*>(piece + line * 64 +
                                                          ((q ^ (line % 16)) * 4));
#pragma unroll
          for (int d = 0; d < 4; ++d) x[4 * t + d] = v[d];
        }
        e.columns(row, x, m0 + i * kMulFrag + lane % 32,
                  n0 + h * (kWide * kMulFrag) + lane / 32 * kHalf, m_all);
        if (h + 1 == kTurns)
          e.finish(row, m0 + i * kMulFrag + lane % 32, n0 / (FN * kMulFrag), m_all);
      }
      if (!e.stores()) {
        wave_fence();
        continue;
      }
#pragma unroll kUnroll
      for (uint32_t r = 0; r < kPass; ++r) {
        if (r == kAhead) fetch(step, kAhead);
        const uint32_t line = r * kLines + lane / kLanes;
        const uint64_t m = to.row_of(i, line, m0 + i * kMulFrag + line), n = column(step);
        const float* p = piece + line * 64;
        const uint32_t turn = line % 16;
        const f32x4 u = *reinterpret_cast<const f32x4*>(p + ((2 * c) ^ turn) * 4);
        const f32x4 v = *reinterpret_cast<const f32x4*>(p + ((2 * c + 1) ^ turn) * 4);
        float y[8] = {u[0], u[1], u[2], u[3], v[0], v[1], v[2], v[3]};
        if constexpr (E::kPairs) {
          const f32x4 u2 = *reinterpret_cast<const f32x4*>(p + ((8 + 2 * c) ^ turn) * 4);
          const f32x4 v2 = *reinterpret_cast<const f32x4*>(p + ((9 + 2 * c) ^ turn) * 4);
          float y2[8] = {u2[0], u2[1], u2[2], u2[3], v2[0], v2[1], v2[2], v2[3]};
          to.template put<T>(split, m, n, m_all, y, y2);
        } else if constexpr (kOld) {
          to.template put<T>(m, n, y, old[r % kAhead]);
        } else {
          to.template put<T>(split, m, n, m_all, y);
        }
      }
      wave_fence();                                           // before the next turn's writes
    }
  }
}

// The same of two waves that have a fragment each, of the same columns of the two stacked
// matrices: `which` is this wave's.  They share `piece`, and store half of its rows each.
// All of a workgroup's waves call it together.
template <typename T, typename E>
__device__ __forceinline__ void pair_store(const f32x16& v, float* piece, const E& e,
                                           uint32_t which, uint64_t m0, uint64_t n0,
                                           uint64_t m_all) {
  const uint32_t lane = threadIdx.x % 64, c = lane % 4;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const uint32_t line = lane % 32, q = which * 8 + r * 2 + lane / 32;
    *reinterpret_cast<f32x4*>(piece + line * 64 + ((q ^ (line % 16)) * 4)) =
        f32x4{v[4 * r], v[4 * r + 1], v[4 * r + 2], v[4 * r + 3]};
  }
  __syncthreads();
  const uint32_t line = which * 16 + lane / 4;
  const float* p = piece + line * 64;
  float x[2][8];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4 u = *reinterpret_cast<const f32x4*>(p + ((j * 8 + 2 * c + h) ^ (line % 16)) * 4);
#pragma unroll
      for (int d = 0; d < 4; ++d) x[j][4 * h + d] = u[d];
    }
  e.template put<T>(0, m0 + line, n0 + c * kChunk, m_all, x[0], x[1]);
}

// Operands of any alignment, WM x WN waves.
template <typename T, bool AF, bool BF, int TM, int TN, int WM, int WN, typename E>
__global__ __launch_bounds__(kMulThreads) void product_kernel(Operand a, Operand b, Extents x,
                                                              uint64_t safe, E epilogue) {
  static_assert(WM * WN == 4, "four waves");
  typedef Side<AF, TM> A;
  constexpr bool kShared = E::kPairs && TN / WN == kMulFrag;   // pair_store
  typedef Side<BF, TN, kShared ? kMulFrag : E::kPairs ? TN / WN / 2 : 0> B;
  constexpr int kFm = TM / WM / kMulFrag, kFn = TN / WN / kMulFrag;
  constexpr int kSub = kMulDepth / kMulStep, kMul = kFm * kFn;
  constexpr uint32_t kCols = TN / WN, kPiece = kMulFrag * 64;
  constexpr uint32_t kTiles = A::kElems + B::kElems;        // 32-bit words of two buffers
  constexpr uint32_t kOut = 4 * kPiece;
  __shared__ __attribute__((aligned(16))) float lds[kTiles > kOut ? kTiles : kOut];
  uint16_t* la = reinterpret_cast<uint16_t*>(lds);
  uint16_t* lb = la + 2 * A::kElems;

  uint64_t m_all = x.m, k_all = x.k;
  bool twice = false;
  if (x.count) {
    uint64_t& of = x.count_k ? k_all : m_all;
    of = counted(x, of, &twice);
  }
  const uint32_t tiles_m = static_cast<uint32_t>((m_all + TM - 1) / TM);
  constexpr int kOutN = E::kPairs ? TN / 2 : TN;            // columns of c a tile
  const uint32_t tiles_n = static_cast<uint32_t>((x.n + kOutN - 1) / kOutN);
  const uint32_t splits = splits_of(x.splits, x.most, x.fill, tiles_m * tiles_n);
  const uint32_t wgs = tiles_m * tiles_n * splits;
  if (blockIdx.x >= wgs) return;
  epilogue.cut(splits, m_all, twice);
  const Spot at = spot_of(blockIdx.x, wgs, tiles_m, tiles_n);
  const uint64_t m0 = static_cast<uint64_t>(at.m) * TM, n0 = static_cast<uint64_t>(at.n) * kOutN;
  const uint64_t per = ((k_all + splits - 1) / splits + kMulDepth - 1) / kMulDepth * kMulDepth;
  const uint64_t k_lo = at.split * per < k_all ? at.split * per : k_all;
  const uint64_t k_hi = k_lo + per < k_all ? k_lo + per : k_all;
  const uint32_t tid = threadIdx.x, wave = tid / 64;
  const uint32_t wm = wave / WN * (TM / WM), wn = wave % WN * kCols;

  A sa;
  B sb;
  sa.begin(a, m0);
  sb.begin(b, n0);
  constexpr int kItems = A::kPass + B::kPass;
  u32x4 reg[kItems];                                        // a's loads, then b's
  auto load_any = [&](uint64_t k) __attribute__((always_inline)) {
#pragma unroll (kItems % 8 ? kItems : 1)
    for (int i = 0; i < kItems; ++i) {
      const u32x4 v = i < A::kPass ? sa.load_checked(k, k_hi, i)
                                   : sb.load_checked(k, k_hi, i - A::kPass);
#pragma unroll
      for (int q = 0; q < kItems; ++q)                      // registers take fixed indexes
        if (q == i) reg[q] = v;
    }
  };
  auto load_one = [&](uint64_t k, int i) __attribute__((always_inline)) {
    reg[i] = i < A::kPass ? sa.load(k, i) : sb.load(k, i - A::kPass);
  };
  auto stage = [&](int buf, int i) __attribute__((always_inline)) {
    if (i < A::kPass) sa.stage(la + buf * A::kElems, i, reg[i]);
    else sb.stage(lb + buf * B::kElems, i - A::kPass, reg[i]);
  };
  const uint64_t whole = k_hi < safe ? k_hi : safe;
  auto load = [&](uint64_t k) __attribute__((always_inline)) {
    if (k + kMulDepth <= whole) {
#pragma unroll
      for (int i = 0; i < kItems; ++i) load_one(k, i);
    } else {
      load_any(k);
    }
  };

  f32x16 acc[kFm][kFn];
#pragma unroll
  for (int i = 0; i < kFm; ++i)
#pragma unroll
    for (int j = 0; j < kFn; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  // Fragments of a step in the order of their use: a0, b0 .. b(kFn-1), a1 .. a(kFm-1).
  u32x4 fa[2][kFm], fb[2][kFn];
  constexpr int kReads = kFm * A::kReads + kFn * B::kReads;
  auto read = [&](int buf, int s, int to, int q) __attribute__((always_inline)) {
    if (q < A::kReads) {
      A::read(la + buf * A::kElems, s, wm, q, fa[to][0]);
    } else if (q < A::kReads + kFn * B::kReads) {
      const int i = (q - A::kReads) / B::kReads;
      B::read(lb + buf * B::kElems, s, wn + i * kMulFrag, (q - A::kReads) % B::kReads, fb[to][i]);
    } else {
      const int w = q - kFn * B::kReads, i = w / A::kReads;
      A::read(la + buf * A::kElems, s, wm + i * kMulFrag, w % A::kReads, fa[to][i]);
    }
  };

  load(k_lo);
#pragma unroll
  for (int i = 0; i < kItems; ++i) stage(0, i);
  load(k_lo + kMulDepth);
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kReads; ++q) read(0, 0, 0, q);
  uint32_t buf = 0;
  uint64_t k0 = k_lo;
  static_assert(kSub % 2 == 0, "the operands' registers take turns");
  // A turn: all of tile k0's steps; tile k0 + 64 from registers to the other buffer
  // (last read before the barrier of the turn before) over all steps but the last;
  // then the barrier, behind which the next tile's first operands are read while the
  // last step runs.  Other work goes between the matrix instructions in equal parts,
  // and the compiler keeps it there.
  constexpr int kSlots = (kSub - 1) * kMul;
  constexpr int kItemsEach = (kItems + kSlots - 1) / kSlots;
  constexpr int kReadsEach = (kReads + kMul - 1) / kMul;
  auto turn = [&](auto refill) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < kSub; ++s) {
      const bool last = s + 1 == kSub;
      if (last) __syncthreads();
#pragma unroll
      for (int w = 0; w < kMul; ++w) {
        const int i = w / kFn, j = w % kFn;
        acc[i][j] = mul<T>(fb[s & 1][j], fa[s & 1][i], acc[i][j]);
#pragma unroll
        for (int d = 0; d < kReadsEach; ++d) {
          const int q = w * kReads / kMul + d;
          if (q < (w + 1) * kReads / kMul)
            read(last ? buf ^ 1 : buf, last ? 0 : s + 1, (s + 1) & 1, q);
        }
#pragma unroll
        for (int d = 0; d < kItemsEach; ++d) {
          const int slot = s * kMul + w, q = slot * kItems / kSlots + d;
          if (last || q >= (slot + 1) * kItems / kSlots) continue;
          stage(buf ^ 1, q);
          refill(q);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    buf ^= 1;
  };
#pragma unroll 1
  for (; k0 + 3 * kMulDepth <= whole; k0 += kMulDepth)
    turn([&](int i) { load_one(k0 + 2 * kMulDepth, i); });
#pragma unroll 1
  for (; k0 < k_hi; k0 += kMulDepth) {
    turn([](int) {});
    load_any(k0 + 2 * kMulDepth);                           // zeros past the end
  }
  __syncthreads();

  if constexpr (kShared)
    pair_store<T>(acc[0][0], lds + wave / 2 * kPiece, epilogue, wave % 2, m0,
                  n0 + wave / 2 * kMulFrag, m_all);
  else
    wave_store<T, false>(acc, lds + wave * kPiece, epilogue, epilogue, at.split, m0 + wm,
                         n0 + (E::kPairs ? wn / 2 : wn), m_all);
}

// ------------------------------------------------------------ whole chunks

// The same product where every 16-byte chunk of both operands is whole and aligned
// (ring_takes): 256 x 256 tiles and stages of 64 k that go from memory straight to
// shared memory, one under way while the other is worked on, and workgroups that stay
// for several tiles, so that the next tile's first stage is read while this one's sums
// are stored.  Without registers between, a stage's loads are issued with little else,
// right behind the barrier that frees its place.
//
// Loads past an operand's end are out of their descriptor's range: they give 0 and
// touch no memory.  Places in shared memory are those of Side.  A wave's load is 1 KiB
// of a stage: eight rows of 64 k (k fast) or two of 256 columns (k slow); in either case
// whole 128-byte lines, which the caches hand out twice as fast as halves (stages of 32
// k, four of them, took 1266 where this takes 1391 TFLOP/s with k fast in both operands,
// 4096 x 4096 over 65536).
constexpr int kRingTile = 256;
constexpr uint32_t kRingSide = kRingTile * kMulDepth * 2;    // bytes of an operand's stage
constexpr uint32_t kRingStage = 2 * kRingSide;
constexpr uint32_t kRingOut = 8192;                          // of a wave: 32 rows of 64 sums
constexpr uint32_t kRingWgs = 256;                           // one a compute unit
constexpr int kSlimCols = 128, kSlimStages = 4;
constexpr uint32_t kSlimRows = kMulFrag * kMulDepth * 2;     // bytes of a's stage
constexpr uint32_t kSlimStage = kSlimRows + kSlimCols * kMulDepth * 2;

// One operand's loads, TILE and PAIR as Side's.
template <bool FAST, int TILE, int PAIR = 0>
struct RingSide {
  static constexpr int kLoads = TILE / 32;                   // of a thread, a stage
  static constexpr int kReads = FAST ? 1 : 2;                // shared loads a fragment
  static constexpr uint32_t kNone = 0x80000000u, kAll = 0x7FFFFFF0u;
  static constexpr uint32_t kLanes = FAST ? kMulDepth / kChunk : TILE / kChunk;
  static constexpr uint32_t kRows = 64 / kLanes;             // of memory, a wave's load
  u32x4 srd;                  // the descriptor of the stage to load next
  uint64_t stride;            // bytes
  uint32_t off[kLoads];   // of this lane's chunk in each of its loads, or kNone

  // The chunk of a row that this lane loads, by the place it has in shared memory.
  static __device__ __forceinline__ uint32_t chunk_of(uint32_t wave) {
    const uint32_t lane = threadIdx.x % 64;
    if constexpr (FAST) return lane % 8 ^ (wave % 2 * 4 + lane / 16);
    const uint32_t row = wave * kRows + lane / kLanes;
    return ((lane % kLanes / 4) ^ (row & 3)) * 4 + lane % 4;
  }

  __device__ __forceinline__ void go_to(uint64_t base) {
    srd[0] = static_cast<uint32_t>(base);
    srd[1] = static_cast<uint32_t>(base >> 32);              // addresses have 48 bits
  }

  __device__ __forceinline__ void begin(const Operand& o, uint64_t first, uint64_t k,
                                        uint32_t wave) {
    stride = o.stride * 2;
    srd[2] = kAll;
    srd[3] = 0x00027000u;
    const uint64_t p = reinterpret_cast<uint64_t>(o.p);
    go_to(FAST ? p + first * stride + k * 2 : p + k * stride);
    const uint32_t chunk = chunk_of(wave);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint32_t r = (i * 4 + wave) * kRows + threadIdx.x % 64 / kLanes;
      if constexpr (!FAST) {
        const uint64_t c = first + chunk * kChunk;
        off[i] = c < o.extent ? static_cast<uint32_t>(r * stride + c * 2) : kNone;
      } else if constexpr (PAIR != 0) {
        const uint32_t c = r / (2 * PAIR) * PAIR + r % PAIR;
        const uint64_t row = c + (r / PAIR % 2 ? o.extent : 0);
        off[i] = first + c < o.extent ? static_cast<uint32_t>(row * stride) + chunk * 16 : kNone;
      } else {
        off[i] = first + r < o.extent ? static_cast<uint32_t>(r * stride) + chunk * 16 : kNone;
      }
    }
  }

  // The stage to load next has `left` < 64 k: the rest is out of range.
  __device__ __forceinline__ void cut(uint32_t left, uint32_t wave) {
    if constexpr (FAST) {
      const bool in = chunk_of(wave) * kChunk < left;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) off[i] = in ? off[i] : kNone;
    } else {
      srd[2] = static_cast<uint32_t>(left * stride);
    }
  }

  // One load, to shared memory from `to` + TO on (a scalar).  It writes no register; the
  // loop's own waits are what orders it.
  template <int TO>
  __device__ __forceinline__ void load(uint32_t to, uint32_t from) const {
    asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(to), "v"(from), "s"(srd), "i"(TO)
                 : "memory", "scc", "m0");
  }

  // The descriptor in scalar registers, whatever the compiler made of it.
  __device__ __forceinline__ void settle() {
#pragma unroll
    for (int i = 0; i < 4; ++i) srd[i] = __builtin_amdgcn_readfirstlane(srd[i]);
  }

  __device__ __forceinline__ void next() {
    go_to((static_cast<uint64_t>(srd[1]) << 32 | srd[0]) +
          (FAST ? kMulDepth * 2 : kMulDepth * stride));
  }

  // This lane's place, in bytes from an operand's stage on, of part q of the fragment at
  // rows [at, at + 32) and 16 k from step * 16 on.
  static __device__ __forceinline__ uint32_t place(int step, uint32_t at, int q) {
    const uint32_t lane = threadIdx.x % 64;
    if constexpr (FAST) {
      // chunks 2 step and 2 step + 1, before their permutation
      const uint32_t r = at + lane % 32;
      return ((r * kMulDepth + ((lane / 32) ^ (r / 2 % 8)) * kChunk) * 2) ^ (step * 32);
    } else {
      const uint32_t r = step * kMulStep + (lane / 32) * 8 + (lane % 16) / 4 + q * 4;
      const uint32_t c = at + (lane / 16 % 2) * 16 + lane % 4 * 4;
      return (r * TILE + ((((c >> 5) ^ (r & 3)) << 5) | (c & 31))) * 2;
    }
  }

  static __device__ __forceinline__ void read(uint32_t at, int q, u32x4& to) {
    typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    if constexpr (FAST) {
      to = *reinterpret_cast<lds_u32x4*>(at);
    } else {
      const u32x2 v = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s16x4*>(at)));
      to[2 * q] = v[0];
      to[2 * q + 1] = v[1];
    }
  }
};

// Load `which` of a stage: a's, then b's.
template <int I, typename A, typename B>
__device__ __forceinline__ void ring_load(const A& a, const B& b, uint32_t to, int which) {
  if (which == I) {
    if constexpr (I < A::kLoads)
      a.template load<I * 4096>(to, a.off[I]);
    else
      b.template load<I * 4096>(to, b.off[I - A::kLoads]);
  } else if constexpr (I + 1 < A::kLoads + B::kLoads) {
    ring_load<I + 1>(a, b, to, which);
  }
}

template <typename T, bool AF, bool BF, typename E>
__global__ __launch_bounds__(kMulThreads, 1) void ring_kernel(Operand a, Operand b, Extents x,
                                                              E epilogue) {
  typedef RingSide<AF, kRingTile> A;
  typedef RingSide<BF, kRingTile, E::kPairs ? 64 : 0> B;
  constexpr int kF = 4, kMul = kF * kF, kReads = kF * (A::kReads + B::kReads);
  constexpr int kSteps = kMulDepth / kMulStep;
  static_assert(kRingSide == A::kLoads * 4096, "a workgroup's load is 4 KiB");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kRingStage + 4 * kRingOut];
  const uint32_t lds0 = static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds));

  const float by = epilogue.load_factor();
  uint64_t m_all = x.m, k_all = x.k;
  bool twice = false;
  if (x.count) {
    uint64_t& of = x.count_k ? k_all : m_all;
    of = counted(x, of, &twice);
  }
  constexpr int kOutN = E::kPairs ? kRingTile / 2 : kRingTile;
  const uint32_t tiles_m = static_cast<uint32_t>((m_all + kRingTile - 1) / kRingTile);
  const uint32_t tiles_n = static_cast<uint32_t>((x.n + kOutN - 1) / kOutN);
  const uint32_t splits = splits_of(x.splits, x.most, x.fill, tiles_m * tiles_n);
  const uint32_t wgs = tiles_m * tiles_n * splits;
  if (blockIdx.x >= wgs) return;
  epilogue.cut(splits, m_all, twice);
  const uint64_t per = ((k_all + splits - 1) / splits + kMulDepth - 1) / kMulDepth * kMulDepth;
  const uint32_t lane = threadIdx.x % 64;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const uint32_t wm = wave / 2 * 128, wn = wave % 2 * 128;

  // The loads' side: which tile it is at, the k left of it, and where a stage goes.
  A sa;
  B sb;
  uint32_t id = blockIdx.x;
  int32_t left = 0, rest = 0;      // k is at most 2^25
  uint64_t load_m = 0, load_n = 0, load_k = 0;
  const uint32_t fill0 = lds0 + wave * 1024;
  uint32_t fill = fill0;
  const auto enter = [&]() __attribute__((always_inline)) {
    const Spot at = spot_of(id, wgs, tiles_m, tiles_n);
    const uint64_t lo = at.split * per < k_all ? at.split * per : k_all;
    const uint64_t hi = lo + per < k_all ? lo + per : k_all;
    // Neighbouring tiles begin up to seven stages further on and end with what they
    // left out: rows whose stride is a power of two begin in the same channels of the
    // caches, which all tiles would ask together (4096 x 131072 over 4096: 1264 -> 1335
    // TFLOP/s with k fast, 1279 -> 1287 with k slow).
    const uint32_t stages = static_cast<uint32_t>((hi - lo + kMulDepth - 1) / kMulDepth);
    rest = stages ? static_cast<int32_t>((at.m + at.n) % 8 % stages) * kMulDepth : 0;
    left = static_cast<int32_t>(hi - lo) - rest;
    load_m = static_cast<uint64_t>(at.m) * kRingTile;
    load_n = static_cast<uint64_t>(at.n) * kOutN;
    load_k = lo;
    sa.begin(a, load_m, lo + rest, wave);
    sb.begin(b, load_n, lo + rest, wave);
  };
  // The stage to load next is the range's last, or past it: on to the part that was left
  // out, to the next tile, or to nothing.
  const auto turn = [&]() __attribute__((always_inline)) {
    while (left <= 0 && id < wgs) {
      if (rest > 0) {
        left = rest;
        rest = 0;
        sa.begin(a, load_m, load_k, wave);
        sb.begin(b, load_n, load_k, wave);
      } else {
        id += gridDim.x;
        if (id < wgs) enter();
      }
    }
    if (left < kMulDepth) {
      const uint32_t some = left > 0 ? static_cast<uint32_t>(left) : 0;
      sa.cut(some, wave);
      sb.cut(some, wave);
    }
  };
  const auto stage_done = [&]() __attribute__((always_inline)) {
    fill = fill == fill0 ? fill0 + kRingStage : fill0;
    sa.next();
    sb.next();
    left -= kMulDepth;
    if (left < kMulDepth) turn();
  };

  // Fragments of a step in the order of their use: a0, b0 .. b3, a1 .. a3.
  u32x4 fa[2][kF], fb[2][kF];
  f32x16 acc[kF][kF];
  uint32_t ring = lds0;     // the stage that is worked on
  const uint32_t pa = A::place(0, wm, 0), pb = B::place(0, wn, 0);
  const auto read = [&](uint32_t stage, int s, int to, int q) __attribute__((always_inline)) {
    constexpr uint32_t kNext = kMulFrag * kMulDepth * 2;   // bytes to a next fragment, k fast
    const bool of_b = q >= A::kReads && q < A::kReads + kF * B::kReads;
    if (of_b) {
      const int i = (q - A::kReads) / B::kReads, h = (q - A::kReads) % B::kReads;
      const uint32_t at = BF ? (pb ^ s * 32) + i * kNext : B::place(s, wn + i * kMulFrag, h);
      B::read(stage + kRingSide + at, h, fb[to][i]);
    } else {
      const int w = q < A::kReads ? q : q - kF * B::kReads, i = w / A::kReads, h = w % A::kReads;
      const uint32_t at = AF ? (pa ^ s * 32) + i * kNext : A::place(s, wm + i * kMulFrag, h);
      A::read(stage + at, h, fa[to][i]);
    }
  };

  enter();
  turn();
  // The first kFirst loads of a stage go between the matrix instructions of the step
  // behind the barrier, the others evenly into the two steps after it, so that the last
  // has a step left to arrive (8, 12 and 16 first: 1302, 1391 and 1318 TFLOP/s).
  constexpr int kLoads = A::kLoads + B::kLoads, kFirst = 12;
  constexpr int kRest = (kLoads - kFirst + kSteps - 2) / (kSteps - 1);
#pragma unroll
  for (int q = 0; q < kLoads; ++q) ring_load<0>(sa, sb, fill, q);
  stage_done();
#pragma unroll
  for (int q = 0; q < kFirst; ++q) ring_load<0>(sa, sb, fill, q);
  asm volatile("s_waitcnt vmcnt(%0)" ::"i"(kFirst) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");

#pragma unroll 1
  for (uint32_t tile = blockIdx.x; tile < wgs; tile += gridDim.x) {
    // again for a next tile, whose first stage is there: registers that the stores need
#pragma unroll
    for (int q = 0; q < kReads; ++q) read(ring, 0, 0, q);
    const Spot at = spot_of(tile, wgs, tiles_m, tiles_n);
    const uint64_t lo = at.split * per < k_all ? at.split * per : k_all;
    const uint64_t hi = lo + per < k_all ? lo + per : k_all;
    const uint32_t stages = static_cast<uint32_t>((hi - lo + kMulDepth - 1) / kMulDepth);
#pragma unroll
    for (int i = 0; i < kF; ++i)
#pragma unroll
      for (int j = 0; j < kF; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    constexpr int kOver = kMul - 3;       // a step's reads end three instructions early
#pragma unroll 1
    for (uint32_t s = 0; s < stages; ++s) {
      const uint32_t then = ring == lds0 ? lds0 + kRingStage : lds0;
      // step p beside the reads of step p + 1; the last one's are the next stage's
#pragma unroll
      for (int p = 0; p < kSteps; ++p) {
        const bool last = p + 1 == kSteps;
        const int l0 = last ? 0 : kFirst + p * kRest;
        const int l1 = last ? kFirst : l0 + kRest < kLoads ? l0 + kRest : kLoads;
        if (last) {
          stage_done();
          // this wave has read all of this stage, and its loads of the next one are
          // there: so have and are, behind the barrier, all waves'
          asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
          __builtin_amdgcn_s_barrier();
          asm volatile("" ::: "memory");
        }
#pragma unroll
        for (int w = 0; w < kMul; ++w) {
          acc[w / kF][w % kF] = mul<T>(fb[p & 1][w % kF], fa[p & 1][w / kF], acc[w / kF][w % kF]);
#pragma unroll
          for (int d = 0; d < (kReads + kOver - 1) / kOver; ++d) {
            const int q = w * kReads / kOver + d;
            if (q < (w + 1) * kReads / kOver && q < kReads)
              read(last ? then : ring, last ? 0 : p + 1, (p + 1) & 1, q);
          }
          const int n = l1 - l0;
          if (n > 0 && (w + 1) * n / kMul > w * n / kMul)
            ring_load<0>(sa, sb, fill, l0 + w * n / kMul);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      ring = then;
    }

    const uint64_t m0 = static_cast<uint64_t>(at.m) * kRingTile + wm;
    const uint64_t n0 = static_cast<uint64_t>(at.n) * kOutN + (E::kPairs ? wn / 2 : wn);
    float* piece = reinterpret_cast<float*>(lds + 2 * kRingStage + wave * kRingOut);
    const bool whole = static_cast<uint64_t>(at.m + 1) * kRingTile <= m_all &&
                       static_cast<uint64_t>(at.n + 1) * kOutN <= x.n;
    if (whole && epilogue.simple()) {
      if (E::kAdds && epilogue.adds())
        wave_store<T, true>(acc, piece, epilogue,
                            epilogue.template now<E::kAdds>(at.split, m0, by), at.split, m0, n0,
                            m_all);
      else
        wave_store<T, true>(acc, piece, epilogue, epilogue.template now<false>(at.split, m0, by),
                            at.split, m0, n0, m_all);
    } else
      wave_store<T, false>(acc, piece, epilogue, epilogue, at.split, m0, n0, m_all);
    // vmcnt(0), seen by the compiler: it would wait for the epilogue's loads in every
    // turn of the next tile otherwise, and with them for the stage under way
    if (!(whole && epilogue.simple())) __builtin_amdgcn_s_waitcnt(0x0F70);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // nothing lands in shared memory later
}

// 32 rows of c, whole chunks: bound by how fast b comes from memory, so what counts is how
// much of it is under way, and that its rows are not all asked from the same channels.
// Tiles of 32 x 128, stages of 64 k (20 KiB), all but one of them under way while that one
// is worked on; two workgroups a unit.  1 or 32 x 32768 over 4096, b in memory: 46 us, 5.8
// TB/s, where product_kernel takes 61 and reading b in order 47; six to eight stages, one
// workgroup a unit, are no faster.  A counted x is rows (k is not slow in a).
template <typename T, bool BF, typename E>
__global__ __launch_bounds__(kMulThreads) void slim_kernel(Operand a, Operand b, Extents x,
                                                           E epilogue) {
  typedef RingSide<true, kMulFrag> A;
  typedef RingSide<BF, kSlimCols, E::kPairs ? kMulFrag : 0> B;
  constexpr int kSteps = kMulDepth / kMulStep, kLoads = A::kLoads + B::kLoads;
  constexpr uint32_t kPiece = kMulFrag * 64;
  constexpr uint32_t kLds = kSlimStages * kSlimStage;
  static_assert(kLds >= 4 * kPiece * 4, "the epilogue's pieces");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];
  const uint32_t lds0 = static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds));

  bool twice = false;
  const uint64_t m_all = x.count ? counted(x, x.m, &twice) : x.m;
  constexpr int kOutN = E::kPairs ? kSlimCols / 2 : kSlimCols;
  const uint32_t tiles_m = static_cast<uint32_t>((m_all + kMulFrag - 1) / kMulFrag);
  const uint32_t tiles_n = static_cast<uint32_t>((x.n + kOutN - 1) / kOutN);
  const uint32_t splits = splits_of(x.splits, x.most, x.fill, tiles_m * tiles_n);
  const uint32_t wgs = tiles_m * tiles_n * splits;
  if (blockIdx.x >= wgs) return;
  epilogue.cut(splits, m_all, twice);
  const Spot at = spot_of(blockIdx.x, wgs, tiles_m, tiles_n);
  const uint64_t m0 = static_cast<uint64_t>(at.m) * kMulFrag;
  const uint64_t n0 = static_cast<uint64_t>(at.n) * kOutN;
  const uint64_t per = ((x.k + splits - 1) / splits + kMulDepth - 1) / kMulDepth * kMulDepth;
  const uint64_t lo = at.split * per < x.k ? at.split * per : x.k;
  const uint64_t hi = lo + per < x.k ? lo + per : x.k;
  const uint32_t stages = static_cast<uint32_t>((hi - lo + kMulDepth - 1) / kMulDepth);
  const uint32_t tail = static_cast<uint32_t>(hi - lo) - (stages - 1) * kMulDepth;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);

  // Neighbouring tiles begin at different stages, as in the ring.
  A sa;
  B sb;
  uint32_t turn = stages ? at.n % stages : 0, loaded = 0, fill = lds0 + wave * 1024;
  const auto begin = [&]() __attribute__((always_inline)) {
    sa.begin(a, m0, lo + turn * static_cast<uint64_t>(kMulDepth), wave);
    sb.begin(b, n0, lo + turn * static_cast<uint64_t>(kMulDepth), wave);
  };
  const auto load = [&]() __attribute__((always_inline)) {
    const uint32_t some = loaded >= stages ? 0 : turn + 1 == stages ? tail : kMulDepth;
    if (some < kMulDepth) {
      sa.cut(some, wave);
      sb.cut(some, wave);
    }
    sa.settle();
    sb.settle();
#pragma unroll
    for (int q = 0; q < kLoads; ++q) ring_load<0>(sa, sb, fill, q);
    fill = fill + kSlimStage < lds0 + kLds ? fill + kSlimStage : lds0 + wave * 1024;
    sa.next();
    sb.next();
    ++loaded;
    if (++turn >= stages) {
      turn = 0;
      begin();
    }
  };
  begin();
#pragma unroll 1
  for (int s = 0; s + 1 < kSlimStages; ++s) load();

  f32x16 acc[1][1];
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[0][0][r] = 0.f;
  uint32_t stage = lds0;
#pragma unroll 1
  for (uint32_t s = 0; s < stages; ++s) {
    // this wave's loads of the stage are there, and it has read the one before: so are
    // and have, behind the barrier, all waves'
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"i"(kLoads * (kSlimStages - 2)) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    load();
#pragma unroll
    for (int p = 0; p < kSteps; ++p) {
      u32x4 fa, fb;
      A::read(stage + A::place(p, 0, 0), 0, fa);
#pragma unroll
      for (int h = 0; h < B::kReads; ++h)
        B::read(stage + kSlimRows + B::place(p, wave * kMulFrag, h), h, fb);
      acc[0][0] = mul<T>(fb, fa, acc[0][0]);
    }
    stage = stage + kSlimStage < lds0 + kLds ? stage + kSlimStage : lds0;
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");   // nothing lands later
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");

  float* pieces = reinterpret_cast<float*>(lds);
  if constexpr (E::kPairs)
    pair_store<T>(acc[0][0], pieces + wave / 2 * kPiece, epilogue, wave % 2, m0,
                  n0 + wave / 2 * kMulFrag, m_all);
  else
    wave_store<T, false>(acc, pieces + wave * kPiece, epilogue, epilogue, at.split, m0,
                         n0 + wave * kMulFrag, m_all);
}

// Whether the ring takes an operand: whole, aligned chunks, and a tile's (k fast) or a
// stage's (k slow) offsets within 31 bits.
inline bool ring_takes(const Operand& o, bool fast, uint64_t k, bool pairs = false) {
  constexpr uint64_t kFar = 1ull << 30;
  if (reinterpret_cast<uintptr_t>(o.p) % 16 || o.stride % kChunk) return false;
  if (o.stride >= kFar / 512) return false;
  if (!o.padded && (fast ? k : o.extent) % kChunk) return false;
  return fast ? ((pairs ? o.extent : 0) + 256) * o.stride < kFar
              : o.stride * kMulDepth + o.extent < kFar;
}

// Where sums go: partial sums of splits (fp32, `lead` apart, joined afterwards by
// join_kernel), running sums over several products, or the result itself, scaled and
// rounded once.
struct Sink {
  static constexpr bool kPairs = false, kRows = false, kJoins = true, kAdds = true;
  void* out;
  uint64_t stride;
  int dtype, accumulate;   // kF16, kBf16 or kF32
  uint64_t cols;
  const uint32_t* rows;    // the result's row of row m, or nullptr: m
  const float* factor;     // in device memory, or nullptr
  float* partial;          // [splits][rows][lead], or nullptr: one split
  uint64_t split_size;     // elements: rows * lead
  float* sums;             // [rows][lead] running sums, or nullptr
  int add, last;           // add what `sums` holds; the result is final
  uint64_t lead;           // cols, rounded up to a chunk
  uint32_t twice;          // 1: rows of c may stand twice (Extents): row m and the row half
                           // of them further on are added up

  template <typename T>
  __device__ __forceinline__ void finish(uint64_t m, uint64_t n, float (&x)[8]) const {
    if (sums) {
      f32x4* s = reinterpret_cast<f32x4*>(sums + m * lead + n);
      if (add) {
        const f32x4 u = s[0], v = s[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = u[i] + x[i];
          x[4 + i] = v[i] + x[4 + i];
        }
      }
      if (!last) {
        s[0] = f32x4{x[0], x[1], x[2], x[3]};
        s[1] = f32x4{x[4], x[5], x[6], x[7]};
        return;
      }
    }
    if (factor) {
      const float f = *factor;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= f;
    }
    const uint64_t row = (rows ? rows[m] : m) * stride;
    if (dtype == kF32) {
      float* o = static_cast<float*>(out) + row + n;
      if (n + kChunk <= cols) {
        f32x4_at4* w = reinterpret_cast<f32x4_at4*>(o);
        f32x4 u = {x[0], x[1], x[2], x[3]}, v = {x[4], x[5], x[6], x[7]};
        if (accumulate) {
          u += w[0];
          v += w[1];
        }
        w[0] = u;
        w[1] = v;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (n + i < cols) o[i] = accumulate ? o[i] + x[i] : x[i];
      }
      return;
    }
    uint16_t* o = static_cast<uint16_t*>(out) + row;
    if (accumulate) {
      float old[8];
      unpack8<T>(load8(o, n, cols), old);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] += old[i];
    }
    store8<false>(o, n, cols, pack8<T>(x));
  }

  static constexpr bool kOld = false;
  struct Row {};
  struct Old {};

  __device__ __forceinline__ void cut(uint32_t splits, uint64_t m_all, bool stand_twice) {
    twice = twice && stand_twice;
    if (splits == 1 && !twice) partial = nullptr;
    split_size = m_all * lead;
  }

  __device__ __forceinline__ bool stores() const { return true; }
  __device__ __forceinline__ uint64_t row_of(int, uint32_t, uint64_t m) const { return m; }

  // Whole tiles: all but the last running sums on top of an old result.
  __device__ __forceinline__ bool simple() const { return !(sums && add && last && accumulate); }

  // What is stored, and what is added to it: old running sums before the factor, or an old
  // result after it.
  template <bool OLD>
  struct Now {
    static constexpr bool kOld = OLD;
    struct Old {
      u32x4 a, b;
    };
    uint8_t* out;
    uint64_t stride;        // bytes, as all here
    const uint8_t* old;
    uint64_t old_stride;
    bool wide, old_wide, old_first;   // fp32
    float factor;
    bool mapped;
    uint32_t rows[4];       // mapped: the rows of lane % 32 in each 32 of the wave's

    __device__ __forceinline__ uint64_t row_of(int i, uint32_t line, uint64_t m) const {
      if (!mapped) return m;
      return static_cast<uint32_t>(__builtin_amdgcn_ds_bpermute(static_cast<int>(line * 4),
                                                                static_cast<int>(rows[i])));
    }

    __device__ __forceinline__ Old fetch(uint64_t m, uint64_t n) const {
      const uint8_t* p = old + m * old_stride + n * (old_wide ? 4 : 2);
      Old o;
      o.a = *reinterpret_cast<const u32x4_at2*>(p);
      o.b = *reinterpret_cast<const u32x4_at2*>(p + (old_wide ? 16 : 0));
      return o;
    }

    template <typename T>
    __device__ __forceinline__ void put(uint64_t m, uint64_t n, float (&x)[8], Old o) const {
      float y[8];
      forget(o.b);            // arrived in any case: no wait is left for the next tile
      if (old_wide) {
        const f32x4 u = __builtin_bit_cast(f32x4, o.a), v = __builtin_bit_cast(f32x4, o.b);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[i] = u[i];
          y[4 + i] = v[i];
        }
      } else {
        unpack8<T>(o.a, y);
      }
      if (old_first) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (y[i] + x[i]) * factor;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * factor + y[i];
      }
      store<T>(m, n, x);
    }

    template <typename T>
    __device__ __forceinline__ void put(uint32_t, uint64_t m, uint64_t n, uint64_t,
                                        float (&x)[8]) const {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= factor;
      store<T>(m, n, x);
    }

    template <typename T>
    __device__ __forceinline__ void store(uint64_t m, uint64_t n, const float (&x)[8]) const {
      if (wide) {
        f32x4_at4* w = reinterpret_cast<f32x4_at4*>(out + m * stride + n * 4);
        w[0] = f32x4{x[0], x[1], x[2], x[3]};
        w[1] = f32x4{x[4], x[5], x[6], x[7]};
      } else {
        *reinterpret_cast<u32x4_at2*>(out + m * stride + n * 2) = pack8<T>(x);
      }
    }
  };

  // In a scalar register, so that no load is under way when the products begin.
  __device__ __forceinline__ float load_factor() const {
    return factor ? __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(
                                                  __builtin_bit_cast(int, *factor)))
                  : 1.0f;
  }

  __device__ __forceinline__ bool adds() const {
    return !partial && (sums ? add != 0 : accumulate != 0);
  }

  template <bool OLD>
  __device__ __forceinline__ Now<OLD> now(uint32_t split, uint64_t m0, float by) const {
    Now<OLD> n = {};
    if (partial || (sums && !last)) {
      n.out = reinterpret_cast<uint8_t*>(partial ? partial + split * split_size : sums);
      n.stride = lead * 4;
      n.wide = true;
      n.factor = 1.0f;
    } else {
      n.out = static_cast<uint8_t*>(out);
      n.wide = dtype == kF32;
      n.stride = stride * (n.wide ? 4 : 2);
      n.factor = by;
      n.mapped = rows != nullptr;
    }
    if (OLD && sums) {
      n.old = reinterpret_cast<const uint8_t*>(sums);
      n.old_stride = lead * 4;
      n.old_wide = n.old_first = true;
    } else if (OLD) {
      n.old = n.out;
      n.old_stride = n.stride;
      n.old_wide = n.wide;
    }
    if (n.mapped) {
#pragma unroll
      for (int i = 0; i < 4; ++i) n.rows[i] = rows[m0 + i * 32 + threadIdx.x % 32];
#pragma unroll
      for (int i = 0; i < 4; ++i) forget(n.rows[i]);
    }
    return n;
  }

  template <typename T>
  __device__ __forceinline__ void put(uint32_t split, uint64_t m, uint64_t n, uint64_t m_all,
                                      float (&x)[8]) const {
    if (m >= m_all || n >= cols) return;
    if (partial) {
      f32x4* p = reinterpret_cast<f32x4*>(partial + split * split_size + m * lead + n);
      p[0] = f32x4{x[0], x[1], x[2], x[3]};
      p[1] = f32x4{x[4], x[5], x[6], x[7]};
      return;
    }
    finish<T>(m, n, x);
  }
};

// Adds the splits' partial sums, and those of rows that stand twice, in their order, eight
// neighbouring columns a thread.
template <typename T>
__global__ __launch_bounds__(kMulThreads) void join_kernel(Sink s, Extents x, uint32_t tile_m,
                                                           uint32_t tiles_n) {
  bool twice = false;
  const uint64_t m_all = x.count && !x.count_k ? counted(x, x.m, &twice) : x.m;
  const uint32_t tiles = static_cast<uint32_t>((m_all + tile_m - 1) / tile_m) * tiles_n;
  const uint32_t splits = splits_of(x.splits, x.most, x.fill, tiles);
  s.cut(splits, m_all, twice);
  if (splits == 1 && !s.twice) return;
  const uint64_t rows = m_all >> s.twice;
  const uint64_t per_row = s.lead / kChunk;
  const uint64_t id = static_cast<uint64_t>(blockIdx.x) * kMulThreads + threadIdx.x;
  const uint64_t m = id / per_row, n = id % per_row * kChunk;
  if (m >= rows) return;
  f32x4 u = {0.f, 0.f, 0.f, 0.f}, v = u;
  const float* from = s.partial + m * s.lead + n;
  // sixteen sums' loads under way together, however many there are
  constexpr uint32_t kAhead = 16;
  const uint32_t all = splits << s.twice;
#pragma unroll 1
  for (uint32_t i0 = 0; i0 < all; i0 += kAhead) {
    f32x4 a[kAhead], b[kAhead];
#pragma unroll
    for (uint32_t j = 0; j < kAhead; ++j) {
      const uint32_t i = i0 + j;
      a[j] = b[j] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (i >= all) continue;
      const float* p = from + (i >> s.twice) * s.split_size + (i & s.twice) * rows * s.lead;
      a[j] = *reinterpret_cast<const f32x4*>(p);
      b[j] = *reinterpret_cast<const f32x4*>(p + 4);
    }
#pragma unroll
    for (uint32_t j = 0; j < kAhead; ++j) {
      u += a[j];
      v += b[j];
    }
  }
  float sum[8] = {u[0], u[1], u[2], u[3], v[0], v[1], v[2], v[3]};
  s.finish<T>(m, n, sum);
}

// How a product is cut: the tile of c (256 x 256, 128 x 128, or 32 rows x 128), the splits
// of k, and their most where rows are counted on the device.
struct MulPlan {
  int tile;
  uint32_t splits, most, fill;
  uint64_t tiles, tiles_n;
};

// What may be: splits at all; tiles of 32 rows (k fast in a); rows that are counted on
// the device; operands of whole chunks (ring_takes).
struct MulWays {
  bool split, few_rows, counted, whole;
};

// The same cut over m rows of c and n columns of b.
inline MulPlan plan_of(MulPlan p, uint64_t m, uint64_t n) {
  const uint64_t tn = p.tile == 256 ? 256 : 128;
  p.tiles_n = (n + tn - 1) / tn;
  p.tiles = (m + p.tile - 1) / p.tile * p.tiles_n;
  return p;
}

// The cut with the least estimated time.  Microseconds of a round of workgroups that the
// chip holds together, as measured on MI355X: a fixed part, and one for each k, which is
// less where fewer workgroups share a compute unit.  256 x 256: 7 + 0.026 k (14 + 0.0285 k
// where the operands are not whole chunks); 128 x 128, two a unit: 6.7 + 0.0141 k, one:
// 0.0075 k; 32 x 128, four a unit (two of whole chunks): 4.3 + 0.0123 k, two: 0.0075 k, one: 0.0056 k.  A join
// costs a launch, and its partial sums' way out and back.  (4096 x 4096 over 1024, k slow:
// 43, 55 us in 256, 128; 200 x 4096 over 1024, k fast: 35, 18, 11 us in 256, 128, 32.)
inline MulPlan plan_product(uint64_t m, uint64_t n, uint64_t k, const MulWays& may) {
  constexpr uint64_t kUnits = 256;
  MulPlan best = {};
  double least = 0;
  for (const int tile : {256, 128, 32}) {
    if (tile == 32 && !may.few_rows) continue;
    MulPlan p = {tile, 1, 1, 0, 0, 0};
    p = plan_of(p, m, n);
    const uint64_t at_once = tile == 256 ? kUnits
                             : tile == 128 || may.whole ? 2 * kUnits : 4 * kUnits;
    p.fill = static_cast<uint32_t>(at_once);
    for (const uint32_t s : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
      if (s > 1 && (!may.split || k < 256 * s)) break;
      p.splits = s;
      p.most = s;
      const uint64_t per = ((k + s - 1) / s + 63) / 64 * 64, wgs = p.tiles * s;
      const double rounds = static_cast<double>((wgs + at_once - 1) / at_once);
      const double each = tile == 256 ? (may.whole ? 0.026 : 0.0285)
                          : tile == 128 ? (wgs > kUnits ? 0.0141 : 0.0075)
                                 : (wgs > 2 * kUnits ? 0.0123 : wgs > kUnits ? 0.0075 : 0.0056);
      const double fix = tile == 256 ? (may.whole ? 7.0 : 14.0) : tile == 128 ? 6.7 : 4.3;
      double us = rounds * (fix + each * static_cast<double>(per));
      if (s > 1) us += 4.0 + s * static_cast<double>(m) * static_cast<double>(n) * 8 / 5e6;
      if (best.tiles == 0 || us < least) {
        least = us;
        best = p;
      }
    }
  }
  if (may.counted && may.split) {
    const uint64_t most = k / 256 < 32 ? k / 256 : 32;
    if (most > best.most) best.most = static_cast<uint32_t>(most);
  }
  return best;
}

// Rows of partial sums that the cut's splits of m rows may need: with fewer rows there may
// be more splits, but no more than fill the chip.
inline uint64_t partial_rows(const MulPlan& p, uint64_t m) {
  if (p.most <= 1) return 0;
  const uint64_t planned = p.splits > 1 ? p.splits * m : 0;
  if (p.most == p.splits) return planned;
  const uint64_t filled = p.fill / p.tiles_n * p.tile;
  return filled > planned ? filled : planned;
}

inline uint64_t chunks_up(uint64_t n, uint64_t to) { return (n + to - 1) / to * to; }

// Elements between 16-bit rows of a workspace: whole 128-byte lines, and not a multiple of
// 4 KiB, whose rows begin in the same channels of the caches (4096 x 4096 over 131072, k
// fast in a: 1311 -> 1395 TFLOP/s).
inline uint64_t row_lead(uint64_t n) {
  const uint64_t lead = chunks_up(n, 64);
  return lead % 2048 ? lead : lead + 64;
}

// Whether a product, and the join of its splits, is one launch each.
inline bool product_fits(const MulPlan& p, uint64_t m, uint64_t n) {
  constexpr uint64_t kMost = most_workgroups(kMulThreads);
  const uint64_t joins = p.most > 1 ? (m * (chunks_up(n, kChunk) / kChunk)) / kMulThreads + 1 : 0;
  return p.tiles <= kMost / p.splits && joins <= kMost;
}

// Enqueues the product (and the join of its splits, if E is a Sink).  m, n and k are
// not 0.  n: columns of c.
template <typename T, bool AF, bool BF, typename E>
hipError_t run_product(const MulPlan& p, const Operand& a, const Operand& b, Extents x, const E& e,
                       hipStream_t stream) {
  x.splits = p.splits;
  x.most = p.most;
  x.fill = p.fill;
  uint64_t wgs = p.tiles * p.splits;
  if (p.most > p.splits && wgs < p.fill) wgs = p.fill;
  if (!product_fits(p, x.m, x.n)) return hipErrorInvalidConfiguration;
  const uint64_t sa = safe_k(a, AF, x.k), sb = safe_k(b, BF, x.k, E::kPairs);
  const uint64_t safe = sa < sb ? sa : sb;
  const uint32_t grid = static_cast<uint32_t>(wgs);
  const bool whole = ring_takes(a, AF, x.k) && ring_takes(b, BF, x.k, E::kPairs);
  if (p.tile == 256 && whole)
    ring_kernel<T, AF, BF, E><<<grid < kRingWgs ? grid : kRingWgs, kMulThreads, 0, stream>>>(
        a, b, x, e);
  else if (p.tile == 256)
    product_kernel<T, AF, BF, 256, 256, 2, 2, E>
        <<<grid, kMulThreads, 0, stream>>>(a, b, x, safe, e);
  else if (p.tile == 128)
    product_kernel<T, AF, BF, 128, 128, 2, 2, E>
        <<<grid, kMulThreads, 0, stream>>>(a, b, x, safe, e);
  else if constexpr (AF) {
    if (whole)
      slim_kernel<T, BF, E><<<grid, kMulThreads, 0, stream>>>(a, b, x, e);
    else
      product_kernel<T, AF, BF, 32, 128, 1, 4, E>
          <<<grid, kMulThreads, 0, stream>>>(a, b, x, safe, e);
  }
  hipError_t err = hipGetLastError();
  if constexpr (!E::kPairs && E::kJoins) {
    if (err != hipSuccess || (p.most == 1 && !e.twice)) return err;
    const uint64_t joins = (x.m * (e.lead / kChunk) + kMulThreads - 1) / kMulThreads;
    join_kernel<T><<<static_cast<uint32_t>(joins), kMulThreads, 0, stream>>>(
        e, x, static_cast<uint32_t>(p.tile), static_cast<uint32_t>(p.tiles_n));
    err = hipGetLastError();
  }
  return err;
}

}  // namespace act
}  // namespace zero

#endif  // ZERO_ACT_PRODUCT_H_
