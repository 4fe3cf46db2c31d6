// A linear layer's weight gradient straight from the 8-bit checkpoint of its
// input: dW[n][k] (+)= sum over tokens t of dY[t][n] * x^[t][k], where x^ is what
// the checkpoint holds.
//
// Every held value is exact in 16 bits, so the products run on the 16-bit matrix
// instructions with the dequantised values themselves, and sums are fp32.  8192
// tokens, 4096 -> 16384 takes 0.93-0.95 ms with e4m3 codes and 1.03-1.10 ms with int8
// ones, 1.00-1.18 PFLOP/s, where a library's plain 16-bit product of the same values,
// dequantised beforehand, takes 0.92-0.97 ms.  Bound by the matrix unit, which is busy
// in half of the cycles beside the codes' arithmetic, and by the clock: 2.05 million
// cycles a pass whatever it takes, 1.09-1.36 ms at 1.9-1.5 GHz in a row of traced
// passes.  Over few tokens the prologue and epilogue of a tile overlap with nothing:
// 256 tokens, 4096 -> 16384 takes 75-78 us, the library 61-63.  The
// long axis t is the slow one of both operands; the matrix instructions want it
// in each lane's registers, so tiles lie in shared memory as they come (t by
// columns, 16 bits) and are read with the transposing shared-memory loads.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act/format.h"
#include "act/launch.h"

namespace zero {
namespace act {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef __bf16 bhalf8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;   // four waves, two by two
constexpr int kFrag = 32;       // rows and columns of a matrix instruction
constexpr int kDepth = 16;      // tokens of a matrix instruction

// Offset of (t, col) in a shared tile of COLS 16-bit columns: rows of 64-byte
// granules whose order is permuted by t, so that the four rows a transposing
// load touches together lie in different banks.
template <int COLS>
__device__ __forceinline__ uint32_t place(uint32_t t, uint32_t col) {
  return t * COLS + ((((col >> 5) ^ (t & 3)) << 5) | (col & 31));
}

__device__ __forceinline__ s16x4 read_tr(const uint16_t* p) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (lds_s16x4*)(__attribute__((address_space(3))) uint16_t*)p);
}

// Half of a 32 x 16 operand: lane l gets column col + l % 32 of four tokens, from
// t + 8 (l / 32) + 4 half on.
template <int COLS>
__device__ __forceinline__ u32x2 half_fragment(const uint16_t* tile, uint32_t t, uint32_t col,
                                               int half) {
  const uint32_t lane = threadIdx.x % 64;
  const uint32_t r = t + (lane / 32) * 8 + (lane % 16) / 4 + half * 4;
  const uint32_t c = col + (lane / 16 % 2) * 16 + lane % 4 * 4;
  return __builtin_bit_cast(u32x2, read_tr(tile + place<COLS>(r, c)));
}

template <typename T>
__device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (T::kType == kF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, a),
                                                  __builtin_bit_cast(half8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bhalf8, a),
                                                   __builtin_bit_cast(bhalf8, b), c, 0, 0, 0);
}

// Orders one wave's shared-memory accesses before and after this point.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Where sums go: dW, or a split's fp32 partial sums.
struct Dest {
  void* p;
  uint64_t stride;
  int dtype, accumulate;
};

__device__ __forceinline__ Dest destination(const WeightGradLaunch& a, uint32_t split,
                                            uint64_t per_split) {
  if (per_split < a.rows)
    return {a.partial + split * a.n * a.k, a.k, kF32, 0};
  return {a.dw, a.dw_stride, a.dw_dtype, a.accumulate};
}

__device__ __forceinline__ void put(const Dest& d, uint64_t at, float s) {
  if (d.dtype == kF32) {
    float* o = static_cast<float*>(d.p) + at;
    *o = d.accumulate ? *o + s : s;
  } else {
    uint16_t* o = static_cast<uint16_t*>(d.p) + at;
    if (d.dtype == kF16)
      *o = static_cast<uint16_t>(pack16<F16>(d.accumulate ? lo16<F16>(*o) + s : s, 0.f));
    else
      *o = static_cast<uint16_t>(pack16<Bf16>(d.accumulate ? lo16<Bf16>(*o) + s : s, 0.f));
  }
}

template <typename T>
__device__ __forceinline__ void put8_16(uint16_t* o, int accumulate, float (&x)[8]) {
  u32x4_at2* w = reinterpret_cast<u32x4_at2*>(o);
  if (accumulate) {
    float old[8];
    unpack8<T>(*w, old);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] += old[i];
  }
  *w = pack8<T>(x);
}

// Eight neighbouring sums of row n from column k on.
__device__ __forceinline__ void put8(const Dest& d, uint64_t n, uint64_t k, uint64_t cols, f32x4 u,
                                     f32x4 v) {
  const uint64_t at = n * d.stride + k;
  float x[8] = {u[0], u[1], u[2], u[3], v[0], v[1], v[2], v[3]};
  if (k + kChunk <= cols) {
    if (d.dtype == kF32) {
      f32x4_at4* o = reinterpret_cast<f32x4_at4*>(static_cast<float*>(d.p) + at);
      if (d.accumulate) {
        u += o[0];
        v += o[1];
      }
      o[0] = u;
      o[1] = v;
    } else if (d.dtype == kF16) {
      put8_16<F16>(static_cast<uint16_t*>(d.p) + at, d.accumulate, x);
    } else {
      put8_16<Bf16>(static_cast<uint16_t*>(d.p) + at, d.accumulate, x);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (k + i < cols) put(d, at + i, x[i]);
}

// The split and tile of a workgroup.  Workgroups go to the eight dies in turn, each
// with an L2 of its own: die x takes the x-th eighth of the pieces, and pieces run
// down groups of eight tile rows, so that the 32 that a die has in hand together
// read 8 + 4 column strips of the operands.
struct Piece {
  uint32_t split, n, k;
};

constexpr uint32_t kDies = 8, kGroupRows = 8;

__device__ __forceinline__ Piece piece_of(uint32_t wg, uint32_t wgs, uint32_t tk,
                                          uint32_t tiles) {
  const uint32_t die = wg % kDies, each = wgs / kDies, more = wgs % kDies;
  const uint32_t id = die * each + (die < more ? die : more) + wg / kDies;
  const uint32_t split = id / tiles, tile = id % tiles;
  const uint32_t tn = tiles / tk, group = tile / (kGroupRows * tk);
  const uint32_t rest = tile % (kGroupRows * tk), row0 = group * kGroupRows;
  const uint32_t rows = tn - row0 < kGroupRows ? tn - row0 : kGroupRows;
  return {split, row0 + rest % rows, rest / rows};
}

// A workgroup's TILE x TILE piece of dW over one split of the tokens, DEPTH tokens
// at a time through two buffers of shared memory.  While the matrix unit works on
// one tile, the next one goes from registers to the other buffer, dequantised, and
// the one after it is loaded into those registers; the operands of a matrix step
// are read during the step before it.
//
// Whole tiles below token `safe` are loaded without a branch: chunks that pass a
// row's end read what follows it, which reaches only sums that are not stored.
// Other tiles are loaded with every check.
template <typename T, int FMT, int TILE, int DEPTH>
__global__ __launch_bounds__(kThreads) void weight_grad_kernel(WeightGradLaunch a,
                                                               uint64_t safe, uint64_t per_split,
                                                               uint32_t tk, uint32_t tiles) {
  constexpr int kF = TILE / 2 / kFrag;                    // fragments of a wave, each way
  constexpr uint32_t kRowLanes = TILE / kChunk;           // lanes of a tile row
  constexpr uint32_t kStep = kThreads / kRowLanes;        // rows a pass of the workgroup
  constexpr int kPass = DEPTH / kStep;                    // passes a tile
  constexpr int kSub = DEPTH / kDepth;                    // matrix steps a tile
  // two tiles of each operand; at the end, 32 rows of each wave's sums
  constexpr uint32_t kCols = TILE / 2, kPitch = kCols + 8;
  constexpr uint32_t kTiles = 2 * DEPTH * TILE, kOut = 4 * kFrag * kPitch;
  __shared__ float lds[kTiles > kOut ? kTiles : kOut];
  uint16_t (*ly)[DEPTH * TILE] = reinterpret_cast<uint16_t (*)[DEPTH * TILE]>(lds);
  uint16_t (*lx)[DEPTH * TILE] = ly + 2;
  const Piece piece_at = piece_of(blockIdx.x, gridDim.x, tk, tiles);
  const uint32_t split = piece_at.split;
  const uint64_t n0 = static_cast<uint64_t>(piece_at.n) * TILE;
  const uint64_t k0 = static_cast<uint64_t>(piece_at.k) * TILE;
  const uint64_t t_lo = split * per_split;
  const uint64_t t_hi = t_lo + per_split < a.rows ? t_lo + per_split : a.rows;
  const uint32_t tid = threadIdx.x, wave = tid / 64;
  const uint32_t wn = wave / 2 * (TILE / 2), wk = wave % 2 * (TILE / 2);

  u32x4 ry[kPass];
  u32x2 rx[kPass];
  uint32_t rs[kPass];
  const uint32_t st = tid / kRowLanes, sc = tid % kRowLanes * kChunk;
  const bool in_n = n0 + sc < a.n, in_k = k0 + sc < a.k;
  // with every check: t < t_hi, columns inside, any alignment
  auto load_any = [&](uint64_t t0) {
#pragma unroll 1
    for (int i = 0; i < kPass; ++i) {
      const uint64_t t = t0 + i * kStep + st;
      u32x4 y = {0, 0, 0, 0};
      u32x2 x = {0, 0};
      uint32_t b = 0;
      if (t < t_hi) {
        if (in_n) y = load8(a.dy + t * a.dy_stride, n0 + sc, a.n);
        if (in_k) {
          x = load_codes(a.x.codes + t * a.x.code_stride, k0 + sc, a.k);
          b = a.x.scales[t * a.x.scale_stride + (k0 + sc) / kBlock];
        }
      }
#pragma unroll
      for (int q = 0; q < kPass; ++q)                     // registers take fixed indexes
        if (q == i) {
          ry[q] = y;
          rx[q] = x;
          rs[q] = b;
        }
    }
  };
  // Bytes from a pass's first row to the lane's columns (column 0 where the tile
  // passes the matrix's edge); the row itself is the same for all lanes.
  const uint32_t oy = st * static_cast<uint32_t>(a.dy_stride) * 2 +
                      static_cast<uint32_t>(in_n ? n0 + sc : 0) * 2;
  const uint32_t ox = st * static_cast<uint32_t>(a.x.code_stride) +
                      static_cast<uint32_t>(in_k ? k0 + sc : 0);
  const uint32_t os = st * static_cast<uint32_t>(a.x.scale_stride) +
                      static_cast<uint32_t>(in_k ? (k0 + sc) / kBlock : 0);
  auto load_one = [&](uint64_t t0, int i) {               // tokens below `whole`
    const uint64_t t = t0 + i * kStep;
    ry[i] = *reinterpret_cast<const u32x4_at2*>(
        reinterpret_cast<const uint8_t*>(a.dy + t * a.dy_stride) + oy);
    rx[i] = *reinterpret_cast<const u32x2_at1*>(a.x.codes + t * a.x.code_stride + ox);
    rs[i] = *(a.x.scales + t * a.x.scale_stride + os);
  };
  // A pass from registers to shared memory in kParts parts, the loads that refill
  // its registers last.
  constexpr int kParts = 6;
  Scale16<T, FMT> scale;
  u32x4 held;
  auto stage = [&](int buf, int i, int part) {
    const uint32_t t = i * kStep + st;
    switch (part) {
      case 0:
        // keeps the compiler from taking the codes apart where they are loaded,
        // which would wait for the load there
        asm("" : "+v"(rx[i][0]), "+v"(rx[i][1]), "+v"(rs[i]));
        scale.set(rs[i]);
        break;
      case 1: held[0] = scale.template pair<0>(rx[i]); break;
      case 2: held[1] = scale.template pair<1>(rx[i]); break;
      case 3: held[2] = scale.template pair<2>(rx[i]); break;
      case 4: held[3] = scale.template pair<3>(rx[i]); break;
      default:
        *reinterpret_cast<u32x4*>(&ly[buf][place<TILE>(t, sc)]) = ry[i];
        *reinterpret_cast<u32x4*>(&lx[buf][place<TILE>(t, sc)]) = held;
    }
  };
  const uint64_t whole = t_hi < safe ? t_hi : safe;
  auto load = [&](uint64_t t0) {
    if (t0 + DEPTH <= whole) {
#pragma unroll
      for (int i = 0; i < kPass; ++i) load_one(t0, i);
    } else {
      load_any(t0);
    }
  };

  f32x16 acc[kF][kF];
#pragma unroll
  for (int i = 0; i < kF; ++i)
#pragma unroll
    for (int j = 0; j < kF; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  // Operands of a step: 4 kF transposing loads, in the order of their use.
  u32x4 fy[2][kF], fx[2][kF];
  auto read = [&](int buf, int s, int to, int q) {
    const int f = q / 2, half = q % 2;
    // fragments in order: y0, x0 .. x(kF-1), y1 .. y(kF-1)
    const bool of_x = f >= 1 && f <= kF;
    const int i = of_x ? f - 1 : f == 0 ? 0 : f - kF;
    const uint16_t* tile_at = of_x ? lx[buf] : ly[buf];
    const u32x2 v = half_fragment<TILE>(tile_at, s * kDepth, (of_x ? wk : wn) + i * kFrag, half);
    u32x4& reg = of_x ? fx[to][i] : fy[to][i];
    reg[2 * half] = v[0];
    reg[2 * half + 1] = v[1];
  };
  auto read_all = [&](int buf, int s, int to) {
#pragma unroll
    for (int q = 0; q < 4 * kF; ++q) read(buf, s, to, q);
  };

  load(t_lo);
#pragma unroll
  for (int i = 0; i < kPass; ++i)
#pragma unroll
    for (int q = 0; q < kParts; ++q) stage(0, i, q);
  load(t_lo + DEPTH);
  __syncthreads();
  read_all(0, 0, 0);
  uint32_t buf = 0;
  uint64_t t0 = t_lo;
  static_assert(kSub % 2 == 0, "the operands' registers take turns");
  // A turn: all of tile t0's steps; tile t0 + DEPTH from registers to the other
  // buffer (last read before the barrier of the turn before) over all steps but the
  // last; then the barrier, behind which the next tile's first operands are read
  // while the last step runs.  Between two matrix instructions goes about as much
  // other work as one of them takes, and the compiler keeps it there: left to
  // itself it gathers the arithmetic in long runs, beside which the matrix unit
  // stands idle.
  constexpr int kMul = kF * kF;                            // matrix instructions a step
  constexpr int kSlots = (kSub - 1) * kMul;
  constexpr int kPerSlot = (kPass * kParts + kSlots - 1) / kSlots;
  auto turn = [&](auto refill) {
#pragma unroll
    for (int s = 0; s < kSub; ++s) {
      const bool last = s + 1 == kSub;
      if (last) __syncthreads();
#pragma unroll
      for (int m = 0; m < kMul; ++m) {
        const int i = m / kF, j = m % kF;
        acc[i][j] = mfma<T>(fy[s & 1][i], fx[s & 1][j], acc[i][j]);
#pragma unroll
        for (int q = m * 4 / kF; q < (m + 1) * 4 / kF; ++q)
          read(last ? buf ^ 1 : buf, last ? 0 : s + 1, (s + 1) & 1, q);
        if (!last) {
#pragma unroll
          for (int q = 0; q < kPerSlot; ++q) {
            const int w = (s * kMul + m) * kPerSlot + q;
            if (w >= kPass * kParts) continue;
            stage(buf ^ 1, w / kParts, w % kParts);
            if (w % kParts == kParts - 1) refill(w / kParts);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    buf ^= 1;
  };
#pragma unroll 1
  for (; t0 + 3 * DEPTH <= whole; t0 += DEPTH)
    turn([&](int i) { load_one(t0 + 2 * DEPTH, i); });
#pragma unroll 1
  for (; t0 < t_hi; t0 += DEPTH) {
    turn([](int) {});
    load_any(t0 + 2 * DEPTH);   // zeros past the end
  }
  __syncthreads();

  // Through shared memory, so that a lane stores eight neighbouring columns: each
  // wave turns 32 rows at a time in a piece of its own, whose rows lie kPitch
  // words apart (4 kPitch = 32 mod 64: the two halves of a wave, four rows apart,
  // meet different banks).
  const uint32_t lane = tid % 64;
  static_assert((4 * kPitch) % 64 == 32, "");
  float* piece = lds + wave * kFrag * kPitch;
  const Dest out = destination(a, split, per_split);
  // a whole tile that is only stored, in 16-byte pieces
  const bool inside = !out.accumulate && n0 + TILE <= a.n && k0 + TILE <= a.k;
#pragma unroll
  for (int i = 0; i < kF; ++i) {
#pragma unroll
    for (int j = 0; j < kF; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        piece[(r / 4 * 8 + lane / 32 * 4 + r % 4) * kPitch + j * kFrag + lane % 32] =
            acc[i][j][r];
    wave_order();
    constexpr uint32_t kLanes = kCols / kChunk;           // lanes of a row
    constexpr int kRows = kFrag * kLanes / 64;            // passes over the 32 rows
    const uint32_t q = lane / kLanes, c = lane % kLanes * kChunk;
    const uint64_t n = n0 + wn + i * kFrag + q, k = k0 + wk + c;
    const float* p = piece + q * kPitch + c;
    f32x4 u[kRows], v[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      u[r] = *reinterpret_cast<const f32x4*>(p + r * (64 / kLanes) * kPitch);
      v[r] = *reinterpret_cast<const f32x4*>(p + r * (64 / kLanes) * kPitch + 4);
    }
    if (inside && out.dtype == T::kType) {
      uint16_t* o = static_cast<uint16_t*>(out.p) + n * out.stride + k;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float x[8] = {u[r][0], u[r][1], u[r][2], u[r][3], v[r][0], v[r][1], v[r][2], v[r][3]};
        *reinterpret_cast<u32x4_at2*>(o + r * (64 / kLanes) * out.stride) = pack8<T>(x);
      }
    } else if (inside) {
      float* o = static_cast<float*>(out.p) + n * out.stride + k;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        *reinterpret_cast<f32x4_at4*>(o + r * (64 / kLanes) * out.stride) = u[r];
        *reinterpret_cast<f32x4_at4*>(o + r * (64 / kLanes) * out.stride + 4) = v[r];
      }
    } else {
#pragma unroll 1
      for (int r = 0; r < kRows; ++r) {
        const float* pr = p + r * (64 / kLanes) * kPitch;
        const uint64_t row = n + r * (64 / kLanes);
        if (row < a.n && k < a.k)
          put8(out, row, k, a.k, *reinterpret_cast<const f32x4*>(pr),
               *reinterpret_cast<const f32x4*>(pr + 4));
      }
    }
    wave_order();
  }
}

// Adds the splits' partial sums in their order, eight neighbouring columns a thread.
__global__ __launch_bounds__(kThreads) void weight_grad_join_kernel(WeightGradLaunch a,
                                                                    uint32_t splits) {
  const uint64_t per_row = (a.k + kChunk - 1) / kChunk, count = a.n * a.k;
  const uint64_t id = static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const uint64_t n = id / per_row, k = id % per_row * kChunk;
  if (n >= a.n) return;
  const bool whole = k + kChunk <= a.k;
  f32x4 u = {0.f, 0.f, 0.f, 0.f}, v = u;
  const float* p = a.partial + n * a.k + k;
#pragma unroll 8
  for (uint32_t s = 0; s < splits; ++s, p += count) {
    if (whole) {
      u += *reinterpret_cast<const f32x4_at4*>(p);
      v += *reinterpret_cast<const f32x4_at4*>(p + 4);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (k + i < a.k) u[i] += p[i];
        if (k + 4 + i < a.k) v[i] += p[4 + i];
      }
    }
  }
  put8({a.dw, a.dw_stride, a.dw_dtype, a.accumulate}, n, k, a.k, u, v);
}

struct Plan {
  int tile;
  uint64_t tn, tk, splits, per_split;
};

// Estimated microseconds of a choice, from measurements on MI355X: a workgroup of
// 256 x 256 has a compute unit to itself and takes 14 us and 0.028 a token; one of
// 128 x 128 takes 7 us and 0.015 a token alone on its unit, 0.021 beside a second
// one; a join costs a launch, and its partial sums' way out and back.
double estimate(int tile, uint64_t wgs, uint64_t splits, uint64_t per_split, uint64_t outs) {
  constexpr uint64_t kUnits = 256;
  const uint64_t at_once = tile == 256 ? kUnits : 2 * kUnits;
  const double rounds = static_cast<double>((wgs + at_once - 1) / at_once);
  const double token = tile == 256 ? 0.028 : wgs > kUnits ? 0.021 : 0.015;
  const double run = rounds * ((tile == 256 ? 14.0 : 7.0) + token * static_cast<double>(per_split));
  return splits == 1 ? run
                     : run + 3.0 + static_cast<double>(splits) * static_cast<double>(outs) * 8 / 6e6;
}

// The tile and the number of splits with the least estimate.  Small tiles fill the
// chip with less output, splits with more tokens: at 16001 x 1032 -> 776 the best
// choice takes 53 us where one split of 256 x 256 tiles takes 395.
Plan plan(uint64_t rows, uint64_t k, uint64_t n) {
  Plan best;
  double least = 0;
  bool first = true;
  for (int tile = 128; tile <= 256; tile *= 2) {
    Plan p;
    p.tile = tile;
    p.tn = (n + tile - 1) / tile;
    p.tk = (k + tile - 1) / tile;
    for (const uint64_t s : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64}) {
      if (s > 1 && rows < 256 * s) break;   // a split sums 256 tokens at least
      p.per_split = rows ? ((rows + s - 1) / s + 63) / 64 * 64 : 64;
      p.splits = rows ? (rows + p.per_split - 1) / p.per_split : 1;
      const double us = estimate(tile, p.tn * p.tk * p.splits, p.splits, p.per_split, n * k);
      if (first || us < least) {
        least = us;
        best = p;
        first = false;
      }
    }
  }
  return best;
}

template <typename T, int FMT>
void run(const WeightGradLaunch& a, const Plan& p, uint32_t wgs, uint64_t safe,
         hipStream_t stream) {
  const uint32_t tk = static_cast<uint32_t>(p.tk), tiles = static_cast<uint32_t>(p.tn * p.tk);
  if (p.tile == 256)
    weight_grad_kernel<T, FMT, 256, 64>
        <<<wgs, kThreads, 0, stream>>>(a, safe, p.per_split, tk, tiles);
  else
    weight_grad_kernel<T, FMT, 128, 64>
        <<<wgs, kThreads, 0, stream>>>(a, safe, p.per_split, tk, tiles);
}

// Rows of a rows x cols matrix whose chunks all end inside it, though the last one
// may pass its own row's end.
uint64_t safe_rows(uint64_t rows, uint64_t cols, uint64_t stride) {
  const uint64_t over = (kChunk - cols % kChunk) % kChunk;
  if (over == 0) return rows;
  const uint64_t back = rows > 1 ? (over + stride - 1) / stride : rows;
  return back < rows ? rows - back : 0;
}

}  // namespace

uint64_t weight_grad_workspace(uint64_t rows, uint64_t k, uint64_t n) {
  const Plan p = plan(rows, k, n);
  return p.splits > 1 ? p.splits * n * k * sizeof(float) : 0;
}

hipError_t launch_weight_grad(const WeightGradLaunch& a, hipStream_t stream) {
  const Plan p = plan(a.rows, a.k, a.n);
  const uint64_t wgs = p.tn * p.tk * p.splits;
  const uint64_t joins = (a.n * ((a.k + kChunk - 1) / kChunk) + kThreads - 1) / kThreads;
  // past what one launch holds dw would take 2^38 elements, or its splits' sums 2^38
  // bytes beside it: more memory than the chip has
  constexpr uint64_t kMost = most_workgroups(kThreads);
  if (wgs > kMost || (p.splits > 1 && joins > kMost)) return hipErrorInvalidConfiguration;
  const uint64_t of_y = safe_rows(a.rows, a.n, a.dy_stride);
  const uint64_t of_x = safe_rows(a.rows, a.k, a.x.code_stride);
  uint64_t safe = of_y < of_x ? of_y : of_x;
  // offsets inside a pass of 16 rows are 32 bits wide
  constexpr uint64_t kFar = 1ull << 26;
  if (a.dy_stride >= kFar || a.x.code_stride >= kFar || a.x.scale_stride >= kFar) safe = 0;
  if (a.dtype == kF16) {
    if (a.x.format == kInt8) run<F16, kInt8>(a, p, wgs, safe, stream);
    else run<F16, kE4m3>(a, p, wgs, safe, stream);
  } else {
    if (a.x.format == kInt8) run<Bf16, kInt8>(a, p, wgs, safe, stream);
    else run<Bf16, kE4m3>(a, p, wgs, safe, stream);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  weight_grad_join_kernel<<<static_cast<uint32_t>(joins), kThreads, 0, stream>>>(
      a, static_cast<uint32_t>(p.splits));
  return hipGetLastError();
}

}  // namespace act
}  // namespace zero
