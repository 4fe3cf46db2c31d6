// A linear layer's weight gradient straight from the 8-bit checkpoint of its
// input: dW[n][k] (+)= sum over tokens t of dY[t][n] * x^[t][k], where x^ is what
// the checkpoint holds.
//
// Every held value is exact in 16 bits, so the products run on the 16-bit matrix
// instructions with the dequantised values themselves, and sums are fp32.  The
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
constexpr int kTileN = 128, kTileK = 128, kTileT = 32;
constexpr int kFrag = 32;       // rows and columns of a matrix instruction
constexpr int kFn = kTileN / 2 / kFrag, kFk = kTileK / 2 / kFrag;

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

// A 32 x 16 operand: lane l gets column col + l % 32 of rows t .. t + 7 or
// t + 8 .. t + 15 (upper lanes).
template <int COLS>
__device__ __forceinline__ u32x4 fragment(const uint16_t* tile, uint32_t t, uint32_t col) {
  const uint32_t lane = threadIdx.x % 64;
  const uint32_t r = t + (lane / 32) * 8 + (lane % 16) / 4;
  const uint32_t c = col + (lane / 16 % 2) * 16 + lane % 4 * 4;
  const s16x4 a = read_tr(tile + place<COLS>(r, c));
  const s16x4 b = read_tr(tile + place<COLS>(r + 4, c));
  const u32x2 x = __builtin_bit_cast(u32x2, a), y = __builtin_bit_cast(u32x2, b);
  return u32x4{x[0], x[1], y[0], y[1]};
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

__device__ __forceinline__ void put(void* dw, uint64_t at, int dtype, int accumulate, float s) {
  if (dtype == kF32) {
    float* o = static_cast<float*>(dw) + at;
    *o = accumulate ? *o + s : s;
  } else {
    uint16_t* o = static_cast<uint16_t*>(dw) + at;
    if (dtype == kF16)
      *o = static_cast<uint16_t>(pack16<F16>(accumulate ? lo16<F16>(*o) + s : s, 0.f));
    else
      *o = static_cast<uint16_t>(pack16<Bf16>(accumulate ? lo16<Bf16>(*o) + s : s, 0.f));
  }
}

template <typename T, int FMT>
__global__ __launch_bounds__(kThreads) void weight_grad_kernel(WeightGradLaunch a, int dy_wide,
                                                               uint64_t per_split) {
  __shared__ uint16_t ly[2][kTileT * kTileN];
  __shared__ uint16_t lx[2][kTileT * kTileK];
  const uint64_t n0 = static_cast<uint64_t>(blockIdx.y) * kTileN;
  const uint64_t k0 = static_cast<uint64_t>(blockIdx.x) * kTileK;
  const uint64_t t_lo = blockIdx.z * per_split;
  const uint64_t t_hi = t_lo + per_split < a.rows ? t_lo + per_split : a.rows;
  const uint32_t tid = threadIdx.x, wave = tid / 64;
  const uint32_t wn = wave / 2 * (kTileN / 2), wk = wave % 2 * (kTileK / 2);

  u32x4 ry[2];
  u32x2 rx[2];
  uint32_t rs[2];
  constexpr uint32_t kRowLanes = kTileN / kChunk;   // lanes of a tile row
  constexpr uint32_t kStep = kThreads / kRowLanes;  // rows a pass
  const uint32_t st = tid / kRowLanes, sc = tid % kRowLanes * kChunk;
  auto load = [&](uint64_t t0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t t = t0 + i * kStep + st;
      ry[i] = u32x4{0, 0, 0, 0};
      rx[i] = u32x2{0, 0};
      rs[i] = 0;
      if (t >= t_hi) continue;
      if (n0 + sc < a.n) ry[i] = load8(a.dy + t * a.dy_stride, n0 + sc, a.n, dy_wide);
      if (k0 + sc < a.k) {
        rx[i] = load_codes(a.x.codes + t * a.x.code_stride, k0 + sc, a.k, a.x.wide);
        rs[i] = a.x.scales[t * a.x.scale_stride + (k0 + sc) / kBlock];
      }
    }
  };
  f32x16 acc[kFn][kFk];
#pragma unroll
  for (int i = 0; i < kFn; ++i)
#pragma unroll
    for (int j = 0; j < kFk; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  load(t_lo);
  int buf = 0;
  for (uint64_t t0 = t_lo; t0 < t_hi; t0 += kTileT, buf ^= 1) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t t = i * kStep + st;
      *reinterpret_cast<u32x4*>(&ly[buf][place<kTileN>(t, sc)]) = ry[i];
      float x[8];
      decode8<FMT>(rx[i], scale_of(rs[i]), x);
      *reinterpret_cast<u32x4*>(&lx[buf][place<kTileK>(t, sc)]) = pack8<T>(x);
    }
    // the other buffer was last read before the barrier of the turn before
    __syncthreads();
    if (t0 + kTileT < t_hi) load(t0 + kTileT);
#pragma unroll
    for (int s = 0; s < kTileT; s += 16) {
      u32x4 fy[kFn], fx[kFk];
#pragma unroll
      for (int i = 0; i < kFn; ++i) fy[i] = fragment<kTileN>(ly[buf], s, wn + i * kFrag);
#pragma unroll
      for (int j = 0; j < kFk; ++j) fx[j] = fragment<kTileK>(lx[buf], s, wk + j * kFrag);
#pragma unroll
      for (int i = 0; i < kFn; ++i)
#pragma unroll
        for (int j = 0; j < kFk; ++j) acc[i][j] = mfma<T>(fy[i], fx[j], acc[i][j]);
    }
  }

  const uint32_t lane = tid % 64;
  float* part = gridDim.z > 1 ? a.partial + blockIdx.z * a.n * a.k : nullptr;
#pragma unroll
  for (int i = 0; i < kFn; ++i)
#pragma unroll
    for (int j = 0; j < kFk; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const uint64_t n = n0 + wn + i * kFrag + r / 4 * 8 + lane / 32 * 4 + r % 4;
        const uint64_t k = k0 + wk + j * kFrag + lane % 32;
        if (n >= a.n || k >= a.k) continue;
        if (part) part[n * a.k + k] = acc[i][j][r];
        else put(a.dw, n * a.dw_stride + k, a.dw_dtype, a.accumulate, acc[i][j][r]);
      }
}

// Adds the splits' partial sums in their order.
__global__ __launch_bounds__(kThreads) void weight_grad_join_kernel(WeightGradLaunch a,
                                                                    uint32_t splits) {
  const uint64_t count = a.n * a.k;
  for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x; i < count;
       i += static_cast<uint64_t>(gridDim.x) * kThreads) {
    float s = 0.f;
    for (uint32_t p = 0; p < splits; ++p) s += a.partial[p * count + i];
    put(a.dw, i / a.k * a.dw_stride + i % a.k, a.dw_dtype, a.accumulate, s);
  }
}

struct Plan {
  uint64_t tn, tk, splits, per_split;
};

Plan plan(uint64_t rows, uint64_t k, uint64_t n) {
  Plan p;
  p.tn = (n + kTileN - 1) / kTileN;
  p.tk = (k + kTileK - 1) / kTileK;
  const uint64_t tiles = p.tn * p.tk;
  uint64_t s = tiles < 512 ? 512 / tiles : 1;
  const uint64_t most = rows / 256;  // a split sums 256 tokens at least
  if (s > most) s = most;
  if (s < 1) s = 1;
  p.per_split = ((rows + s - 1) / s + kTileT - 1) / kTileT * kTileT;
  if (p.per_split == 0) p.per_split = kTileT;
  p.splits = (rows + p.per_split - 1) / p.per_split;
  if (p.splits == 0) p.splits = 1;
  return p;
}

}  // namespace

uint64_t weight_grad_workspace(uint64_t rows, uint64_t k, uint64_t n) {
  const Plan p = plan(rows, k, n);
  return p.splits > 1 ? p.splits * n * k * sizeof(float) : 0;
}

hipError_t launch_weight_grad(const WeightGradLaunch& a, hipStream_t stream) {
  const Plan p = plan(a.rows, a.k, a.n);
  if (p.tk > 0x7FFFFFFFull || p.tn > 65535) return hipErrorInvalidConfiguration;
  const int dy_wide = reinterpret_cast<uintptr_t>(a.dy) % 16 == 0 && a.dy_stride % 8 == 0;
  const dim3 grid(static_cast<uint32_t>(p.tk), static_cast<uint32_t>(p.tn),
                  static_cast<uint32_t>(p.splits));
  if (a.dtype == kF16) {
    if (a.x.format == kInt8)
      weight_grad_kernel<F16, kInt8><<<grid, kThreads, 0, stream>>>(a, dy_wide, p.per_split);
    else
      weight_grad_kernel<F16, kE4m3><<<grid, kThreads, 0, stream>>>(a, dy_wide, p.per_split);
  } else {
    if (a.x.format == kInt8)
      weight_grad_kernel<Bf16, kInt8><<<grid, kThreads, 0, stream>>>(a, dy_wide, p.per_split);
    else
      weight_grad_kernel<Bf16, kE4m3><<<grid, kThreads, 0, stream>>>(a, dy_wide, p.per_split);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const uint64_t wgs = (a.n * a.k + kThreads - 1) / kThreads;
  weight_grad_join_kernel<<<static_cast<uint32_t>(wgs < 4096 ? wgs : 4096), kThreads, 0, stream>>>(
      a, static_cast<uint32_t>(p.splits));
  return hipGetLastError();
}

}  // namespace act
}  // namespace zero
