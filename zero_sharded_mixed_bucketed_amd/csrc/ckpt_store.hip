// 8-bit activation checkpoints: storing 16-bit activations as codes with a
// power-of-two scale per block of 32 columns, and reading them back.
//
// One pass each: a thread takes eight neighbouring columns (a 16-byte load and
// an 8-byte store when writing, the reverse when reading), and the four lanes of
// a block share its largest magnitude by two lane exchanges.  Bound by memory:
// 3 + 1/32 bytes an element each way.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act/format.h"
#include "act/launch.h"

namespace zero {
namespace act {
namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 4;                        // chunks a thread handles
constexpr uint32_t kTile = kThreads * kPerThread;    // chunks of a workgroup

struct Where {  // a chunk's row and its index in the row
  uint64_t row;
  uint32_t chunk;
};

// Chunks are counted row by row, each row padded to whole blocks so that a
// block's lanes are a quad; the workgroup's first chunk is split into row and
// column once, in 64 bits, and the rest by a short division.
__device__ __forceinline__ Where where(uint64_t row0, uint32_t first, uint32_t i,
                                       uint32_t per_row) {
  const uint32_t at = first + i;
  const uint32_t q = at / per_row;
  return {row0 + q, at - q * per_row};
}

template <typename T, int FMT>
__global__ __launch_bounds__(kThreads) void ckpt_write_kernel(StoreLaunch a, uint32_t per_row) {
  const uint64_t base = static_cast<uint64_t>(blockIdx.x) * kTile;
  const uint64_t row0 = base / per_row;
  const uint32_t first = static_cast<uint32_t>(base - row0 * per_row);
  const uint16_t* x = static_cast<const uint16_t*>(a.x);
  u32x4 w[kPerThread];
  Where at[kPerThread];
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    at[j] = where(row0, first, j * kThreads + threadIdx.x, per_row);
    w[j] = u32x4{0, 0, 0, 0};
    const uint64_t col = static_cast<uint64_t>(at[j].chunk) * kChunk;
    if (at[j].row < a.rows && col < a.cols) w[j] = load8(x + at[j].row * a.x_stride, col, a.cols);
  }
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    uint32_t scale;
    const u32x2 codes = encode8<T, FMT>(w[j], &scale);
    if (at[j].row >= a.rows) continue;
    store_codes(a.c.codes + at[j].row * a.c.code_stride,
                static_cast<uint64_t>(at[j].chunk) * kChunk, a.cols, codes);
    if ((at[j].chunk & (kQuad - 1)) == 0)
      a.c.scales[at[j].row * a.c.scale_stride + at[j].chunk / kQuad] =
          static_cast<uint8_t>(scale);
  }
}

template <int DTYPE, int FMT>
__global__ __launch_bounds__(kThreads) void ckpt_read_kernel(StoreLaunch a, uint32_t per_row) {
  const uint64_t base = static_cast<uint64_t>(blockIdx.x) * kTile;
  const uint64_t row0 = base / per_row;
  const uint32_t first = static_cast<uint32_t>(base - row0 * per_row);
  u32x2 w[kPerThread];
  uint32_t s[kPerThread];
  Where at[kPerThread];
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    at[j] = where(row0, first, j * kThreads + threadIdx.x, per_row);
    w[j] = u32x2{0, 0};
    s[j] = 0;
    const uint64_t col = static_cast<uint64_t>(at[j].chunk) * kChunk;
    if (at[j].row < a.rows && col < a.cols) {
      w[j] = load_codes(a.c.codes + at[j].row * a.c.code_stride, col, a.cols);
      s[j] = a.c.scales[at[j].row * a.c.scale_stride + at[j].chunk / kQuad];
    }
  }
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const uint64_t col = static_cast<uint64_t>(at[j].chunk) * kChunk;
    if (at[j].row >= a.rows || col >= a.cols) continue;
    float x[8];
    decode8<FMT>(w[j], scale_of(s[j]), x);
    if constexpr (DTYPE == kF32) {
      float* row = static_cast<float*>(a.x) + at[j].row * a.x_stride;
      if (col + kChunk <= a.cols) {
        *reinterpret_cast<f32x4_at4*>(row + col) = f32x4{x[0], x[1], x[2], x[3]};
        *reinterpret_cast<f32x4_at4*>(row + col + 4) = f32x4{x[4], x[5], x[6], x[7]};
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (col + i < a.cols) row[col + i] = x[i];
      }
    } else {
      using T = typename std::conditional<DTYPE == kF16, F16, Bf16>::type;
      store8(static_cast<uint16_t*>(a.x) + at[j].row * a.x_stride, col, a.cols, pack8<T>(x));
    }
  }
}

// Chunks of a row, in whole blocks, and the grid; 0 workgroups: too large.
uint32_t plan(const StoreLaunch& a, uint32_t* per_row) {
  const uint64_t blocks = (a.cols + kBlock - 1) / kBlock;
  if (blocks > (0x7FFFFFFFull - kTile) / kQuad) return 0;
  *per_row = static_cast<uint32_t>(blocks * kQuad);
  if (a.rows > (0x7FFFFFFFull * kTile) / *per_row) return 0;
  const uint64_t wgs = (a.rows * *per_row + kTile - 1) / kTile;
  return wgs > 0x7FFFFFFFull ? 0 : static_cast<uint32_t>(wgs);
}

}  // namespace

hipError_t launch_ckpt_write(const StoreLaunch& a, hipStream_t stream) {
  uint32_t per_row = 0;
  const uint32_t wgs = plan(a, &per_row);
  if (wgs == 0) return hipErrorInvalidConfiguration;
  if (a.dtype == kF16) {
    if (a.c.format == kInt8)
      ckpt_write_kernel<F16, kInt8><<<wgs, kThreads, 0, stream>>>(a, per_row);
    else
      ckpt_write_kernel<F16, kE4m3><<<wgs, kThreads, 0, stream>>>(a, per_row);
  } else {
    if (a.c.format == kInt8)
      ckpt_write_kernel<Bf16, kInt8><<<wgs, kThreads, 0, stream>>>(a, per_row);
    else
      ckpt_write_kernel<Bf16, kE4m3><<<wgs, kThreads, 0, stream>>>(a, per_row);
  }
  return hipGetLastError();
}

hipError_t launch_ckpt_read(const StoreLaunch& a, hipStream_t stream) {
  uint32_t per_row = 0;
  const uint32_t wgs = plan(a, &per_row);
  if (wgs == 0) return hipErrorInvalidConfiguration;
#define ZERO_READ(D)                                                                \
  (a.c.format == kInt8 ? ckpt_read_kernel<D, kInt8><<<wgs, kThreads, 0, stream>>>(a, per_row) \
                       : ckpt_read_kernel<D, kE4m3><<<wgs, kThreads, 0, stream>>>(a, per_row))
  if (a.dtype == kF16)
    ZERO_READ(kF16);
  else if (a.dtype == kBf16)
    ZERO_READ(kBf16);
  else
    ZERO_READ(kF32);
#undef ZERO_READ
  return hipGetLastError();
}

}  // namespace act
}  // namespace zero
