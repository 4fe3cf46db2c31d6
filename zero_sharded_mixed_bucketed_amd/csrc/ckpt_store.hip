// 8-bit activation checkpoints: storing 16-bit activations as codes with a
// power-of-two scale per block of 32 columns, and reading them back.
//
// One pass each: a thread takes eight neighbouring columns (a 16-byte load and an
// 8-byte store when writing, the reverse when reading), and the four lanes of a
// block share its largest magnitude by two lane exchanges.  Bound by memory, 3 + 1/32
// bytes an element: 16384 x 4096 bf16 is written in 33 us (6.2 TB/s) and read back in
// 38 (5.4 TB/s), or in 30 while its codes still lie in the last-level cache.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "act/format.h"
#include "act/launch.h"

namespace zero {
namespace act {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kUnits = 4;                        // units a wave takes, loaded together
constexpr uint64_t kMostUnits = most_workgroups(kThreads) * kWaves * kUnits;  // of a launch

// A wave's unit: 512 columns of a row (64 lanes of eight), or, where rows have at
// most 256 columns, 64 / lanes whole rows, lanes the least power of two that holds
// one (a block's four lanes never part).  Rows and pieces are the wave's, not the
// lane's, so finding them costs no vector arithmetic: with a division a lane instead
// a write of 16384 x 4096 took 42 us where it now takes 33.
struct Shape {
  uint64_t row0;      // of the launch
  uint32_t units;
  uint32_t segments;  // units of a row, NARROW: 1
  uint32_t lanes;     // of a row
};

template <bool NARROW>
struct Place {
  uint64_t row;
  uint32_t col;
  bool live;

  __device__ __forceinline__ Place(const Shape& s, uint64_t rows, uint32_t unit) {
    const uint32_t lane = threadIdx.x % 64;
    if constexpr (NARROW) {
      const uint32_t each = 64 / s.lanes;
      row = s.row0 + static_cast<uint64_t>(unit) * each + lane / s.lanes;
      col = lane % s.lanes * kChunk;
      live = unit < s.units && row < rows;
    } else {
      const uint32_t r = unit / s.segments;
      row = s.row0 + r;
      col = (unit - r * s.segments) * (64 * kChunk) + lane * kChunk;
      live = unit < s.units;
    }
  }
};

__device__ __forceinline__ uint32_t first_unit() {
  return (blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / 64)) * kUnits;
}

template <typename T, int FMT, bool NARROW>
__global__ __launch_bounds__(kThreads) void ckpt_write_kernel(StoreLaunch a, Shape s) {
  const uint32_t unit = first_unit(), cols = static_cast<uint32_t>(a.cols);
  const uint16_t* x = static_cast<const uint16_t*>(a.x);
  u32x4 w[kUnits];
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const Place<NARROW> p(s, a.rows, unit + j);
    w[j] = u32x4{0, 0, 0, 0};
    if (p.live && p.col < cols) w[j] = stream8(x + p.row * a.x_stride, p.col, cols);
  }
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const Place<NARROW> p(s, a.rows, unit + j);
    uint32_t scale;
    const u32x2 codes = encode8<T, FMT>(w[j], &scale);
    if (!p.live || p.col >= cols) continue;
    store_codes(a.c.codes + p.row * a.c.code_stride, p.col, cols, codes);
    if (p.col % kBlock == 0)
      a.c.scales[p.row * a.c.scale_stride + p.col / kBlock] = static_cast<uint8_t>(scale);
  }
}

template <int DTYPE, int FMT, bool NARROW>
__global__ __launch_bounds__(kThreads) void ckpt_read_kernel(StoreLaunch a, Shape s) {
  const uint32_t unit = first_unit(), cols = static_cast<uint32_t>(a.cols);
  u32x2 w[kUnits];
  uint32_t b[kUnits];
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const Place<NARROW> p(s, a.rows, unit + j);
    w[j] = u32x2{0, 0};
    b[j] = 0;
    if (p.live && p.col < cols) {
      w[j] = load_codes(a.c.codes + p.row * a.c.code_stride, p.col, cols);
      b[j] = a.c.scales[p.row * a.c.scale_stride + p.col / kBlock];
    }
  }
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const Place<NARROW> p(s, a.rows, unit + j);
    if (!p.live || p.col >= cols) continue;
    float x[8];
    decode8<FMT>(w[j], scale_of(b[j]), x);
    if constexpr (DTYPE == kF32) {
      float* row = static_cast<float*>(a.x) + p.row * a.x_stride;
      if (p.col + kChunk <= cols) {
        __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]},
                                    reinterpret_cast<f32x4_at4*>(row + p.col));
        __builtin_nontemporal_store(f32x4{x[4], x[5], x[6], x[7]},
                                    reinterpret_cast<f32x4_at4*>(row + p.col + 4));
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (p.col + i < cols) row[p.col + i] = x[i];
      }
    } else {
      using T = typename std::conditional<DTYPE == kF16, F16, Bf16>::type;
      store8(static_cast<uint16_t*>(a.x) + p.row * a.x_stride, p.col, cols, pack8<T>(x));
    }
  }
}

// Calls launch(narrow, workgroups, shape) for as many launches as the rows take.
template <typename F>
hipError_t for_units(const StoreLaunch& a, F launch) {
  if (a.cols > (1ull << 31)) return hipErrorInvalidConfiguration;
  const uint32_t chunks = static_cast<uint32_t>((a.cols + kBlock - 1) / kBlock) * kQuad;
  Shape s;
  s.lanes = kQuad;
  while (s.lanes < chunks && s.lanes < 64) s.lanes *= 2;
  const bool narrow = s.lanes < 64;
  s.segments = narrow ? 1 : (chunks + 63) / 64;
  const uint64_t per = narrow ? 64 / s.lanes : 1;           // rows of a unit
  const uint64_t most = kMostUnits / s.segments * per;      // rows of a launch
  for (s.row0 = 0; s.row0 < a.rows; s.row0 += most) {
    const uint64_t rows = a.rows - s.row0 < most ? a.rows - s.row0 : most;
    s.units = static_cast<uint32_t>((rows + per - 1) / per * s.segments);
    launch(narrow, (s.units - 1) / (kWaves * kUnits) + 1, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T, int FMT>
hipError_t write(const StoreLaunch& a, hipStream_t stream) {
  return for_units(a, [&](bool narrow, uint32_t wgs, const Shape& s) {
    if (narrow) ckpt_write_kernel<T, FMT, true><<<wgs, kThreads, 0, stream>>>(a, s);
    else ckpt_write_kernel<T, FMT, false><<<wgs, kThreads, 0, stream>>>(a, s);
  });
}

template <int DTYPE, int FMT>
hipError_t read(const StoreLaunch& a, hipStream_t stream) {
  return for_units(a, [&](bool narrow, uint32_t wgs, const Shape& s) {
    if (narrow) ckpt_read_kernel<DTYPE, FMT, true><<<wgs, kThreads, 0, stream>>>(a, s);
    else ckpt_read_kernel<DTYPE, FMT, false><<<wgs, kThreads, 0, stream>>>(a, s);
  });
}

}  // namespace

hipError_t launch_ckpt_write(const StoreLaunch& a, hipStream_t stream) {
  if (a.dtype == kF16)
    return a.c.format == kInt8 ? write<F16, kInt8>(a, stream) : write<F16, kE4m3>(a, stream);
  return a.c.format == kInt8 ? write<Bf16, kInt8>(a, stream) : write<Bf16, kE4m3>(a, stream);
}

hipError_t launch_ckpt_read(const StoreLaunch& a, hipStream_t stream) {
  const bool i8 = a.c.format == kInt8;
  if (a.dtype == kF16) return i8 ? read<kF16, kInt8>(a, stream) : read<kF16, kE4m3>(a, stream);
  if (a.dtype == kBf16) return i8 ? read<kBf16, kInt8>(a, stream) : read<kBf16, kE4m3>(a, stream);
  return i8 ? read<kF32, kInt8>(a, stream) : read<kF32, kE4m3>(a, stream);
}

}  // namespace act
}  // namespace zero
