// The norms before and after a block, fused with the block's gate and residual
// scale: per token, in fp32,
//   o  = post(b);  h' = h + s * (g . o);  z = pre(h')
// with post and pre an RMS or layer norm (or none), and their backward from the
// 8-bit checkpoints of b and h'.
//
// A row is held by W waves, two chunks of eight columns a thread, from the first
// load to the last store: each input is read once and each output written once,
// and the row sums go through lane exchanges and, between waves, shared memory.
// Bound by memory: 8 bytes an element forward, about 10 backward.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act/format.h"
#include "act/launch.h"
#include "zero.h"

namespace zero {
namespace act {
namespace {

constexpr int kHeld = 2;  // chunks a thread holds

template <int W>
struct Shape {
  static constexpr int kLanes = 64 * W;                            // of a row
  static constexpr int kThreads = kLanes < 256 ? 256 : kLanes;     // of a workgroup
  static constexpr int kGroups = kThreads / kLanes;                // rows at a time
};

// Sums of N values over the row's lanes, in every lane, in a fixed order.  The
// two halves of `red` take turns, so one barrier a call is enough: whoever
// writes a half again has passed the barrier that followed its last reads.
template <int W, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* red, int& turn) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (W > 1) {
    constexpr int kWaves = Shape<W>::kThreads / 64;
    const int wave = threadIdx.x / 64;
    float* half = red + turn * (kWaves * N);
    turn ^= 1;
    if (threadIdx.x % 64 == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) half[wave * N + i] = v[i];
    }
    __syncthreads();
    const int first = wave / W * W;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < W; ++k) s += half[(first + k) * N + i];
      v[i] = s;
    }
  }
}

template <typename T>
__device__ __forceinline__ void row_of(const Rows& r, uint64_t c, uint32_t cols, float absent,
                                       float (&x)[8]) {
  if (r.p && c < cols) {
    unpack8<T>(load8(r.p, c, cols), x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = absent;
  }
}

template <typename T>
__device__ __forceinline__ void emit(const Ckpt& c, uint64_t row, uint32_t chunk, uint32_t cols,
                                     bool live, u32x4 w) {
  uint32_t scale;
  const u32x2 codes = c.format == kInt8 ? encode8<T, kInt8>(w, &scale)
                                        : encode8<T, kE4m3>(w, &scale);
  const uint32_t col = chunk * kChunk;
  if (!live || col >= cols) return;
  store_codes(c.codes + row * c.code_stride, col, cols, codes);
  if (chunk % kQuad == 0) c.scales[row * c.scale_stride + chunk / kQuad] = static_cast<uint8_t>(scale);
}

// (mean, 1 / deviation) of the row; columns beyond the row hold 0.
template <int W>
__device__ __forceinline__ void row_stats(const float (&x)[kHeld][8], int kind, float eps,
                                          uint32_t cols, float inv_n, uint32_t lane, float* red,
                                          int& turn, float* mean, float* rstd) {
  float m = 0.f;
  if (kind == ZERO_NORM_LAYER) {
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += x[j][i];
    row_sums<W>(s, red, turn);
    m = s[0] * inv_n;
  }
  float q[1] = {0.f};
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    const uint32_t col = (j * Shape<W>::kLanes + lane) * kChunk;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = col + i < cols ? x[j][i] - m : 0.f;
      q[0] += d * d;
    }
  }
  row_sums<W>(q, red, turn);
  *mean = m;
  *rstd = 1.0f / sqrtf(q[0] * inv_n + eps);
}

template <typename T, int W>
__global__ __launch_bounds__(Shape<W>::kThreads) void block_norm_kernel(BlockNormLaunch a) {
  using S = Shape<W>;
  __shared__ float red[2 * S::kThreads / 64];
  int turn = 0;
  const uint32_t lane = threadIdx.x % S::kLanes;
  const uint32_t group = threadIdx.x / S::kLanes;
  const float inv_n = 1.0f / static_cast<float>(a.cols);
  // every group of a workgroup makes the same number of turns, so the barriers
  // of row_sums meet; a group without a row computes on zeros and stores nothing
  for (uint64_t base = static_cast<uint64_t>(blockIdx.x) * S::kGroups; base < a.rows;
       base += static_cast<uint64_t>(gridDim.x) * S::kGroups) {
    const uint64_t row = base + group;
    const bool live = row < a.rows;
    float x[kHeld][8];   // h, then h'
    float b[kHeld][8];
    float st[4] = {0.f, 1.f, 0.f, 1.f};
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const uint32_t chunk = j * S::kLanes + lane;
      u32x4 wx = {0, 0, 0, 0}, wb = {0, 0, 0, 0};
      if (live && chunk * kChunk < a.cols) {
        wx = load8(a.res.p + row * a.res.stride, chunk * kChunk, a.cols);
        if (a.block.p)
          wb = load8(a.block.p + row * a.block.stride, chunk * kChunk, a.cols);
      }
      unpack8<T>(wx, x[j]);
      unpack8<T>(wb, b[j]);
      if (a.c_block.codes) emit<T>(a.c_block, row, chunk, a.cols, live, wb);
    }
    if (a.block.p) {
      if (a.post.kind != ZERO_NORM_NONE)
        row_stats<W>(b, a.post.kind, a.post.eps, a.cols, inv_n, lane, red, turn, &st[0], &st[1]);
#pragma unroll
      for (int j = 0; j < kHeld; ++j) {
        const uint32_t col = (j * S::kLanes + lane) * kChunk;
        float w[8], c[8], g[8];
        row_of<T>(a.post.w, col, a.cols, 1.f, w);
        row_of<T>(a.post.b, col, a.cols, 0.f, c);
        Rows gate = a.gate;
        if (gate.p && live) gate.p += row * gate.stride;
        row_of<T>(gate, col, a.cols, 1.f, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float o = (b[j][i] - st[0]) * st[1] * w[i] + c[i];
          x[j][i] = col + i < a.cols ? x[j][i] + a.scale * (g[i] * o) : 0.f;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const uint32_t chunk = j * S::kLanes + lane;
      const u32x4 w = pack8<T>(x[j]);
      if (a.out.p && live)
        store8(a.out.p + row * a.out.stride, chunk * kChunk, a.cols, w);
      if (a.c_out.codes) emit<T>(a.c_out, row, chunk, a.cols, live, w);
    }
    if (a.pre.kind != ZERO_NORM_NONE) {
      // from h' before its rounding to 16 bits: z is then rounded once
      row_stats<W>(x, a.pre.kind, a.pre.eps, a.cols, inv_n, lane, red, turn, &st[2], &st[3]);
#pragma unroll
      for (int j = 0; j < kHeld; ++j) {
        const uint32_t chunk = j * S::kLanes + lane;
        float w[8], c[8], z[8];
        row_of<T>(a.pre.w, chunk * kChunk, a.cols, 1.f, w);
        row_of<T>(a.pre.b, chunk * kChunk, a.cols, 0.f, c);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          z[i] = chunk * kChunk + i < a.cols ? (x[j][i] - st[2]) * st[3] * w[i] + c[i] : 0.f;
        const u32x4 wz = pack8<T>(z);
        if (live) store8(a.z.p + row * a.z.stride, chunk * kChunk, a.cols, wz);
        if (a.c_z.codes) emit<T>(a.c_z, row, chunk, a.cols, live, wz);
      }
    }
    if (live && lane == 0 && a.stats) {
      float* p = a.stats + row * 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = st[i];
    }
  }
}

// ------------------------------------------------------------ backward

// Row streams that keep partial sums of the parameter gradients, at most.
constexpr uint64_t kStreams = 512;

uint64_t padded(uint64_t cols) { return (cols + kChunk - 1) / kChunk * kChunk; }

// The gradient through one norm: q the gradient of the normalised value, xn that
// value, sums {sum q xn, sum q} over the row.
__device__ __forceinline__ float back(float q, float xn, float rstd, float mean_qx, float mean_q) {
  return rstd * (q - xn * mean_qx - mean_q);
}

// SETS: 2 -- the norms' weights; 3 -- and a gate per channel; 5 -- and biases.
template <typename T, int W, int SETS>
__global__ __launch_bounds__(Shape<W>::kThreads) void block_norm_grad_kernel(
    BlockNormGradLaunch a, uint64_t streams, uint64_t pad) {
  using S = Shape<W>;
  __shared__ float red[2 * 2 * S::kThreads / 64];
  int turn = 0;
  const uint32_t lane = threadIdx.x % S::kLanes;
  const uint32_t group = threadIdx.x / S::kLanes;
  const float inv_n = 1.0f / static_cast<float>(a.cols);
  const bool pre = a.pre.kind != ZERO_NORM_NONE;
  const bool block = a.block != 0;
  const float layer1 = a.pre.kind == ZERO_NORM_LAYER ? inv_n : 0.f;
  const float layer2 = a.post.kind == ZERO_NORM_LAYER ? inv_n : 0.f;
  float sum[SETS][kHeld][8];
#pragma unroll
  for (int s = 0; s < SETS; ++s)
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[s][j][i] = 0.f;

  for (uint64_t base = static_cast<uint64_t>(blockIdx.x) * S::kGroups; base < a.rows;
       base += static_cast<uint64_t>(gridDim.x) * S::kGroups) {
    const uint64_t row = base + group;
    const bool live = row < a.rows;
    float st[4] = {0.f, 1.f, 0.f, 1.f};
    if (live && a.stats) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(a.stats + row * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) st[i] = v[i];
    }
    float d[kHeld][8];   // dh', then the whole gradient of h'
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      u32x4 w = {0, 0, 0, 0};
      if (live && a.dout.p && (j * S::kLanes + lane) * kChunk < a.cols)
        w = load8(a.dout.p + row * a.dout.stride, (j * S::kLanes + lane) * kChunk, a.cols);
      unpack8<T>(w, d[j]);
    }
    if (pre) {
      float q[kHeld][8], xn[kHeld][8];
      float t[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < kHeld; ++j) {
        const uint32_t chunk = j * S::kLanes + lane, col = chunk * kChunk;
        u32x4 w = {0, 0, 0, 0};
        u32x2 c = {0, 0};
        uint32_t sb = 0;
        if (live && col < a.cols) {
          w = load8(a.dz.p + row * a.dz.stride, col, a.cols);
          c = load_codes(a.c_out.codes + row * a.c_out.code_stride, col, a.cols);
          sb = a.c_out.scales[row * a.c_out.scale_stride + chunk / kQuad];
        }
        unpack8<T>(w, q[j]);
        if (a.c_out.format == kInt8) decode8<kInt8>(c, scale_of(sb), xn[j]);
        else decode8<kE4m3>(c, scale_of(sb), xn[j]);
        float wt[8];
        row_of<T>(a.pre.w, col, a.cols, 1.f, wt);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool in = live && col + i < a.cols;
          xn[j][i] = in ? (xn[j][i] - st[2]) * st[3] : 0.f;
          sum[kDwPre][j][i] += q[j][i] * xn[j][i];
          if constexpr (SETS == 5) sum[kDbPre][j][i] += q[j][i];
          q[j][i] *= wt[i];
          t[0] += q[j][i] * xn[j][i];
          t[1] += q[j][i];
        }
      }
      row_sums<W>(t, red, turn);
#pragma unroll
      for (int j = 0; j < kHeld; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          d[j][i] += back(q[j][i], xn[j][i], st[3], t[0] * inv_n, t[1] * layer1);
    }
    if (a.dres.p && live) {
#pragma unroll
      for (int j = 0; j < kHeld; ++j)
        store8(a.dres.p + row * a.dres.stride, (j * S::kLanes + lane) * kChunk, a.cols, pack8<T>(d[j]));
    }
    if (block) {
      float v[kHeld][8], xn[kHeld][8];
      float t[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < kHeld; ++j) {
        const uint32_t chunk = j * S::kLanes + lane, col = chunk * kChunk;
        u32x2 c = {0, 0};
        uint32_t sb = 0;
        if (live && col < a.cols && a.c_block.codes) {
          c = load_codes(a.c_block.codes + row * a.c_block.code_stride, col, a.cols);
          sb = a.c_block.scales[row * a.c_block.scale_stride + chunk / kQuad];
        }
        if (a.c_block.format == kInt8) decode8<kInt8>(c, scale_of(sb), xn[j]);
        else decode8<kE4m3>(c, scale_of(sb), xn[j]);
        float wt[8], bt[8], g[8], dg[8];
        row_of<T>(a.post.w, col, a.cols, 1.f, wt);
        row_of<T>(a.post.b, col, a.cols, 0.f, bt);
        Rows gate = a.gate;
        if (gate.p && live) gate.p += row * gate.stride;
        row_of<T>(gate, col, a.cols, 1.f, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool in = live && col + i < a.cols;
          xn[j][i] = in ? (xn[j][i] - st[0]) * st[1] : 0.f;
          const float u = in ? a.scale * d[j][i] : 0.f;
          dg[i] = u * (xn[j][i] * wt[i] + bt[i]);
          const float p = u * g[i];
          if constexpr (SETS == 3) sum[2][j][i] += dg[i];
          if constexpr (SETS == 5) sum[kDgate][j][i] += dg[i];
          if constexpr (SETS == 5) sum[kDbPost][j][i] += p;
          sum[kDwPost][j][i] += p * xn[j][i];
          v[j][i] = p * wt[i];
          t[0] += v[j][i] * xn[j][i];
          t[1] += v[j][i];
        }
        if (a.dgate.p && live)
          store8(a.dgate.p + row * a.dgate.stride, col, a.cols, pack8<T>(dg));
      }
      if (a.dblock.p) {
        if (a.post.kind != ZERO_NORM_NONE) {
          row_sums<W>(t, red, turn);
#pragma unroll
          for (int j = 0; j < kHeld; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              v[j][i] = back(v[j][i], xn[j][i], st[1], t[0] * inv_n, t[1] * layer2);
        }
        if (live) {
#pragma unroll
          for (int j = 0; j < kHeld; ++j)
            store8(a.dblock.p + row * a.dblock.stride, (j * S::kLanes + lane) * kChunk, a.cols, pack8<T>(v[j]));
        }
      }
    }
  }
  if (!a.partial) return;
  const uint64_t stream = static_cast<uint64_t>(blockIdx.x) * S::kGroups + group;
#pragma unroll
  for (int s = 0; s < SETS; ++s)
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const uint64_t col = static_cast<uint64_t>(j * S::kLanes + lane) * kChunk;
      if (col >= pad) continue;
      float* p = a.partial + (static_cast<uint64_t>(s) * streams + stream) * pad + col;
      *reinterpret_cast<f32x4*>(p) =
          f32x4{sum[s][j][0], sum[s][j][1], sum[s][j][2], sum[s][j][3]};
      *reinterpret_cast<f32x4*>(p + 4) =
          f32x4{sum[s][j][4], sum[s][j][5], sum[s][j][6], sum[s][j][7]};
    }
}

// Joins the streams' partial sums in a fixed order: 64 columns a workgroup, 16
// waves each taking every 16th stream, then the 16 sums in turn.
struct JoinArgs {
  const float* partial;
  uint64_t streams, pad;
  uint32_t cols;
  int n;
  int set[kSums];
  void* out[kSums];
  int dtype, accumulate;
};

constexpr int kJoinWaves = 16;

__global__ __launch_bounds__(64 * kJoinWaves) void join_sums_kernel(JoinArgs a) {
  __shared__ float part[kJoinWaves][64];
  const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const uint32_t col = blockIdx.x * 64 + lane;
  const float* p = a.partial + static_cast<uint64_t>(a.set[blockIdx.y]) * a.streams * a.pad + col;
  float s = 0.f;
  if (col < a.cols)
    for (uint64_t k = wave; k < a.streams; k += kJoinWaves) s += p[k * a.pad];
  part[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || col >= a.cols) return;
#pragma unroll
  for (int k = 1; k < kJoinWaves; ++k) s += part[k][lane];
  void* out = a.out[blockIdx.y];
  if (a.dtype == kF32) {
    float* o = static_cast<float*>(out) + col;
    *o = a.accumulate ? *o + s : s;
  } else {
    uint16_t* o = static_cast<uint16_t*>(out) + col;
    if (a.dtype == kF16) {
      if (a.accumulate) s += lo16<F16>(*o);
      *o = static_cast<uint16_t>(pack16<F16>(s, 0.f));
    } else {
      if (a.accumulate) s += lo16<Bf16>(*o);
      *o = static_cast<uint16_t>(pack16<Bf16>(s, 0.f));
    }
  }
}

// Waves of a row: the least power of two whose threads hold it.
int waves_of(uint64_t cols) {
  int w = 1;
  while (static_cast<uint64_t>(w) * 64 * kHeld * kChunk < cols) w *= 2;
  return w;
}

uint64_t groups_of(int waves) { return waves < 4 ? 4 / waves : 1; }

constexpr uint64_t kForwardWgs = 2048;  // eight workgroups for each of 256 compute units

template <typename T>
void forward(const BlockNormLaunch& a, hipStream_t stream) {
  const int w = waves_of(a.cols);
  const uint64_t need = (a.rows + groups_of(w) - 1) / groups_of(w);
  const uint32_t wgs = static_cast<uint32_t>(need < kForwardWgs ? need : kForwardWgs);
  switch (w) {
    case 1: block_norm_kernel<T, 1><<<wgs, Shape<1>::kThreads, 0, stream>>>(a); break;
    case 2: block_norm_kernel<T, 2><<<wgs, Shape<2>::kThreads, 0, stream>>>(a); break;
    case 4: block_norm_kernel<T, 4><<<wgs, Shape<4>::kThreads, 0, stream>>>(a); break;
    case 8: block_norm_kernel<T, 8><<<wgs, Shape<8>::kThreads, 0, stream>>>(a); break;
    default: block_norm_kernel<T, 16><<<wgs, Shape<16>::kThreads, 0, stream>>>(a); break;
  }
}

template <typename T, int SETS>
void backward(const BlockNormGradLaunch& a, uint32_t wgs, uint64_t streams, hipStream_t stream) {
  const uint64_t pad = padded(a.cols);
  switch (waves_of(a.cols)) {
    case 1:
      block_norm_grad_kernel<T, 1, SETS><<<wgs, Shape<1>::kThreads, 0, stream>>>(a, streams, pad);
      break;
    case 2:
      block_norm_grad_kernel<T, 2, SETS><<<wgs, Shape<2>::kThreads, 0, stream>>>(a, streams, pad);
      break;
    case 4:
      block_norm_grad_kernel<T, 4, SETS><<<wgs, Shape<4>::kThreads, 0, stream>>>(a, streams, pad);
      break;
    case 8:
      block_norm_grad_kernel<T, 8, SETS><<<wgs, Shape<8>::kThreads, 0, stream>>>(a, streams, pad);
      break;
    default:
      block_norm_grad_kernel<T, 16, SETS><<<wgs, Shape<16>::kThreads, 0, stream>>>(a, streams,
                                                                                     pad);
      break;
  }
}

uint64_t grad_wgs(uint64_t rows, uint64_t cols) {
  const uint64_t g = groups_of(waves_of(cols)), need = (rows + g - 1) / g;
  const uint64_t most = kStreams / g;
  return need < most ? need : most;
}

}  // namespace

uint64_t norm_grad_workspace(uint64_t rows, uint64_t cols) {
  return grad_wgs(rows, cols) * groups_of(waves_of(cols)) * padded(cols) * kSums * sizeof(float);
}

hipError_t launch_block_norm(const BlockNormLaunch& a, hipStream_t stream) {
  if (a.dtype == kF16) forward<F16>(a, stream);
  else forward<Bf16>(a, stream);
  return hipGetLastError();
}

hipError_t launch_block_norm_grad(const BlockNormGradLaunch& in, hipStream_t stream) {
  BlockNormGradLaunch a = in;
  bool any = false;
  for (void* p : a.sums) any = any || p != nullptr;
  if (!any) a.partial = nullptr;
  const uint32_t wgs = static_cast<uint32_t>(grad_wgs(a.rows, a.cols));
  const uint64_t streams = wgs * groups_of(waves_of(a.cols));
  const int sets = a.sums[kDbPre] || a.sums[kDbPost] ? 5 : a.sums[kDgate] ? 3 : 2;
  if (wgs) {
    if (a.dtype == kF16) {
      if (sets == 2) backward<F16, 2>(a, wgs, streams, stream);
      else if (sets == 3) backward<F16, 3>(a, wgs, streams, stream);
      else backward<F16, 5>(a, wgs, streams, stream);
    } else {
      if (sets == 2) backward<Bf16, 2>(a, wgs, streams, stream);
      else if (sets == 3) backward<Bf16, 3>(a, wgs, streams, stream);
      else backward<Bf16, 5>(a, wgs, streams, stream);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!any) return hipSuccess;
  JoinArgs j;
  j.partial = a.partial;
  j.streams = streams;
  j.pad = padded(a.cols);
  j.cols = a.cols;
  j.dtype = a.grad_dtype;
  j.accumulate = a.accumulate;
  j.n = 0;
  for (int s = 0; s < kSums; ++s) {
    if (!a.sums[s]) continue;
    j.set[j.n] = s == kDgate && sets == 3 ? 2 : s;
    j.out[j.n++] = a.sums[s];
  }
  join_sums_kernel<<<dim3((a.cols + 63) / 64, j.n), 64 * kJoinWaves, 0, stream>>>(j);
  return hipGetLastError();
}

}  // namespace act
}  // namespace zero
