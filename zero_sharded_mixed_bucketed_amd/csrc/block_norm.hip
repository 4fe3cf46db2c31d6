// The norms before and after a block, fused with the block's gate and residual
// scale: per token, in fp32,
//   o  = post(b);  h' = h + s * (g . o);  z = pre(h')
// with post and pre an RMS or layer norm (or none), and their backward from the
// 8-bit checkpoints of b and h'.
//
// One workgroup holds a row from the first load to the last store: each input is
// read once and each output written once, but for the backward of rows over 8192
// columns, which reads its inputs again for the parameters' gradients (and a third
// time where outputs replace them).  A thread holds chunks of eight columns; row sums
// go through lane exchanges and, where a row has several waves, shared memory.  Bound
// by memory at whole widths from 4096 columns on (8 bytes an element forward, about
// 10 backward); elsewhere by empty lanes, registers and latency, as noted below.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "act/format.h"
#include "act/launch.h"
#include "zero.h"

namespace zero {
namespace act {
namespace {

// Sums of N values over the workgroup's `waves` waves, in every lane, in a fixed
// order.  The two halves of `red` take turns, so one barrier a call is enough:
// whoever writes a half again has passed the barrier that followed its last reads.
template <int MAX_WAVES, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* red, int& turn, int waves) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (MAX_WAVES > 1) {
    if (waves == 1) return;
    float* half = red + turn * (MAX_WAVES * N);
    turn ^= 1;
    if (threadIdx.x % 64 == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) half[threadIdx.x / 64 * N + i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = half[i];
    for (int k = 1; k < waves; ++k)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += half[k * N + i];
  }
}

template <typename T>
__device__ __forceinline__ void emit(const Ckpt& c, uint64_t row, uint32_t chunk, uint32_t cols,
                                     u32x4 w) {
  uint32_t scale;
  const u32x2 codes = c.format == kInt8 ? encode8<T, kInt8>(w, &scale)
                                        : encode8<T, kE4m3>(w, &scale);
  const uint32_t col = chunk * kChunk;
  if (col >= cols) return;
  store_codes(c.codes + row * c.code_stride, col, cols, codes);
  if (chunk % kQuad == 0)
    c.scales[row * c.scale_stride + chunk / kQuad] = static_cast<uint8_t>(scale);
}

// ------------------------------------------------------------ forward

// Up to eight chunks a thread: rows of up to 4096 columns take one wave, and its
// sums no barrier.  Nothing is kept from row to row; many rows at once on a compute
// unit hide the loads, and the norms' weights come from the caches.  16384 x 4096
// bf16 with a gate a channel takes 97-100 us with RMS norms, 5.4-5.5 TB/s (143 us, 5.2
// TB/s with all three checkpoints), and 103 with layer norms.  As many elements in rows
// of 2560 columns take 118 and 135 us (a sixth of the lanes hold nothing), of 5000 108
// and 118, of 8191 156 and 174 (every lane shifts its last chunk, and eight chunks a
// thread spill in rows that are not whole), of 16384 97 and 102.
template <typename T, int WAVES, int HELD, bool FULL>
__global__ __launch_bounds__(64 * WAVES, HELD > 5 ? 3 : 4) void block_norm_kernel(
    BlockNormLaunch a, uint64_t row0) {
  constexpr uint32_t kLanes = 64 * WAVES;
  // short rows that end inside a line share it, and meet in the caches
  constexpr bool kStream = FULL || WAVES * HELD > 1;
  __shared__ float red[2 * WAVES];
  int turn = 0;
  const uint64_t row = row0 + blockIdx.x;
  const uint32_t lane = threadIdx.x, cols = a.cols;
  const float inv_n = 1.0f / static_cast<float>(cols);
  const uint16_t* res = a.res.p + row * a.res.stride;
  const uint16_t* block = a.block.p + row * a.block.stride;
  const uint16_t* gate = a.gate.p + row * a.gate.stride;
  const bool has_block = a.block.p != nullptr;

  u32x4 wx[HELD], wb[HELD];
#pragma unroll
  for (int j = 0; j < HELD; ++j) {
    const uint32_t c = (j * kLanes + lane) * kChunk;
    wx[j] = stream8_early<FULL, kStream>(res, c, cols);
    wb[j] = u32x4{0, 0, 0, 0};
    if (has_block) wb[j] = stream8_early<FULL, kStream>(block, c, cols);
  }
#pragma unroll
  for (int j = 0; j < HELD; ++j) {
    const uint32_t c = (j * kLanes + lane) * kChunk;
    mend8<FULL>(wx[j], res, c, cols);
    if (has_block) mend8<FULL>(wb[j], block, c, cols);
  }

  // (mean, 1 / deviation) from values of the row; columns beyond it hold 0
  auto stats = [&](auto value, int kind, float eps, float* mean, float* rstd) {
    float m = 0.f;
    if (kind == ZERO_NORM_LAYER) {
      float s[1] = {0.f};
#pragma unroll
      for (int j = 0; j < HELD; ++j) {
        float x[8];
        value(j, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] += x[i];
      }
      row_sums<WAVES>(s, red, turn, WAVES);
      m = s[0] * inv_n;
    }
    float q[1] = {0.f};
#pragma unroll
    for (int j = 0; j < HELD; ++j) {
      const uint32_t c = (j * kLanes + lane) * kChunk;
      float x[8];
      value(j, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = FULL || c + i < cols ? x[i] - m : 0.f;
        q[0] += d * d;
      }
    }
    row_sums<WAVES>(q, red, turn, WAVES);
    *mean = m;
    *rstd = 1.0f / sqrtf(q[0] * inv_n + eps);
  };
  auto row_of = [&](const uint16_t* p, uint32_t c, float absent, float (&x)[8]) {
    if (p) {
      unpack8<T>(load8_row<FULL>(p, c, cols), x);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = absent;
    }
  };

  float m2 = 0.f, r2 = 1.f, m1 = 0.f, r1 = 1.f;
  if (a.post.kind != ZERO_NORM_NONE)
    stats([&](int j, float (&x)[8]) {
      forget(wb[j]);
      unpack8<T>(wb[j], x);
    }, a.post.kind, a.post.eps, &m2, &r2);
  if (a.c_block.codes) {
#pragma unroll
    for (int j = 0; j < HELD; ++j) emit<T>(a.c_block, row, j * kLanes + lane, cols, wb[j]);
  }
  float x[HELD][8];   // h'
#pragma unroll
  for (int j = 0; j < HELD; ++j) {
    forget(wb[j]);
    unpack8<T>(wx[j], x[j]);
    if (!has_block) continue;
    const uint32_t c = (j * kLanes + lane) * kChunk;
    float b[8], w[8], bias[8], g[8];
    unpack8<T>(wb[j], b);
    row_of(a.post.w.p, c, 1.f, w);
    row_of(a.post.b.p, c, 0.f, bias);
    row_of(a.gate.p ? gate : nullptr, c, 1.f, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float o = (b[i] - m2) * r2 * w[i] + bias[i];
      x[j][i] = FULL || c + i < cols ? x[j][i] + a.scale * (g[i] * o) : 0.f;
    }
  }
  if (a.out.p) {
#pragma unroll
    for (int j = 0; j < HELD; ++j)
      store8_row<FULL, kStream>(a.out.p + row * a.out.stride, (j * kLanes + lane) * kChunk, cols,
                       pack8<T>(x[j]));
  }
  if (a.c_out.codes) {
#pragma unroll
    for (int j = 0; j < HELD; ++j)
      emit<T>(a.c_out, row, j * kLanes + lane, cols, pack8<T>(x[j]));
  }
  if (a.pre.kind != ZERO_NORM_NONE) {
    // from h' before its rounding to 16 bits: z is then rounded once
    stats([&](int j, float (&v)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = x[j][i];
    }, a.pre.kind, a.pre.eps, &m1, &r1);
#pragma unroll
    for (int j = 0; j < HELD; ++j) {
      const uint32_t c = (j * kLanes + lane) * kChunk;
      float w[8], bias[8];
      row_of(a.pre.w.p, c, 1.f, w);
      row_of(a.pre.b.p, c, 0.f, bias);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[j][i] = FULL || c + i < cols ? (x[j][i] - m1) * r1 * w[i] + bias[i] : 0.f;
      store8_row<FULL, kStream>(a.z.p + row * a.z.stride, c, cols, pack8<T>(x[j]));
    }
    if (a.c_z.codes) {
#pragma unroll
      for (int j = 0; j < HELD; ++j)
        emit<T>(a.c_z, row, j * kLanes + lane, cols, pack8<T>(x[j]));
    }
  }
  if (lane == 0 && a.stats)
    *reinterpret_cast<f32x4*>(a.stats + row * 4) = f32x4{m2, r2, m1, r1};
}

// ------------------------------------------------------------ backward

uint64_t padded(uint64_t cols) { return (cols + kChunk - 1) / kChunk * kChunk; }

// Chunks a thread holds, and waves of a row (at most 8, or 12 of one chunk).  One
// chunk a thread leaves room for 12 waves on a compute unit, against 8 of two chunks,
// and wastes less of a row's last wave; two leave each wave more loads in flight.
// Measured with 16384 x 4096 elements and a gate a channel, one chunk (two):
//   RMS norms, bf16:   768 columns 195 (191) us, 1100: 197 (297), 1900: 160 (191),
//     2304: 229 (222), 2560: 174 (193), 2900: 268 (223), 4096: 149 (144), 5000: 164 (206),
//     5120: 146 (151)
//   layer norms, fp16: 1100 columns 600 (336) us, 2560: 256 (238), 4096: 188 (151),
//     4608: 199 (260), 5000: 300 (252), 5120: 190 (208); their rows that end inside a
//     wave run out of registers with one chunk
// Rows of up to 512 columns are one wave's, so short ones leave lanes empty, and layer
// norms' spill there too (48-58 registers): as many elements in rows of 72 columns take
// 678 us (RMS) and 993 (layer norms), of 200 266 and 385, of 300 231 and 316.
int grad_held(uint64_t cols, int sets) {
  const bool whole = cols % (64 * kChunk) == 0;
  if (cols > 8192) return 4;
  if (cols <= 512) return 1;
  if (cols >= 4096) return cols > 4096 && cols <= 6144 && (sets == 3 || whole) ? 1 : 2;
  return sets == 3 && cols > 1024 && (whole || cols <= 2048) ? 1 : 2;
}

int grad_waves(uint64_t cols, int sets) {
  const uint64_t per = 64 * grad_held(cols, sets) * kChunk;
  return static_cast<int>((cols + per - 1) / per);
}

bool wide_rows(uint64_t cols) { return cols > 8192; }

// Rows that are worked on at once, at most: what 256 compute units hold, with eight
// waves each, or 12 of one chunk a thread (a workgroup more would wait for the
// others' last rows).
uint64_t grad_wgs(uint64_t rows, uint64_t cols, int sets) {
  const uint64_t most =
      256 * ((grad_held(cols, sets) == 1 ? 12 : 8) / grad_waves(cols, sets));
  return rows < most ? rows : most;
}

// Partial sums of each column of the parameters' gradients: one of each row that is
// worked on, or of 128 stretches of wide rows.
uint64_t grad_streams(uint64_t rows, uint64_t cols, int sets) {
  if (!wide_rows(cols)) return grad_wgs(rows, cols, sets);
  return rows < 128 ? rows : 128;
}

// Everything of a row that a thread loads.
template <int HELD, bool FULL>
struct GradRow {
  static constexpr bool kStream = FULL || HELD > 1;   // as in block_norm_kernel

  u32x4 d[HELD], z[HELD], g[HELD];
  u32x2 out[HELD], block[HELD];
  uint32_t s_out[HELD], s_block[HELD];
  f32x4 st;

  __device__ __forceinline__ void clear() {   // what is absent stays 0
#pragma unroll
    for (int j = 0; j < HELD; ++j) {
      d[j] = z[j] = g[j] = u32x4{0, 0, 0, 0};
      out[j] = block[j] = u32x2{0, 0};
      s_out[j] = s_block[j] = 0;
    }
  }

  __device__ __forceinline__ void load(const BlockNormGradLaunch& a, uint64_t row, uint32_t lanes,
                                       bool token_gate) {
    const uint16_t* pd = a.dout.p + row * a.dout.stride;
    const uint16_t* pz = a.dz.p + row * a.dz.stride;
    const uint16_t* pg = a.gate.p + row * a.gate.stride;
    const uint8_t* po = a.c_out.codes + row * a.c_out.code_stride;
    const uint8_t* pb = a.c_block.codes + row * a.c_block.code_stride;
    const uint8_t* so = a.c_out.scales + row * a.c_out.scale_stride;
    const uint8_t* sb = a.c_block.scales + row * a.c_block.scale_stride;
    st = f32x4{0.f, 1.f, 0.f, 1.f};
    if (a.stats) st = *reinterpret_cast<const f32x4*>(a.stats + row * 4);
#pragma unroll
    for (int j = 0; j < HELD; ++j) {
      const uint32_t chunk = j * lanes + threadIdx.x, c = chunk * kChunk;
      const uint32_t b = FULL || c < a.cols ? chunk / kQuad : 0;
      if (a.dout.p) d[j] = stream8_early<FULL, kStream>(pd, c, a.cols);
      if (a.c_out.codes) {
        z[j] = stream8_early<FULL, kStream>(pz, c, a.cols);
        out[j] = stream_codes_early<FULL, kStream>(po, c, a.cols);
        s_out[j] = so[b];
      }
      if (a.c_block.codes) {
        block[j] = stream_codes_early<FULL, kStream>(pb, c, a.cols);
        s_block[j] = sb[b];
      }
      if (token_gate) g[j] = stream8_early<FULL, kStream>(pg, c, a.cols);
    }
  }

  // Where the loads are waited for.
  __device__ __forceinline__ void settle(const BlockNormGradLaunch& a, uint64_t row,
                                         uint32_t lanes, bool token_gate) {
    forget(st);
#pragma unroll
    for (int j = 0; j < HELD; ++j) {
      forget(d[j]);
      forget(z[j]);
      forget(out[j]);
      forget(block[j]);
      forget(s_out[j]);
      forget(s_block[j]);
      if (token_gate) forget(g[j]);
      if constexpr (!FULL) {
        const uint32_t c = (j * lanes + threadIdx.x) * kChunk, cols = a.cols;
        if (c + kChunk <= cols) continue;
        if (a.dout.p) mend8<FULL>(d[j], a.dout.p + row * a.dout.stride, c, cols);
        if (a.c_out.codes) {
          mend8<FULL>(z[j], a.dz.p + row * a.dz.stride, c, cols);
          mend_codes<FULL>(out[j], a.c_out.codes + row * a.c_out.code_stride, c, cols);
        }
        if (a.c_block.codes)
          mend_codes<FULL>(block[j], a.c_block.codes + row * a.c_block.code_stride, c, cols);
        if (token_gate) mend8<FULL>(g[j], a.gate.p + row * a.gate.stride, c, cols);
      }
    }
  }
};

// Threads of a workgroup, at most, and waves on each of a compute unit's four units.
constexpr int grad_threads(int held, int sets, bool full) {
  return 64 * (held > 1 ? 8 : sets == 3 || full ? 12 : 1);
}
template <typename T>
constexpr bool rows_shared(int sets) { return sets == 5 && T::kType == kBf16; }
constexpr int grad_fit(int held) { return held == 1 ? 3 : 2; }

// One workgroup takes rows blockIdx.x, blockIdx.x + gridDim.x, ..., loading one
// while it works on the one before, and keeps the parameters' gradients of its rows
// in registers; SETS: 3 -- those of the weights and of a gate a channel; 5 -- and of
// biases; 0 -- none.  Two chunks a thread leave room for that.
//
// Both norms' row sums are taken together, behind one barrier.  The gradient of
// post's input needs sums of v = y D and v x2 (y = s g w_post), where
//   D = e - r1 a x1 - r1 m,  e = dout + r1 q,  a = mean(q x1),  m = [mean q]
// is known only after pre's; but it is linear in a and m, so sums of y e, y x1, y
// and their products with x2 give it afterwards.
//
// Up to 8192 columns a thread holds one chunk or two (grad_held), and the values of
// the first half stay in registers for the second.  The biases' sums lie in shared
// memory, each thread's in places of its own: with them in registers the kernel ran
// out and took 2.5 times as long.  In bf16, whose values take a register each once
// unpacked (fp16 ones are read by the multiply-adds as they are), the norms' rows
// lie there too: layer norms over 4000 columns take 174 us instead of 271, over
// 4096 154 instead of 186, where fp16 takes 175 and 152 without and 176 and 155
// with.  16384 x 4096 bf16 with RMS norms and a gate a channel takes 128 us and its
// join 5, 5.1 TB/s.  Wider rows (SETS == 0) take four chunks, load nothing ahead,
// read the norms' weights from the caches, make those values again, and leave the
// parameters' gradients to norm_sums_kernel, with mean(q x1) and [mean q] of each
// row: kept here too, 4096 x 16384 took 520 us (RMS) and 850 (layer norms) where it
// now takes 328 and 337 (its bytes alone: 102).  Rows that are not whole cost more:
// 7455 x 9001 takes 566 and 583.
template <typename T, int FMT, int HELD, int SETS, bool FULL>
__global__ __launch_bounds__(grad_threads(HELD, SETS, FULL), grad_fit(HELD)) void
block_norm_grad_kernel(BlockNormGradLaunch a, uint64_t pad) {
  constexpr bool kAhead = HELD <= 2, kKeep = kAhead;
  constexpr int kMaxWaves = grad_threads(HELD, SETS, FULL) / 64;
  constexpr int kRowSums = 8;
  __shared__ float red[2 * kMaxWaves * kRowSums];
  int turn = 0;
  const uint32_t lanes = blockDim.x, waves = lanes / 64, cols = a.cols;
  const float inv_n = 1.0f / static_cast<float>(cols);
  const bool pre = a.c_out.codes != nullptr;
  const bool post = a.post.kind != ZERO_NORM_NONE;
  // Without post's norm the gradient of b has no part along x2, and 0 times what b
  // holds would be NaN for an infinity or NaN; as a mask it costs nothing that
  // shows, as a branch the kernel ran out of registers (250 -> 387 us).
  const uint32_t of_post = post ? ~0u : 0u;
  const bool layer1 = a.pre.kind == ZERO_NORM_LAYER, layer2 = a.post.kind == ZERO_NORM_LAYER;
  const bool token_gate = a.gate.p && a.gate.stride != 0;
  // The norms' rows, the same for every token; 1 where absent.  Columns past the
  // row's end need no further care: dout, dz and w_post are 0 there, which keeps them
  // out of the row sums, and nothing is stored there.
  constexpr uint32_t kOne = T::kType == kF16 ? 0x3C00u : 0x3F80u;
  u32x4 w1[HELD], w2[HELD], b2[HELD], gc[HELD];
  auto load_rows = [&](int j) {
    uint32_t c = (j * lanes + threadIdx.x) * kChunk;
    if constexpr (!kAhead) forget(c);   // a load each time, not registers in between
    u32x4 ones;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      ones[i] = (FULL || c + 2 * i < cols ? kOne : 0u) |
                (FULL || c + 2 * i + 1 < cols ? kOne : 0u) << 16;
    w1[j] = w2[j] = gc[j] = ones;
    b2[j] = u32x4{0, 0, 0, 0};
    if (a.pre.w.p) w1[j] = load8_row<FULL>(a.pre.w.p, c, cols);
    if (a.post.w.p) w2[j] = load8_row<FULL>(a.post.w.p, c, cols);
    if (a.post.b.p) b2[j] = load8_row<FULL>(a.post.b.p, c, cols);
    if (a.gate.p && !token_gate) gc[j] = load8_row<FULL>(a.gate.p, c, cols);
  };
  // SETS == 5: 4 HELD vectors of sums of each thread, and kShared: as many of the rows
  extern __shared__ f32x4 shared[];
  constexpr bool kShared = rows_shared<T>(SETS);
  auto row_at = [&](int which, int j, uint32_t thread) -> u32x4& {
    return reinterpret_cast<u32x4*>(shared)[(4 * HELD + which * HELD + j) * lanes + thread];
  };
  if constexpr (kAhead) {
#pragma unroll
    for (int j = 0; j < HELD; ++j) {
      load_rows(j);
      if constexpr (kShared) {
        row_at(0, j, threadIdx.x) = w1[j];
        row_at(1, j, threadIdx.x) = w2[j];
        row_at(2, j, threadIdx.x) = b2[j];
        row_at(3, j, threadIdx.x) = gc[j];
      }
    }
  }
  auto fetch_rows = [&](int j) {   // what is not used of them is not read
    uint32_t thread = threadIdx.x;
    forget(thread);
    w1[j] = row_at(0, j, thread);
    w2[j] = row_at(1, j, thread);
    b2[j] = row_at(2, j, thread);
    gc[j] = row_at(3, j, thread);
  };
  float sum[3][SETS ? HELD : 1][8];   // of the weights and the gate
  constexpr int kGate = 2;
  if constexpr (SETS > 0) {
#pragma unroll
    for (int s = 0; s < 3; ++s)
#pragma unroll
      for (int j = 0; j < HELD; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[s][j][i] = 0.f;
  }
  auto bias_at = [&](int set, int j, int half) -> f32x4& {
    return shared[((set * HELD + j) * 2 + half) * lanes + threadIdx.x];
  };
  if constexpr (SETS == 5) {
#pragma unroll
    for (int q = 0; q < 4 * HELD; ++q)
      bias_at(q / (2 * HELD), q / 2 % HELD, q % 2) = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  auto add_bias = [&](int set, int j, const float (&v)[8]) {
    if constexpr (SETS == 5) {
      bias_at(set, j, 0) += f32x4{v[0], v[1], v[2], v[3]};
      bias_at(set, j, 1) += f32x4{v[4], v[5], v[6], v[7]};
    }
  };

  GradRow<HELD, FULL> next;
  next.clear();
  uint64_t row = blockIdx.x;
  if (kAhead && row < a.rows) next.load(a, row, lanes, token_gate);
  for (; row < a.rows; row += gridDim.x) {
    GradRow<HELD, FULL> r;
    if constexpr (kAhead) {
      r = next;
#pragma unroll
      for (int j = 0; j < HELD; ++j) {
        if constexpr (kShared) continue;
        forget(w1[j]);
        forget(w2[j]);
        forget(b2[j]);
        forget(gc[j]);
      }
    } else {
      r.clear();
      r.load(a, row, lanes, token_gate);
    }
    r.settle(a, row, lanes, token_gate);
    if (kAhead && row + gridDim.x < a.rows) next.load(a, row + gridDim.x, lanes, token_gate);
    const float m2 = r.st[0], r2 = r.st[1], m1 = r.st[2], r1 = r.st[3];

    float x1[HELD][8], x2[HELD][8], e[HELD][8];
    // x1, x2, e and the gradient z of the normalised pre value's input
    auto front = [&](int j, float (&z)[8], float (&q)[8]) {
      float k[8], w[8], d[8];
      unpack8<T>(r.z[j], z);
      unpack8<T>(w1[j], w);
      unpack8<T>(r.d[j], d);
      decode8<FMT>(r.out[j], scale_of(r.s_out[j]), k);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x1[j][i] = (k[i] - m1) * r1;
        q[i] = z[i] * w[i];
        e[j][i] = d[i] + r1 * q[i];
      }
      decode8<FMT>(r.block[j], scale_of(r.s_block[j]), k);
#pragma unroll
      for (int i = 0; i < 8; ++i) x2[j][i] = (k[i] - m2) * r2;
    };
    auto gates = [&](int j, float (&g)[8]) { unpack8<T>(token_gate ? r.g[j] : gc[j], g); };

    // sums: q x1, q; y e x2, y x1 x2, y x2; y e, y x1, y
    float t[kRowSums];
#pragma unroll
    for (int i = 0; i < kRowSums; ++i) t[i] = 0.f;
#pragma unroll
    for (int j = 0; j < HELD; ++j) {
      float z[8], q[8], g[8], w[8];
      if constexpr (!kAhead) load_rows(j);
      if constexpr (kShared) fetch_rows(j);
      front(j, z, q);
      gates(j, g);
      unpack8<T>(w2[j], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (SETS > 0) sum[kDwPre][j][i] += z[i] * x1[j][i];
        t[0] += q[i] * x1[j][i];
        const float y = a.scale * g[i] * w[i], yx = y * x2[j][i];
        t[2] += yx * e[j][i];
        t[3] += yx * x1[j][i];
        if constexpr (SETS != 3) {
          t[1] += q[i];
          t[4] += yx;
          t[5] += y * e[j][i];
          t[6] += y * x1[j][i];
          t[7] += y;
        }
      }
      add_bias(0, j, z);
      // one chunk at a time: side by side they need more registers than there are
      if constexpr (HELD > 2) __builtin_amdgcn_sched_barrier(0);
    }
    float mean_qx, mean_q = 0.f, mean_vx, mean_v = 0.f;
    if constexpr (SETS != 3) {
      row_sums<kMaxWaves>(t, red, turn, waves);
      mean_qx = t[0] * inv_n;
      mean_q = layer1 ? t[1] * inv_n : 0.f;
      mean_vx = (t[2] - r1 * (mean_qx * t[3] + mean_q * t[4])) * inv_n;
      mean_v = (t[5] - r1 * (mean_qx * t[6] + mean_q * t[7])) * inv_n;
    } else {
      float u[3] = {t[0], t[2], t[3]};
      row_sums<kMaxWaves>(u, red, turn, waves);
      mean_qx = u[0] * inv_n;
      mean_vx = (u[1] - r1 * mean_qx * u[2]) * inv_n;
    }
    if (!pre) mean_qx = mean_q = 0.f;
    if (!post) mean_vx = 0.f;
    if (!layer2) mean_v = 0.f;
    if (SETS == 0 && a.means && threadIdx.x == 0) {
      a.means[2 * row] = mean_qx;
      a.means[2 * row + 1] = mean_q;
    }

#pragma unroll
    for (int j = 0; j < HELD; ++j) {
      const uint32_t c = (j * lanes + threadIdx.x) * kChunk;
      if constexpr (kShared) fetch_rows(j);
      forget(w2[j]);
      forget(gc[j]);
      forget(r.g[j]);
      if constexpr (!kKeep) {
        forget(r.z[j]);
        forget(r.d[j]);
        forget(r.out[j]);
        forget(r.block[j]);
        forget(w1[j]);
        if constexpr (!kAhead) load_rows(j);
        float z[8], q[8];
        front(j, z, q);
      }
      float d[8], dg[8], db[8], p[8], g[8], w[8], bias[8];
      gates(j, g);
      unpack8<T>(w2[j], w);
      unpack8<T>(b2[j], bias);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        d[i] = e[j][i] - r1 * (x1[j][i] * mean_qx + mean_q);
        const float u = a.scale * d[i];
        p[i] = u * g[i];
        dg[i] = u * (x2[j][i] * w[i] + bias[i]);
        if constexpr (SETS > 0) {
          sum[kGate][j][i] += dg[i];
          sum[kDwPost][j][i] += p[i] * x2[j][i];
        }
        const float along = __builtin_bit_cast(
            float, __builtin_bit_cast(uint32_t, x2[j][i]) & of_post);
        db[i] = r2 * (p[i] * w[i] - along * mean_vx - mean_v);
      }
      add_bias(1, j, p);
      constexpr bool kStream = GradRow<HELD, FULL>::kStream;
      if (a.dres.p)
        store8_row<FULL, kStream>(a.dres.p + row * a.dres.stride, c, cols, pack8<T>(d));
      if (a.dblock.p)
        store8_row<FULL, kStream>(a.dblock.p + row * a.dblock.stride, c, cols, pack8<T>(db));
      if (a.dgate.p)
        store8_row<FULL, kStream>(a.dgate.p + row * a.dgate.stride, c, cols, pack8<T>(dg));
      if constexpr (HELD > 2) __builtin_amdgcn_sched_barrier(0);
    }
  }
  if constexpr (SETS == 0) return;
  if (!a.partial) return;
  constexpr int kSetOf[kSums] = {kDwPre, kDwPost, kDgate, kDbPre, kDbPost};
#pragma unroll
  for (int s = 0; s < SETS; ++s) {
    if (!a.sums[kSetOf[s]]) continue;
#pragma unroll
    for (int j = 0; j < HELD; ++j) {
      const uint64_t col = static_cast<uint64_t>(j * lanes + threadIdx.x) * kChunk;
      if (col >= pad) continue;
      f32x4 u, v;
      if (s < 3) {
        const float (&x)[8] = sum[s < 3 ? s : 0][SETS ? j : 0];
        u = f32x4{x[0], x[1], x[2], x[3]};
        v = f32x4{x[4], x[5], x[6], x[7]};
      } else {
        u = bias_at(s - 3, j, 0);
        v = bias_at(s - 3, j, 1);
      }
      float* p = a.partial +
                 (static_cast<uint64_t>(kSetOf[s]) * gridDim.x + blockIdx.x) * pad + col;
      *reinterpret_cast<f32x4*>(p) = u;
      *reinterpret_cast<f32x4*>(p + 4) = v;
    }
  }
}

// The parameters' gradients of wide rows, from the same inputs and each row's means:
// a thread keeps the sums of eight columns over every gridDim.y-th row, so that
// nothing passes between threads.  Those sums, the norms' rows and two rows in hand
// are more than the registers of three waves a unit: 118-122 spill.
constexpr int kSumThreads = 256;
constexpr uint32_t kSumCols = kSumThreads * kChunk;

template <typename T, int FMT>
__global__ __launch_bounds__(kSumThreads, 3) void norm_sums_kernel(BlockNormGradLaunch a,
                                                                uint64_t pad) {
  const uint32_t c = (blockIdx.x * kSumThreads + threadIdx.x) * kChunk, cols = a.cols;
  const bool token_gate = a.gate.p && a.gate.stride != 0;
  const bool pre = a.c_out.codes != nullptr, block = a.c_block.codes != nullptr;
  constexpr uint32_t kOne = T::kType == kF16 ? 0x3C003C00u : 0x3F803F80u;
  const u32x4 ones = {kOne, kOne, kOne, kOne};
  if (c >= cols) return;
  float w1[8], w2[8], b2[8], gc[8];
  unpack8<T>(a.pre.w.p ? load8(a.pre.w.p, c, cols) : ones, w1);
  unpack8<T>(a.post.w.p ? load8(a.post.w.p, c, cols) : ones, w2);
  unpack8<T>(a.post.b.p ? load8(a.post.b.p, c, cols) : u32x4{0, 0, 0, 0}, b2);
  unpack8<T>(a.gate.p && !token_gate ? load8(a.gate.p, c, cols) : ones, gc);
  float sum[kSums][8];
#pragma unroll
  for (int s = 0; s < kSums; ++s)
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[s][i] = 0.f;
  const uint32_t scale_at = c / kBlock;
#pragma unroll 2
  for (uint64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const uint16_t* pd = a.dout.p + row * a.dout.stride;
    const uint16_t* pz = a.dz.p + row * a.dz.stride;
    const uint16_t* pg = a.gate.p + row * a.gate.stride;
    const uint8_t* po = a.c_out.codes + row * a.c_out.code_stride;
    const uint8_t* pb = a.c_block.codes + row * a.c_block.code_stride;
    u32x4 wd = {0, 0, 0, 0}, wz = wd, wg = wd;
    u32x2 wo = {0, 0}, wb = wo;
    uint32_t so = 0, sb = 0;
    if (a.dout.p) wd = stream8_early<false>(pd, c, cols);
    if (pre) {
      wz = stream8_early<false>(pz, c, cols);
      wo = stream_codes_early<false>(po, c, cols);
      so = a.c_out.scales[row * a.c_out.scale_stride + scale_at];
    }
    if (block) {
      wb = stream_codes_early<false>(pb, c, cols);
      sb = a.c_block.scales[row * a.c_block.scale_stride + scale_at];
    }
    if (token_gate) wg = stream8_early<false>(pg, c, cols);
    const f32x4 st = a.stats ? *reinterpret_cast<const f32x4*>(a.stats + row * 4)
                             : f32x4{0.f, 1.f, 0.f, 1.f};
    const float mean_qx = a.means[2 * row], mean_q = a.means[2 * row + 1];
    if (c + kChunk > cols) {
      if (a.dout.p) mend8<false>(wd, pd, c, cols);
      if (pre) {
        mend8<false>(wz, pz, c, cols);
        mend_codes<false>(wo, po, c, cols);
      }
      if (block) mend_codes<false>(wb, pb, c, cols);
      if (token_gate) mend8<false>(wg, pg, c, cols);
    }
    float d[8], z[8], g[8], x1[8], x2[8];
    unpack8<T>(wd, d);
    unpack8<T>(wz, z);
    unpack8<T>(wg, g);
    decode8<FMT>(wo, scale_of(so), x1);
    decode8<FMT>(wb, scale_of(sb), x2);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float n1 = (x1[i] - st[2]) * st[3], n2 = (x2[i] - st[0]) * st[1];
      const float e = d[i] + st[3] * (z[i] * w1[i]);
      const float u = a.scale * (e - st[3] * (n1 * mean_qx + mean_q));
      const float p = u * (token_gate ? g[i] : gc[i]);
      sum[kDwPre][i] += z[i] * n1;
      sum[kDbPre][i] += z[i];
      sum[kDwPost][i] += p * n2;
      sum[kDbPost][i] += p;
      sum[kDgate][i] += u * (n2 * w2[i] + b2[i]);
    }
  }
#pragma unroll
  for (int s = 0; s < kSums; ++s) {
    if (!a.sums[s]) continue;
    float* p = a.partial + (static_cast<uint64_t>(s) * gridDim.y + blockIdx.y) * pad + c;
    *reinterpret_cast<f32x4*>(p) = f32x4{sum[s][0], sum[s][1], sum[s][2], sum[s][3]};
    *reinterpret_cast<f32x4*>(p + 4) = f32x4{sum[s][4], sum[s][5], sum[s][6], sum[s][7]};
  }
}

// Joins the streams' partial sums in a fixed order: 64 columns a workgroup, 16
// waves each taking every 16th stream, then the 16 sums in turn.
struct JoinArgs {
  const float* partial;
  uint64_t streams, pad;
  uint32_t cols;
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
  if (col < a.cols) {
#pragma unroll 8
    for (uint64_t k = wave; k < a.streams; k += kJoinWaves) s += p[k * a.pad];
  }
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

// ------------------------------------------------------------ launches

template <typename T, int WAVES, int HELD>
hipError_t forward_rows(const BlockNormLaunch& a, hipStream_t stream) {
  constexpr uint64_t kMost = most_workgroups(64 * WAVES);   // rows of a launch
  const bool full = a.cols == 64u * WAVES * HELD * kChunk;
  for (uint64_t row0 = 0; row0 < a.rows; row0 += kMost) {
    const uint64_t left = a.rows - row0;
    const uint32_t wgs = static_cast<uint32_t>(left < kMost ? left : kMost);
    if (full) block_norm_kernel<T, WAVES, HELD, true><<<wgs, 64 * WAVES, 0, stream>>>(a, row0);
    else block_norm_kernel<T, WAVES, HELD, false><<<wgs, 64 * WAVES, 0, stream>>>(a, row0);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T>
hipError_t forward(const BlockNormLaunch& a, hipStream_t stream) {
  // the least waves whose threads hold the row in up to eight chunks, and the least
  // chunks: 16384 x 5120 in 2 x 5 takes 115 us where 2 x 8 took 335
  const uint32_t per = 64 * kChunk;
  const uint32_t waves = a.cols <= 8 * per ? 1 : a.cols <= 16 * per ? 2 : 4;
  const uint32_t held = (a.cols + waves * per - 1) / (waves * per);
  if (waves == 1) {
    if (held <= 1) return forward_rows<T, 1, 1>(a, stream);
    if (held <= 2) return forward_rows<T, 1, 2>(a, stream);
    if (held <= 4) return forward_rows<T, 1, 4>(a, stream);
    if (held <= 6) return forward_rows<T, 1, 6>(a, stream);
    return forward_rows<T, 1, 8>(a, stream);
  }
  if (waves == 2) {
    if (held <= 5) return forward_rows<T, 2, 5>(a, stream);
    if (held <= 6) return forward_rows<T, 2, 6>(a, stream);
    return forward_rows<T, 2, 8>(a, stream);
  }
  if (held <= 5) return forward_rows<T, 4, 5>(a, stream);
  if (held <= 6) return forward_rows<T, 4, 6>(a, stream);
  return forward_rows<T, 4, 8>(a, stream);
}

template <typename T, int FMT>
void backward(const BlockNormGradLaunch& a, int sets, uint32_t wgs, hipStream_t stream) {
  const uint64_t pad = padded(a.cols);
  const int held = grad_held(a.cols, sets);
  const uint32_t threads = 64 * grad_waves(a.cols, sets);
  const bool full = a.cols == static_cast<uint32_t>(held) * threads * kChunk;
  const uint32_t shared =   // at most 128 KiB
      (rows_shared<T>(sets) ? 8 : 4) * held * threads * sizeof(f32x4);
  if (held <= 2) {
    auto run = [&](auto h) {
      constexpr int kHeld = decltype(h)::value;
      if (full && sets == 3)
        block_norm_grad_kernel<T, FMT, kHeld, 3, true><<<wgs, threads, 0, stream>>>(a, pad);
      else if (full)
        block_norm_grad_kernel<T, FMT, kHeld, 5, true><<<wgs, threads, shared, stream>>>(a, pad);
      else if (sets == 3)
        block_norm_grad_kernel<T, FMT, kHeld, 3, false><<<wgs, threads, 0, stream>>>(a, pad);
      else
        block_norm_grad_kernel<T, FMT, kHeld, 5, false><<<wgs, threads, shared, stream>>>(a, pad);
    };
    if (held == 1) run(std::integral_constant<int, 1>());
    else run(std::integral_constant<int, 2>());
  } else {
    auto rows = [&](const BlockNormGradLaunch& l) {
      if (full) block_norm_grad_kernel<T, FMT, 4, 0, true><<<wgs, threads, 0, stream>>>(l, pad);
      else block_norm_grad_kernel<T, FMT, 4, 0, false><<<wgs, threads, 0, stream>>>(l, pad);
    };
    // outputs that replace inputs wait until the sums have read those: the means are
    // then made first, by a pass that stores nothing else
    const bool replaces =
        (a.dres.p && a.dres.p == a.dout.p) || (a.dblock.p && a.dblock.p == a.dz.p);
    BlockNormGradLaunch first = a;
    if (a.partial && replaces) first.dres.p = first.dblock.p = first.dgate.p = nullptr;
    rows(first);
    if (a.partial)
      norm_sums_kernel<T, FMT>
          <<<dim3((a.cols + kSumCols - 1) / kSumCols,
                  static_cast<uint32_t>(grad_streams(a.rows, a.cols, sets))),
             kSumThreads, 0, stream>>>(a, pad);
    if (a.partial && replaces) {
      BlockNormGradLaunch last = a;
      last.means = nullptr;
      rows(last);
    }
  }
}

}  // namespace

uint64_t norm_grad_workspace(uint64_t rows, uint64_t cols) {
  const uint64_t means = wide_rows(cols) ? rows * 2 : 0;
  const uint64_t three = grad_streams(rows, cols, 3), five = grad_streams(rows, cols, 5);
  return ((three > five ? three : five) * padded(cols) * kSums + means) * sizeof(float);
}

hipError_t launch_block_norm(const BlockNormLaunch& a, hipStream_t stream) {
  return a.dtype == kF16 ? forward<F16>(a, stream) : forward<Bf16>(a, stream);
}

hipError_t launch_block_norm_grad(const BlockNormGradLaunch& in, hipStream_t stream) {
  BlockNormGradLaunch a = in;
  bool any = false;
  for (void* p : a.sums) any = any || p != nullptr;
  if (!any) a.partial = nullptr;
  // layer norms need the row sums of the biases' path too
  const bool five = a.sums[kDbPre] || a.sums[kDbPost] || a.pre.kind == ZERO_NORM_LAYER ||
                    a.post.kind == ZERO_NORM_LAYER;
  const int sets = five ? 5 : 3;
  const uint32_t wgs = static_cast<uint32_t>(grad_wgs(a.rows, a.cols, sets));
  const uint64_t streams = grad_streams(a.rows, a.cols, sets);
  a.means = a.partial && wide_rows(a.cols) ? a.partial + streams * padded(a.cols) * kSums : nullptr;
  if (wgs) {
    if (a.dtype == kF16) {
      if (a.format == kInt8) backward<F16, kInt8>(a, sets, wgs, stream);
      else backward<F16, kE4m3>(a, sets, wgs, stream);
    } else {
      if (a.format == kInt8) backward<Bf16, kInt8>(a, sets, wgs, stream);
      else backward<Bf16, kE4m3>(a, sets, wgs, stream);
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
  int n = 0;
  for (int s = 0; s < kSums; ++s) {
    if (!a.sums[s]) continue;
    j.set[n] = s;
    j.out[n++] = a.sums[s];
  }
  join_sums_kernel<<<dim3((a.cols + 63) / 64, n), 64 * kJoinWaves, 0, stream>>>(j);
  return hipGetLastError();
}

}  // namespace act
}  // namespace zero
