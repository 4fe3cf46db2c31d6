// Losses over a vocabulary, from the last hidden states x and the projection W, and
// their gradients, with z = x W^T / tau:
//   cross entropy  l_t = w_t (lse_t - z_ty)
//   distillation   l_t = w_t tau^2 sum over j of q_tj (log q_tj - (z_tj - lse_t)),
//                  q_t the softmax of a teacher's top logits / tau
//   g_t = w_t (p_t - q_t) (p_t the softmax of z_t; q_t is 1 at the target for the first)
//   dx = c g W,  dW = c g^T x,  c = scale * tau
//
// Tokens go in pieces whose logits fit a bounded workspace: the logits of a piece in
// fp32, one pass over each row that replaces them with g in 16 bits, and the two
// products with it.  That is three products for the three that the definition has;
// pieces of the vocabulary with all tokens in each would need a fourth (g needs the
// whole row's sum first).  Cross entropy alone stores no logits; distillation does for
// its entries' sake.  g is the only value that is rounded on the way: at a
// target p - q is formed in fp32 from fp32 logits, so what cancels there is not lost.
//
// Tokens without a target are left out of everything: the others are first brought
// together, so what a left-out token holds (NaN and infinities too) reaches nothing.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "act/format.h"
#include "act/launch.h"
#include "act/layer.h"
#include "act/product.h"

namespace zero {
namespace act {
namespace {

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLowest = -3.402823466e38f;
constexpr int kPickThreads = 1024, kRowThreads = 512;

// fp16 holds g as 2^14 g / 2^e, e the least with all finite weights at most 2^e: |g| 2^-e
// <= 1 leaves the probabilities 28 binary places above its smallest normal value.  bf16
// needs no such factor and takes the same.  Weights that are not finite make their own
// rows so, and have no part in e: they would take the others' range away.
constexpr int kGradBits = 14;

struct Head {
  uint32_t count;           // tokens with a loss
  uint32_t stand;           // rows of g: as many, or twice with kTwice (see kFewTokens)
  float held;               // 2^14 / 2^e
  float unit;               // c 2^e / 2^14
};

// The workspace: what lies where.
struct Room {
  uint64_t piece, pieces;   // tokens of a piece
  uint64_t least;           // rows that g has room for, however small a piece
  uint64_t lead_x, lead_z, lead_w;
  uint64_t wide;            // columns of a row of logits: whole chunks, and -infinity
  uint64_t entries;         // of a row: maxima and sums of parts of it
  uint64_t rows, slots, flags, x, z, stats, ids, sums, partial, bytes;
  MulPlan logits, dx, dw;
};

// Bytes of a piece's logits, about (a piece has 256 tokens at least).  Larger pieces
// add to dW's running sums less often: 8192 tokens x 131072 words at 4096 take 22.4 ms
// in two pieces of 2 GiB with those sums, another 2 GiB, and 22.1 in one of 4 GiB.  Where
// the sums are smaller (fewer columns, dx alone) one piece takes more memory than two;
// callers who want less give parts of the rows.
constexpr uint64_t kPieceBytes = 6ull << 30;
// Of few tokens with a loss, g's entries keep what their rounding leaves out: a token's row
// of g stands a second time, as zeros but for those rests, behind all others, and so does its
// x.  A gradient's entries hold nearly all of it.  Their rounding makes dx's and dw's error
// 1.4 times that of the results' own rounding, however many tokens there are, but only of
// many is that what a call gets: the worst of 60 calls is 2.2 times the results' own for one
// token (fp16, norms relative to 64 bits: 4.6e-4, with rests 2.6e-4), 1.7 for 16, 1.6 for 64
// (3.4e-4; mean 3.05e-4) and 1.5 for 256, with rests 1.05 for 16 and more.  The rests cost 0-1%
// up to 32 tokens (131072 words at 4096, fp16: 770 us), 7% at 64 (797 -> 854 us), 13% at 128
// (903 -> 1011) and 28% at 256 (1131 -> 1450).  It is the tokens with a loss that count,
// known on the device, not the rows given: 64 tokens of 1024 rows, 933 -> 964 us.
constexpr uint32_t kFewTokens = 64;
constexpr uint64_t kMostRows = 1ull << 22;  // of a piece: a workgroup a row in one launch

Room room_of(uint64_t rows, uint64_t cols, uint64_t vocab, uint32_t top, bool dx, bool dw) {
  Room r = {};
  r.lead_x = row_lead(cols);
  r.wide = chunks_up(vocab, 128);    // whole tiles of the logits' product
  r.lead_z = row_lead(2 * r.wide) / 2;
  r.lead_w = chunks_up(cols, kChunk);
  uint64_t most = kPieceBytes / (4 * r.wide) / 256 * 256;
  if (most < 256) most = 256;
  if (most > kMostRows) most = kMostRows;
  r.pieces = rows ? (rows + most - 1) / most : 1;
  r.piece = r.pieces > 1 ? chunks_up((rows + r.pieces - 1) / r.pieces, 256) : rows;
  uint64_t at = 256;
  const auto take = [&](uint64_t bytes) {
    const uint64_t from = at;
    at = chunks_up(at + bytes, 256);
    return from;
  };
  r.rows = take(rows * 4);
  r.slots = take(rows * 4);
  r.flags = take(rows);
  if (dx || dw) r.least = 2 * (rows < kFewTokens ? rows : kFewTokens);
  const uint64_t tokens = r.piece > r.least ? r.piece : r.least;
  r.x = take(tokens * r.lead_x * 2);
  const bool whole = cols % kChunk == 0;
  r.logits = plan_product(r.piece, vocab, cols, {false, true, true, whole});
  const uint64_t tiles = (vocab + (r.logits.tile == 256 ? 255 : 127)) /
                         (r.logits.tile == 256 ? 256 : 128);
  r.entries = tiles * (r.logits.tile == 32 ? 4 : 2);          // one a wave's columns
  r.stats = take(r.piece * r.entries * 8);
  // cross entropy alone needs the target's logit of each row, not the row
  if (dx || dw || top) r.z = take(tokens * r.lead_z * 4);
  else r.ids = take(r.piece * 8);
  uint64_t partial = 0;
  if (dx) {
    r.dx = plan_product(tokens, cols, vocab, {true, true, true, whole});
    uint64_t partials = partial_rows(r.dx, tokens);
    if (partials < r.least) partials = r.least;
    partial = partials * r.lead_w * 4;
  }
  if (dw) {
    r.dw = plan_product(vocab, cols, tokens, {true, false, false, true});
    const uint64_t more = partial_rows(r.dw, vocab) * r.lead_w * 4;
    if (more > partial) partial = more;
    if (r.pieces > 1) r.sums = take(vocab * r.lead_w * 4);
  }
  r.partial = take(partial);
  r.bytes = at;
  return r;
}

__device__ __forceinline__ int64_t id_at(const VocabLaunch& a, uint64_t t, uint32_t j) {
  const uint64_t i = t * a.ids_stride + j;
  return a.ids_64 ? static_cast<const int64_t*>(a.ids)[i] : static_cast<const int32_t*>(a.ids)[i];
}

// Whether a token has entries: a wave a token.
__global__ __launch_bounds__(256) void loss_flags_kernel(VocabLaunch a, uint8_t* flags) {
  const uint64_t t = static_cast<uint64_t>(blockIdx.x) * 4 + threadIdx.x / 64;
  if (t >= a.rows) return;
  bool any = false;
  for (uint32_t j = threadIdx.x % 64; j < a.top; j += 64) any |= id_at(a, t, j) >= 0;
  const bool some = __builtin_amdgcn_ballot_w64(any) != 0;
  if (threadIdx.x % 64 == 0) flags[t] = some;
}

// The tokens that have a loss, in their order; each token's place among them; the
// largest finite weight's power of two.  One workgroup.
__global__ __launch_bounds__(kPickThreads) void loss_pick_kernel(VocabLaunch a,
                                                                 const uint8_t* flags,
                                                                 uint32_t* rows, uint32_t* slots,
                                                                 Head* head, float c,
                                                                 uint32_t few) {
  __shared__ uint32_t counts[kPickThreads / 64];
  __shared__ float tops[kPickThreads / 64];
  const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  uint32_t before = 0;
  float top = 0.0f;
  for (uint64_t t0 = 0; t0 < a.rows; t0 += kPickThreads) {
    const uint64_t t = t0 + threadIdx.x;
    bool in = t < a.rows && (a.top ? flags[t] != 0 : id_at(a, t, 0) >= 0);
    if (in && a.weights) {
      const float w = a.weights[t];
      in = w != 0.0f;                                   // NaN is a weight
      if (fabsf(w) < INFINITY) top = fmaxf(top, fabsf(w));
    }
    const uint64_t votes = __builtin_amdgcn_ballot_w64(in);
    if (lane == 0) counts[wave] = __popcll(votes);
    __syncthreads();
    uint32_t at = before + __popcll(votes & ((1ull << lane) - 1));
    for (uint32_t i = 0; i < kPickThreads / 64; ++i) {
      if (i < wave) at += counts[i];
      before += counts[i];
    }
    if (t < a.rows) slots[t] = in ? at : UINT32_MAX;
    if (in) rows[at] = static_cast<uint32_t>(t);
    __syncthreads();
  }
  for (int i = 1; i < 64; i *= 2) top = fmaxf(top, __shfl_xor(top, i));
  if (lane == 0) tops[wave] = top;
  __syncthreads();
  if (threadIdx.x) return;
  for (uint32_t i = 1; i < kPickThreads / 64; ++i) top = fmaxf(top, tops[i]);
  int e = 0;
  if (a.weights && top > 0.0f) {
    frexpf(top, &e);                                    // top < 2^e, e at most 128
    e = e < -110 ? -110 : e;                            // 2^(14 - e) is finite
  }
  head->count = before;
  head->stand = before <= few ? 2 * before | kTwice : before;
  head->held = ldexpf(1.0f, kGradBits - e);
  head->unit = ldexpf(c, e - kGradBits);
}

// Brings a piece's tokens together: those at places [first, first + most) among the ones
// with a loss.  The first piece also clears the others' loss and dx.  A wave a token.
__global__ __launch_bounds__(256) void loss_rows_kernel(VocabLaunch a, const Head* head,
                                                        const uint32_t* slots, uint64_t first,
                                                        uint64_t most, uint16_t* to, uint64_t lead,
                                                        int32_t* ids) {
  const uint64_t t = static_cast<uint64_t>(blockIdx.x) * 4 + threadIdx.x / 64;
  if (t >= a.rows) return;
  const uint32_t count = head->count, stand = head->stand;
  const uint32_t slot = __builtin_amdgcn_readfirstlane(slots[t]);
  const uint64_t c0 = threadIdx.x % 64 * kChunk;
  if (slot == UINT32_MAX) {
    if (first) return;
    if (threadIdx.x % 64 == 0) a.loss[t] = 0.0f;
    if (a.dx.p)
      for (uint64_t c = c0; c < a.cols; c += 512)
        store8<false>(a.dx.p + t * a.dx.stride, c, a.cols, u32x4{0, 0, 0, 0});
    return;
  }
  if (slot < first || slot >= first + most) return;
  if (ids && threadIdx.x % 64 == 0) {
    const int64_t id = id_at(a, t, 0);
    ids[slot - first] = id < static_cast<int64_t>(a.vocab) ? static_cast<int32_t>(id) : -1;
  }
  const uint16_t* from = a.x.p + t * a.x.stride;
  const bool twice = (stand & kTwice) != 0;              // first is 0
  uint16_t* row = to + (slot - first) * lead;
  for (uint64_t c = c0; c < lead; c += 512) {
    const u32x4 w = c < a.cols ? load8(from, c, a.cols) : u32x4{0, 0, 0, 0};
    *reinterpret_cast<u32x4*>(row + c) = w;
    if (twice) *reinterpret_cast<u32x4*>(row + count * lead + c) = w;
  }
}

__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

struct Part {
  float top, sum;           // of a part of a row: the maximum m, and the sum of exp(z - m)
};

// A piece's logits, scaled: the maximum and sum of each wave's columns of a row, from the
// fp32 sums where they are (a row is then read once less: 4096 x 131072 words, 1060 ->
// 690 us for the pass over them), and what is wanted of the logits themselves: all (those
// past the vocabulary are -infinity up to `wide`), or each row's target's.
struct Logits {
  static constexpr bool kPairs = false, kRows = true, kJoins = false, kOld = false, kAdds = false;
  struct Old {};
  float* z;                 // or nullptr
  uint64_t lead, wide, vocab;
  float scale;
  Part* parts;              // [rows][entries]
  uint64_t entries;
  const int32_t* ids;       // of the targets, without z
  float* caught;

  __device__ __forceinline__ void cut(uint32_t, uint64_t, bool) {}
  __device__ __forceinline__ bool stores() const { return z != nullptr; }
  __device__ __forceinline__ float load_factor() const { return 1.0f; }
  __device__ __forceinline__ uint64_t row_of(int, uint32_t, uint64_t m) const { return m; }

  struct Row {
    float top = kLowest, sum = 0.0f;
  };

  template <int N>
  __device__ __forceinline__ void columns(Row& row, float (&x)[N], uint64_t m, uint64_t n,
                                          uint64_t m_all) const {
    if (n + N > vocab) {
      const int exist = static_cast<int>(static_cast<int64_t>(vocab) - static_cast<int64_t>(n));
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i >= exist) x[i] = -INFINITY;
    }
    float top = row.top;
#pragma unroll
    for (int i = 0; i < N; ++i) top = fmaxf(top, x[i]);
    const float c = scale * kLog2e;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) sum += __builtin_amdgcn_exp2f((x[i] - top) * c);
    row.sum = row.sum * __builtin_amdgcn_exp2f((row.top - top) * c) + sum;
    row.top = top;
    if (!ids) return;
    const int64_t from = (m < m_all ? ids[m] : -1) - static_cast<int64_t>(n);
    const int mine = from >= 0 && from < N ? static_cast<int>(from) : -1;
    if (__builtin_amdgcn_ballot_w64(mine >= 0) == 0) return;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (mine == i) caught[m] = x[i] * scale;
  }

  __device__ __forceinline__ void finish(const Row& row, uint64_t m, uint64_t piece,
                                         uint64_t m_all) const {
    const float c = scale * kLog2e, top = fmaxf(row.top, __shfl_xor(row.top, 32));
    float sum = row.sum * __builtin_amdgcn_exp2f((row.top - top) * c);
    sum += __shfl_xor(sum, 32);
    if (threadIdx.x % 64 < 32 && m < m_all) parts[m * entries + piece] = {top * scale, sum};
  }

  __device__ __forceinline__ bool simple() const { return true; }

  struct Now {
    static constexpr bool kOld = false;
    struct Old {};
    float* z;
    uint64_t lead;
    float scale;

    __device__ __forceinline__ uint64_t row_of(int, uint32_t, uint64_t m) const { return m; }

    template <typename T>
    __device__ __forceinline__ void put(uint32_t, uint64_t m, uint64_t n, uint64_t,
                                        float (&x)[8]) const {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= scale;
      f32x4* p = reinterpret_cast<f32x4*>(z + m * lead + n);
      p[0] = f32x4{x[0], x[1], x[2], x[3]};
      p[1] = f32x4{x[4], x[5], x[6], x[7]};
    }
  };

  __device__ __forceinline__ bool adds() const { return false; }
  template <bool>
  __device__ __forceinline__ Now now(uint32_t, uint64_t, float) const { return {z, lead, scale}; }

  template <typename T>
  __device__ __forceinline__ void put(uint32_t, uint64_t m, uint64_t n, uint64_t m_all,
                                      float (&x)[8]) const {
    if (m >= m_all || n >= wide) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = n + i < vocab ? x[i] * scale : -INFINITY;
    f32x4* p = reinterpret_cast<f32x4*>(z + m * lead + n);
    p[0] = f32x4{x[0], x[1], x[2], x[3]};
    p[1] = f32x4{x[4], x[5], x[6], x[7]};
  }
};

// The sum of v over the workgroup, in every thread; the order is fixed.
__device__ __forceinline__ float group_sum(float v, float* room) {
  v = wave_sum(v);
  __syncthreads();
  if (threadIdx.x % 64 == 0) room[threadIdx.x / 64] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kRowThreads / 64; ++i) s += room[i];
  return s;
}

__device__ __forceinline__ float group_max(float v, float* room) {
  for (int i = 1; i < 64; i *= 2) v = fmaxf(v, __shfl_xor(v, i));
  __syncthreads();
  if (threadIdx.x % 64 == 0) room[threadIdx.x / 64] = v;
  __syncthreads();
  float s = room[0];
#pragma unroll
  for (int i = 1; i < kRowThreads / 64; ++i) s = fmaxf(s, room[i]);
  return s;
}

__device__ __forceinline__ float teacher_at(const VocabLaunch& a, uint64_t t, uint32_t j) {
  const uint64_t i = t * a.logits_stride + j;
  if (a.logits_dtype == kF32) return static_cast<const float*>(a.logits)[i];
  const uint16_t w = static_cast<const uint16_t*>(a.logits)[i];
  return a.logits_dtype == kF16 ? lo16<F16>(w) : lo16<Bf16>(w);
}

// One row a workgroup: its maximum and sum from its parts, its loss, and (GRAD) g in place
// of its logits, 16 bits from the row's begin on, and where g's rows stand twice the rests
// of its entries in the row's second place.
template <typename T, bool GRAD>
__global__ __launch_bounds__(kRowThreads) void loss_row_kernel(
    VocabLaunch a, const Head* head, const uint32_t* rows, uint64_t first, const Part* parts,
    uint64_t entries, const float* caught, float* z_all, uint64_t lead, uint64_t wide) {
  __shared__ float room[kRowThreads / 64];
  __shared__ int32_t ids[kMaxTop];
  __shared__ float shares[kMaxTop];
  const uint64_t slot = first + blockIdx.x;
  if (slot >= head->count) return;
  const uint32_t t = rows[slot];
  float* z = z_all + blockIdx.x * lead;
  const uint32_t tid = threadIdx.x;

  // the maximum m and the sum s of exp(z - m)
  float m = kLowest, s = 0.0f;
  const Part* own_parts = parts + blockIdx.x * entries;
  for (uint64_t e = tid; e < entries; e += kRowThreads) {
    const Part p = own_parts[e];
    const float top = fmaxf(m, p.top);
    s = s * exp_of(m - top) + p.sum * exp_of(p.top - top);
    m = top;
  }
  const float all = group_max(m, room);
  s = group_sum(s * exp_of(m - all), room);
  m = all;
  const float log_s = logf(s);

  float w = a.weights ? a.weights[t] : 1.0f;
  // the entries: their shares q, and the loss
  constexpr int kEach = kMaxTop / kRowThreads;
  float target[kEach];
  float loss;
  bool lost = false;                                    // an id past the vocabulary
  if (a.top == 0) {
    const int64_t id = id_at(a, t, 0);
    lost = id >= static_cast<int64_t>(a.vocab);
    target[0] = lost ? 0.0f : caught ? caught[blockIdx.x] : z[id];
    if (tid == 0) {
      ids[0] = static_cast<int32_t>(id);
      shares[0] = 1.0f;
    }
    loss = w * ((m - target[0]) + log_s);
  } else {
    float e[kEach], at[kEach], most = -INFINITY;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const uint32_t j = tid + i * kRowThreads;
      int64_t id = j < a.top ? id_at(a, t, j) : -1;
      at[i] = target[i] = 0.0f;
      e[i] = -INFINITY;
      if (id >= 0) {
        e[i] = teacher_at(a, t, j) / a.tau;
        most = fmaxf(most, e[i]);
        if (id >= static_cast<int64_t>(a.vocab)) {
          lost = true;
          id = -1;
        } else {
          target[i] = z[id];
        }
        at[i] = 1.0f;
      }
      if (j < a.top) ids[j] = static_cast<int32_t>(id);
    }
    most = group_max(most, room);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      e[i] = at[i] != 0.0f ? e[i] - most : 0.0f;        // log of the share, before the sum
      at[i] = at[i] != 0.0f ? exp_of(e[i]) : 0.0f;
      sum += at[i];
    }
    sum = group_sum(sum, room);
    const float log_sum = logf(sum);
    float part = 0.0f;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const uint32_t j = tid + i * kRowThreads;
      const float q = at[i] / sum;
      if (j < a.top) shares[j] = q;
      // a share of 0 adds nothing, however far its logarithm is
      if (q != 0.0f) part += q * ((e[i] - log_sum) - ((target[i] - m) - log_s));
    }
    loss = group_sum(part, room) * (w * (a.tau * a.tau));
    lost = group_max(lost ? 1.0f : 0.0f, room) != 0.0f;
  }
  if (lost) loss = w = __builtin_nanf("");
  if (tid == 0) a.loss[t] = loss;
  if constexpr (GRAD) {
    const float each = w * head->held / s, held = w * head->held;
    uint16_t* g = reinterpret_cast<uint16_t*>(z);
    const bool twice = (head->stand & kTwice) != 0;
    uint16_t* rests = reinterpret_cast<uint16_t*>(z + head->count * lead);
    const uint32_t some = a.top ? a.top : 1;
    // the entries' own values of g, from fp32 logits: an id that stands there twice
    // takes the shares of both
    float own[kEach];
    __syncthreads();                                    // ids and shares
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const uint32_t j = tid + i * kRowThreads;
      own[i] = 0.0f;
      if (j < some && ids[j] >= 0) {
        float q = 0.0f;
        for (uint32_t l = 0; l < some; ++l)
          if (ids[l] == ids[j]) q += shares[l];
        own[i] = (exp_of(target[i] - m) / s - q) * held;
      }
      forget(own[i]);
    }
    // Chunk i of g goes over logits of chunk i / 2: a barrier at every power of two
    // keeps all threads' loads of those before it.
    constexpr uint64_t kStep = kRowThreads * kChunk;
    uint64_t chunk = 0;
    for (uint64_t c0 = 0; c0 < wide; c0 += kStep, ++chunk) {
      const uint64_t c = c0 + tid * kChunk;
      f32x4 u = {0.f, 0.f, 0.f, 0.f}, v = u;
      if (c < wide) {
        u = *reinterpret_cast<const f32x4*>(z + c);
        v = *reinterpret_cast<const f32x4*>(z + c + 4);
      }
      forget(u);
      forget(v);
      if ((chunk & (chunk - 1)) == 0) __syncthreads();
      float x[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = exp_of(u[i] - m) * each;
        x[4 + i] = exp_of(v[i] - m) * each;
      }
      if (c < wide) *reinterpret_cast<u32x4*>(g + c) = pack8<T>(x);
    }
    if (twice)
      for (uint64_t c = tid * kChunk; c < wide; c += kStep)
        *reinterpret_cast<u32x4*>(rests + c) = u32x4{0, 0, 0, 0};
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const uint32_t j = tid + i * kRowThreads;
      if (j >= some || ids[j] < 0 || ids[j] >= static_cast<int64_t>(a.vocab)) continue;
      const uint16_t near = static_cast<uint16_t>(pack16<T>(own[i], 0.0f));
      g[ids[j]] = near;
      if (!twice) continue;
      const float rest = own[i] - lo16<T>(near);
      rests[ids[j]] = static_cast<uint16_t>(pack16<T>(rest == rest ? rest : 0.0f, 0.0f));
    }
  }
}

template <typename T>
hipError_t run_loss(const VocabLaunch& a, hipStream_t stream) {
  const bool dx = a.dx.p != nullptr, dw = a.dw != nullptr;
  const Room r = room_of(a.rows, a.cols, a.vocab, a.top, dx, dw);
  uint8_t* ws = a.workspace;
  Head* head = reinterpret_cast<Head*>(ws);
  uint32_t* rows = reinterpret_cast<uint32_t*>(ws + r.rows);
  uint32_t* slots = reinterpret_cast<uint32_t*>(ws + r.slots);
  uint16_t* x = reinterpret_cast<uint16_t*>(ws + r.x);
  float* z = r.z ? reinterpret_cast<float*>(ws + r.z) : nullptr;
  Part* parts = reinterpret_cast<Part*>(ws + r.stats);
  int32_t* ids = r.ids ? reinterpret_cast<int32_t*>(ws + r.ids) : nullptr;
  float* caught = r.ids ? reinterpret_cast<float*>(ws + r.ids + 4 * r.piece) : nullptr;
  float* partial = reinterpret_cast<float*>(ws + r.partial);
  const uint32_t waves = static_cast<uint32_t>((a.rows + 3) / 4);
  hipError_t e = hipSuccess;
  if (a.rows) {
    if (a.top) {
      loss_flags_kernel<<<waves, 256, 0, stream>>>(a, ws + r.flags);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    loss_pick_kernel<<<1, kPickThreads, 0, stream>>>(a, ws + r.flags, rows, slots, head,
                                                     static_cast<float>(a.scale * a.tau),
                                                     dx || dw ? kFewTokens : 0);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  for (uint64_t p = 0; p < r.pieces; ++p) {
    const uint64_t first = p * r.piece;
    const uint64_t most = a.rows - first < r.piece ? a.rows - first : r.piece;
    const uint64_t tokens = most > r.least ? most : r.least;
    const Operand xs = {x, r.lead_x, most, true};
    const Operand w_rows = {a.w.p, a.w.stride, a.vocab, false};
    const Operand w_cols = {a.w.p, a.w.stride, a.cols, false};
    const uint64_t lead_g = 2 * r.lead_z;
    const uint16_t* g = reinterpret_cast<const uint16_t*>(z);
    if (a.rows) {
      loss_rows_kernel<<<waves, 256, 0, stream>>>(a, head, slots, first, most, x, r.lead_x, ids);
      if ((e = hipGetLastError()) != hipSuccess) return e;
      const Extents ex = {most, a.vocab, a.cols, 1, 1, 0, &head->count, first, 0};
      const Logits logits = {z, r.lead_z, r.wide, a.vocab, 1.0f / a.tau, parts, r.entries, ids,
                             caught};
      e = run_product<T, true, true>(plan_of(r.logits, most, a.vocab), xs, w_rows, ex, logits,
                                     stream);
      if (e != hipSuccess) return e;
      const uint32_t grid = static_cast<uint32_t>(most);
      if (dx || dw)
        loss_row_kernel<T, true><<<grid, kRowThreads, 0, stream>>>(
            a, head, rows, first, parts, r.entries, caught, z, r.lead_z, r.wide);
      else
        loss_row_kernel<T, false><<<grid, kRowThreads, 0, stream>>>(
            a, head, rows, first, parts, r.entries, caught, z, r.lead_z, r.wide);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (dx && a.rows) {
      const Operand d = {g, lead_g, tokens, true};
      const Extents ex = {tokens, a.cols, a.vocab, 1, 1, 0, &head->stand, first, 0};
      Sink s = {};
      s.out = a.dx.p;
      s.stride = a.dx.stride;
      s.dtype = T::kType;
      s.cols = a.cols;
      s.rows = rows + first;
      s.factor = &head->unit;
      s.lead = r.lead_w;
      s.partial = partial;
      s.twice = 1;
      e = run_product<T, true, false>(plan_of(r.dx, tokens, a.cols), d, w_cols, ex, s, stream);
      if (e != hipSuccess) return e;
    }
    if (dw) {
      const Operand d = {g, lead_g, a.vocab, true}, xc = {x, r.lead_x, a.cols, true};
      const Extents ex = {a.vocab, a.cols, tokens, 1, 1, 0, a.rows ? &head->stand : nullptr, first,
                          1};
      Sink s = {};
      s.out = a.dw;
      s.stride = a.dw_stride;
      s.dtype = a.dw_dtype;
      s.accumulate = a.accumulate;
      s.cols = a.cols;
      s.factor = a.rows ? &head->unit : nullptr;
      s.lead = r.lead_w;
      s.partial = partial;
      s.last = 1;
      if (r.pieces > 1) {
        s.sums = reinterpret_cast<float*>(ws + r.sums);
        s.add = p > 0;
        s.last = p + 1 == r.pieces;
      }
      e = run_product<T, false, false>(r.dw, d, xc, ex, s, stream);
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

}  // namespace

uint64_t vocab_workspace(uint64_t rows, uint64_t cols, uint64_t vocab, uint32_t top, bool dx,
                         bool dw) {
  return room_of(rows, cols, vocab, top, dx, dw).bytes;
}

bool vocab_fits(uint64_t rows, uint64_t cols, uint64_t vocab, bool dx, bool dw) {
  const Room r = room_of(rows, cols, vocab, 0, dx, dw);
  const uint64_t tokens = r.piece > r.least ? r.piece : r.least;
  return product_fits(r.logits, 0, 0) && (!dx || product_fits(r.dx, tokens, cols)) &&
         (!dw || product_fits(r.dw, vocab, cols));
}

hipError_t launch_vocab_loss(const VocabLaunch& a, hipStream_t stream) {
  return a.dtype == kF16 ? run_loss<F16>(a, stream) : run_loss<Bf16>(a, stream);
}

}  // namespace act
}  // namespace zero
