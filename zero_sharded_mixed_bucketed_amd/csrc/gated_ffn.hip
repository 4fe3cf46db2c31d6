// A layer's gated feed-forward block and its backward:
//   a = act(x Wg^T) . (x Wu^T),  W = [Wg; Wu]
// forward in one kernel (both projections, the activation, their product and the
// 8-bit checkpoints of the two projections and of a); backward from the checkpoints:
//   dg = da . u . act'(g), du = da . act(g);  dx = [dg du] W;  dW = [dg du]^T x^.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act/format.h"
#include "act/launch.h"
#include "act/layer.h"
#include "act/product.h"

namespace zero {
namespace act {
namespace {

constexpr float kLog2e = 1.44269504088896341f;

__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * g));
}

// The share p of g that passes, act(g) = g p, and its slope dp/dg.
template <int ACT>
__device__ __forceinline__ float passed(float g, float* slope) {
  if constexpr (ACT == kSilu) {
    const float p = sigmoid(g);
    *slope = p * (1.0f - p);
    return p;
  } else if constexpr (ACT == kGelu) {
    *slope = 0.398942280401432678f * __builtin_amdgcn_exp2f(-0.5f * kLog2e * g * g);
    return 0.5f * erfcf(-0.707106781186547524f * g);
  } else {
    // (1 + tanh(y)) / 2 = sigmoid(2 y)
    const float y2 = 1.59576912160573071f * (g + 0.044715f * g * g * g);
    const float p = sigmoid(y2);
    *slope = p * (1.0f - p) * (1.59576912160573071f + 0.214069822634528751f * g * g);
    return p;
  }
}

// act(g) of eight gates.  Where p has reached 0, g may be anything, -infinity too.
template <int ACT>
__device__ __forceinline__ void activate8(const float (&g)[8], float (&a)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float slope;
    const float p = passed<ACT>(g[i], &slope);
    a[i] = p == 0.0f ? -0.0f : g[i] * p;
  }
}

__device__ __forceinline__ void activate8(int act, const float (&g)[8], float (&a)[8]) {
  if (act == kSilu) activate8<kSilu>(g, a);
  else if (act == kGelu) activate8<kGelu>(g, a);
  else activate8<kGeluTanh>(g, a);
}

// act(g) and act'(g).  Where p has reached an end, the slope is 0 whatever g is.
template <int ACT>
__device__ __forceinline__ void slopes8(const float (&g)[8], float (&a)[8], float (&d)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float slope;
    const float p = passed<ACT>(g[i], &slope);
    d[i] = p == 0.0f || p == 1.0f ? p : p + g[i] * slope;
    a[i] = p == 0.0f ? -0.0f : g[i] * p;
  }
}

__device__ __forceinline__ void slopes8(int act, const float (&g)[8], float (&a)[8],
                                        float (&d)[8]) {
  if (act == kSilu) slopes8<kSilu>(g, a, d);
  else if (act == kGelu) slopes8<kGelu>(g, a, d);
  else slopes8<kGeluTanh>(g, a, d);
}

// The forward's epilogue: both sums of a column to a, and their checkpoints.
struct Gated {
  static constexpr bool kPairs = true, kRows = false, kJoins = false, kAdds = false;
  Rows out;
  Ckpt c_gate, c_up, c_out;
  uint64_t cols;
  int act, format;

  static constexpr bool kOld = false;
  struct Row {};
  struct Old {};

  __device__ __forceinline__ void cut(uint32_t, uint64_t, bool) {}
  __device__ __forceinline__ bool stores() const { return true; }
  __device__ __forceinline__ bool simple() const { return false; }
  __device__ __forceinline__ float load_factor() const { return 1.0f; }
  __device__ __forceinline__ uint64_t row_of(int, uint32_t, uint64_t m) const { return m; }
  __device__ __forceinline__ bool adds() const { return false; }
  template <bool>
  __device__ __forceinline__ const Gated& now(uint32_t, uint64_t, float) const { return *this; }

  template <typename T>
  __device__ __forceinline__ void keep(const Ckpt& c, uint64_t m, uint64_t n, bool in,
                                       u32x4 w) const {
    if (!c.codes) return;
    uint32_t scale;
    const u32x2 codes = format == kInt8 ? encode8<T, kInt8>(w, &scale)
                                        : encode8<T, kE4m3>(w, &scale);
    if (!in) return;
    store_codes(c.codes + m * c.code_stride, n, cols, codes);
    if (n % kBlock == 0) c.scales[m * c.scale_stride + n / kBlock] = static_cast<uint8_t>(scale);
  }

  template <typename T>
  __device__ __forceinline__ void put(uint32_t, uint64_t m, uint64_t n, uint64_t m_all,
                                      float (&g)[8], float (&u)[8]) const {
    const bool in = m < m_all && n < cols;
    if (n + kChunk > cols)
#pragma unroll
      for (int i = 0; i < 8; ++i)       // not in their block's scale
        if (n + i >= cols) g[i] = u[i] = 0.0f;
    float a[8];
    activate8(act, g, a);
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] *= u[i];
    const u32x4 held = pack8<T>(a);
    if (in && out.p) store8(out.p + m * out.stride, n, cols, held);
    keep<T>(c_gate, m, n, in, pack8<T>(g));
    keep<T>(c_up, m, n, in, pack8<T>(u));
    keep<T>(c_out, m, n, in, held);
  }
};

MulWays forward_ways(uint64_t cols) { return {false, true, false, cols % kChunk == 0}; }

template <typename T>
hipError_t forward(const GatedLaunch& a, hipStream_t stream) {
  const MulPlan p = plan_product(a.rows, 2 * a.width, a.cols, forward_ways(a.cols));
  const Operand x = {a.x.p, a.x.stride, a.rows, false}, w = {a.w.p, a.w.stride, a.width, false};
  const Extents e = {a.rows, a.width, a.cols, 1, 1, 0, nullptr, 0, 0};
  const Gated g = {a.out, a.c_gate, a.c_up, a.c_out, a.width, a.act, a.format};
  return run_product<T, true, true>(p, x, w, e, g, stream);
}

// [dg du] of 512 columns of a row a wave: 8-bit codes and one 16-bit row in, two
// 16-bit rows out, bound by memory.
//
// dg and du are rounded to the call's type, as the products take them: kept in 32 bits
// they would need twice the products.  The gradients' error against 64 bits is 1.4 times
// that of their own rounding (2.9e-4 for 2.1e-4 in fp16, 2.35e-3 for 1.67e-3 in bf16).
// In fp16 without a factor: dout comes as loss scaling left it, dg and du are that times
// values of order 1, and no power of two is safe for all.  Among fp16's subnormals they
// lose what dout itself has lost: dw in fp32 is 2.1e-4 off with dout of 2^-10, 4.8e-4 of
// 2^-14, 7e-3 of 2^-18 (dx in fp16, with its own rounding, 2.9e-4, 5.7e-4, 9e-3).
template <typename T, int FMT>
__global__ __launch_bounds__(kMulThreads) void gated_slopes_kernel(GatedGradLaunch a, uint16_t* to,
                                                                   uint64_t lead, uint64_t unit0,
                                                                   uint64_t units,
                                                                   uint32_t segments) {
  const uint64_t unit = unit0 + static_cast<uint64_t>(blockIdx.x) * 4 +
                        __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  if (unit >= units) return;
  const uint64_t row = unit / segments;
  const uint64_t c = unit % segments * 512 + threadIdx.x % 64 * kChunk;
  if (c >= a.width) return;
  float g[8], u[8], d[8], dg[8], du[8];
  const u32x4 w = stream8(a.dout.p + row * a.dout.stride, c, a.width);
  const u32x2 kg = load_codes(a.c_gate.codes + row * a.c_gate.code_stride, c, a.width);
  const u32x2 ku = load_codes(a.c_up.codes + row * a.c_up.code_stride, c, a.width);
  const uint32_t bg = a.c_gate.scales[row * a.c_gate.scale_stride + c / kBlock];
  const uint32_t bu = a.c_up.scales[row * a.c_up.scale_stride + c / kBlock];
  unpack8<T>(w, d);
  decode8<FMT>(kg, scale_of(bg), g);
  decode8<FMT>(ku, scale_of(bu), u);
  float held[8], slope[8];
  slopes8(a.act, g, held, slope);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    dg[i] = d[i] * u[i] * slope[i];
    du[i] = d[i] * held[i];
  }
  uint16_t* o = to + row * lead;
  store8<false>(o, c, a.width, pack8<T>(dg));
  store8<false>(o + a.width, c, a.width, pack8<T>(du));
}

struct GradRoom {
  uint64_t lead;            // of [dg du], in elements
  MulPlan plan, weight;     // of dx, and of dw if held
  bool held;                // dw from x^ in 16 bits
  uint64_t lead_x, slopes, x, bytes;
};

// dw takes x^ in 16 bits first where its product fills the chip with whole 256 x 256 tiles:
// 8192 tokens, 4096 -> 2 x 16384 takes 1.96 + 0.02 ms where the product straight from the
// 8-bit codes, beside their arithmetic, takes 2.20; with fewer tiles, or columns that are
// not in whole chunks, the latter's splits and edges are better.
GradRoom grad_room(uint64_t rows, uint64_t cols, uint64_t width) {
  GradRoom r;
  r.lead = row_lead(2 * width);
  r.lead_x = row_lead(cols);
  const bool whole = (2 * width) % kChunk == 0 && cols % kChunk == 0;
  r.plan = plan_product(rows, cols, 2 * width, {true, true, false, whole});
  r.weight = plan_product(2 * width, cols, rows, {true, false, false, whole});
  r.held = r.weight.tile == 256 && rows && whole;
  r.slopes = chunks_up(rows * r.lead * 2, 256);
  r.x = r.held ? chunks_up(rows * r.lead_x * 2, 256) : 0;
  const uint64_t lead_out = chunks_up(cols, kChunk) * 4;
  uint64_t rest = partial_rows(r.plan, rows) * lead_out;
  const uint64_t weight = !r.held ? weight_grad_workspace(rows, cols, 2 * width)
                          : partial_rows(r.weight, 2 * width) * lead_out;
  if (weight > rest) rest = weight;
  r.bytes = r.slopes + r.x + rest;
  return r;
}

template <typename T>
hipError_t backward(const GatedGradLaunch& a, hipStream_t stream) {
  const GradRoom room = grad_room(a.rows, a.cols, a.width);
  uint16_t* slopes = reinterpret_cast<uint16_t*>(a.workspace);
  uint16_t* held = reinterpret_cast<uint16_t*>(a.workspace + room.slopes);
  float* rest = reinterpret_cast<float*>(a.workspace + room.slopes + room.x);
  if (a.rows) {
    const uint64_t segments = (a.width + 511) / 512, units = a.rows * segments;
    constexpr uint64_t kMost = most_workgroups(kMulThreads);
    for (uint64_t unit = 0; unit < units; unit += 4 * kMost) {
      const uint64_t left = (units - unit + 3) / 4;
      const uint32_t grid = static_cast<uint32_t>(left < kMost ? left : kMost);
      if (a.format == kInt8)
        gated_slopes_kernel<T, kInt8><<<grid, kMulThreads, 0, stream>>>(
            a, slopes, room.lead, unit, units, static_cast<uint32_t>(segments));
      else
        gated_slopes_kernel<T, kE4m3><<<grid, kMulThreads, 0, stream>>>(
            a, slopes, room.lead, unit, units, static_cast<uint32_t>(segments));
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  if (a.dx.p && a.rows) {
    const Operand d = {slopes, room.lead, a.rows, false}, w = {a.w.p, a.w.stride, a.cols, false};
    const Extents x = {a.rows, a.cols, 2 * a.width, 1, 1, 0, nullptr, 0, 0};
    Sink s = {};
    s.out = a.dx.p;
    s.stride = a.dx.stride;
    s.dtype = T::kType;
    s.cols = a.cols;
    s.lead = chunks_up(a.cols, kChunk);
    s.partial = rest;
    const hipError_t e = run_product<T, true, false>(room.plan, d, w, x, s, stream);
    if (e != hipSuccess) return e;
  }
  if (!a.dw) return hipSuccess;
  if (room.held) {
    StoreLaunch read;
    read.c = a.c_x;
    read.x = held;
    read.x_stride = room.lead_x;
    read.dtype = T::kType;
    read.rows = a.rows;
    read.cols = a.cols;
    const hipError_t e = launch_ckpt_read(read, stream);
    if (e != hipSuccess) return e;
    const Operand d = {slopes, room.lead, 2 * a.width, false};
    const Operand x = {held, room.lead_x, a.cols, false};
    const Extents by = {2 * a.width, a.cols, a.rows, 1, 1, 0, nullptr, 0, 0};
    Sink s = {};
    s.out = a.dw;
    s.stride = a.dw_stride;
    s.dtype = a.dw_dtype;
    s.accumulate = a.accumulate;
    s.cols = a.cols;
    s.lead = chunks_up(a.cols, kChunk);
    s.partial = rest;
    return run_product<T, false, false>(room.weight, d, x, by, s, stream);
  }
  WeightGradLaunch L;
  L.x = a.c_x;
  L.rows = a.rows;
  L.k = a.cols;
  L.n = 2 * a.width;
  L.dy = slopes;
  L.dy_stride = room.lead;
  L.dtype = T::kType;
  L.dw = a.dw;
  L.dw_stride = a.dw_stride;
  L.dw_dtype = a.dw_dtype;
  L.accumulate = a.accumulate;
  L.partial = rest;
  return launch_weight_grad(L, stream);
}

}  // namespace

uint64_t gated_grad_workspace(uint64_t rows, uint64_t cols, uint64_t width) {
  return grad_room(rows, cols, width).bytes;
}

bool gated_fits(uint64_t rows, uint64_t cols, uint64_t width, bool dx) {
  if (dx) {
    const GradRoom r = grad_room(rows, cols, width);
    return product_fits(r.plan, rows, cols) && (!r.held || product_fits(r.weight, 2 * width, cols));
  }
  return product_fits(plan_product(rows, 2 * width, cols, forward_ways(cols)), 0, 0);
}

hipError_t launch_gated_ffn(const GatedLaunch& a, hipStream_t stream) {
  return a.dtype == kF16 ? forward<F16>(a, stream) : forward<Bf16>(a, stream);
}

hipError_t launch_gated_ffn_grad(const GatedGradLaunch& a, hipStream_t stream) {
  return a.dtype == kF16 ? backward<F16>(a, stream) : backward<Bf16>(a, stream);
}

}  // namespace act
}  // namespace zero
