// The host side of the gated block's and the losses' entry points under sanitizers,
// with stand-ins for the kernels: every refusal happens before a launch, and what is
// launched has the arguments the call gave.  Prints "layer host check ok" when every
// expectation holds.
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "act/launch.h"
#include "act/layer.h"
#include "kernels.h"
#include "zero.h"

static int g_fail = 0, g_launches = 0;
#define EXPECT(c)                                                            \
  do {                                                                       \
    if (!(c)) {                                                              \
      fprintf(stderr, "%s:%d: expectation failed: %s (last error: %s)\n",    \
              __FILE__, __LINE__, #c, zero_last_error());                    \
      g_fail = 1;                                                            \
    }                                                                        \
  } while (0)

static zero::act::GatedLaunch g_gated;
static zero::act::GatedGradLaunch g_grad;
static zero::act::VocabLaunch g_loss;
static hipError_t g_result = hipSuccess;
static bool g_fits = true;

namespace zero {
const void* reduce_kernel_fn(int) { return nullptr; }
const void* adam_kernel_fn(int) { return nullptr; }
hipError_t launch_reduce(const ReduceLaunch&, const DeviceCaps&, hipStream_t) { return hipErrorUnknown; }
hipError_t launch_adam(const AdamLaunch&, const DeviceCaps&, hipStream_t) { return hipErrorUnknown; }
hipError_t launch_gather(const GatherLaunch&, hipStream_t) { return hipErrorUnknown; }
namespace act {
template <typename L>
static hipError_t keep(L& to, const L& a) {
  to = a;
  ++g_launches;
  return g_result;
}
hipError_t launch_gated_ffn(const GatedLaunch& a, hipStream_t) { return keep(g_gated, a); }
hipError_t launch_gated_ffn_grad(const GatedGradLaunch& a, hipStream_t) { return keep(g_grad, a); }
hipError_t launch_vocab_loss(const VocabLaunch& a, hipStream_t) { return keep(g_loss, a); }
uint64_t gated_grad_workspace(uint64_t, uint64_t, uint64_t) { return 4096; }
uint64_t vocab_workspace(uint64_t, uint64_t, uint64_t, uint32_t, bool dx, bool dw) {
  return 4096 + (dx ? 1024 : 0) + (dw ? 2048 : 0);
}
bool gated_fits(uint64_t, uint64_t, uint64_t, bool) { return g_fits; }
bool vocab_fits(uint64_t, uint64_t, uint64_t, bool, bool) { return g_fits; }
}  // namespace act
}  // namespace zero

int main() {
  char* p = reinterpret_cast<char*>(static_cast<uintptr_t>(0x100000));
  uint8_t* u = reinterpret_cast<uint8_t*>(p);
  zero_ckpt_t gate = {u, u + 0x1000, 6, 70, 72, 5, ZERO_CKPT_E4M3}, up = gate;
  zero_ckpt_t kx = {u, u + 0x1000, 6, 50, 50, 2, ZERO_CKPT_INT8};

  zero_gated_ffn_t f = {};
  f.dtype = ZERO_BF16;
  f.act = ZERO_ACT_GELU;
  f.rows = 6;
  f.cols = 50;
  f.width = 70;
  f.x = p + 2;
  f.x_stride = 51;
  f.w = p + 4;
  f.w_stride = 53;
  f.ckpt_gate = &gate;
  f.ckpt_up = &up;
  EXPECT(zero_gated_ffn(&f, nullptr) == ZERO_OK && g_launches == 1);
  EXPECT(g_gated.out.p == nullptr && g_gated.w.stride == 53 && g_gated.format == ZERO_CKPT_E4M3);
  EXPECT(g_gated.c_out.codes == nullptr && g_gated.c_up.code_stride == 72 && g_gated.width == 70);
  up.format = ZERO_CKPT_INT8;
  EXPECT(zero_gated_ffn(&f, nullptr) == ZERO_E_INVAL && g_launches == 1);
  up.format = ZERO_CKPT_E4M3;
  g_fits = false;
  EXPECT(zero_gated_ffn(&f, nullptr) == ZERO_E_RANGE && g_launches == 1);
  g_fits = true;
  g_result = hipErrorOutOfMemory;
  EXPECT(zero_gated_ffn(&f, nullptr) == ZERO_E_DEVICE && g_launches == 2);
  g_result = hipSuccess;

  zero_gated_ffn_grad_t g = {};
  g.dtype = ZERO_F16;
  g.rows = 6;
  g.cols = 50;
  g.width = 70;
  g.dout = p;
  g.dout_stride = 70;
  g.ckpt_gate = &gate;
  g.ckpt_up = &up;
  g.ckpt_x = &kx;
  g.dw = p + 4;
  g.dw_stride = 60;
  g.dw_dtype = ZERO_F32;
  g.workspace = p;
  g.workspace_bytes = 4096;
  EXPECT(zero_gated_ffn_grad(&g, nullptr) == ZERO_OK && g_launches == 3);   // no w: dw alone
  EXPECT(g_grad.dx.p == nullptr && g_grad.dw_dtype == ZERO_F32 && g_grad.c_x.codes == u);
  g.dx = p;
  g.dx_stride = 50;
  EXPECT(zero_gated_ffn_grad(&g, nullptr) == ZERO_E_INVAL);
  g.w = p;
  g.w_stride = 50;
  EXPECT(zero_gated_ffn_grad(&g, nullptr) == ZERO_OK && g_launches == 4);
  g.workspace_bytes = 4095;
  EXPECT(zero_gated_ffn_grad(&g, nullptr) == ZERO_E_RANGE && g_launches == 4);

  zero_loss_t l = {};
  l.dtype = ZERO_F16;
  l.rows = 5;
  l.cols = 33;
  l.vocab = 100;
  l.x = p;
  l.x_stride = 33;
  l.w = p;
  l.w_stride = 40;
  l.loss = reinterpret_cast<float*>(p);
  l.scale = 0.25;
  l.workspace = p;
  l.workspace_bytes = 4096;
  EXPECT(zero_vocab_loss(&l, p, 4, nullptr) == ZERO_OK && g_launches == 5);
  EXPECT(g_loss.top == 0 && g_loss.tau == 1.0f && !g_loss.ids_64 && g_loss.ids_stride == 1);
  l.dx = p;
  l.dx_stride = 33;
  EXPECT(zero_vocab_loss(&l, p, 8, nullptr) == ZERO_E_RANGE && g_launches == 5);
  l.workspace_bytes = 5120;
  EXPECT(zero_vocab_loss(&l, p, 8, nullptr) == ZERO_OK && g_launches == 6 && g_loss.ids_64);
  zero_top_logits_t t = {16, p, 17, 4, p, 18, ZERO_BF16, 2.5};
  EXPECT(zero_distill_loss(&l, &t, nullptr) == ZERO_OK && g_launches == 7);
  EXPECT(g_loss.top == 16 && g_loss.tau == 2.5f && g_loss.ids_stride == 17 &&
         g_loss.logits_stride == 18 && g_loss.logits_dtype == ZERO_BF16 && g_loss.scale == 0.25);
  t.temperature = NAN;
  EXPECT(zero_distill_loss(&l, &t, nullptr) == ZERO_E_INVAL && g_launches == 7);
  g_fits = false;
  EXPECT(zero_vocab_loss(&l, p, 8, nullptr) == ZERO_E_RANGE && g_launches == 7);
  if (!g_fail) printf("layer host check ok\n");
  return g_fail;
}
