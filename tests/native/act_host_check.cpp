// The host side of the activation entry points under sanitizers, with stand-ins
// for the kernels: every refusal happens before a launch, and what is launched has
// the arguments the call gave.  Prints "act host check ok" when every expectation
// holds.
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "act/launch.h"
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

static zero::act::StoreLaunch g_store;
static zero::act::BlockNormLaunch g_norm;
static zero::act::BlockNormGradLaunch g_grad;
static zero::act::WeightGradLaunch g_weight;

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
  return hipSuccess;
}
hipError_t launch_ckpt_write(const StoreLaunch& a, hipStream_t) { return keep(g_store, a); }
hipError_t launch_ckpt_read(const StoreLaunch& a, hipStream_t) { return keep(g_store, a); }
hipError_t launch_block_norm(const BlockNormLaunch& a, hipStream_t) { return keep(g_norm, a); }
hipError_t launch_block_norm_grad(const BlockNormGradLaunch& a, hipStream_t) {
  return keep(g_grad, a);
}
hipError_t launch_weight_grad(const WeightGradLaunch& a, hipStream_t) { return keep(g_weight, a); }
uint64_t norm_grad_workspace(uint64_t rows, uint64_t cols) { return rows * cols; }
uint64_t weight_grad_workspace(uint64_t rows, uint64_t, uint64_t) { return rows > 100 ? 4096 : 0; }
}  // namespace act
}  // namespace zero

int main() {
  char* p = reinterpret_cast<char*>(static_cast<uintptr_t>(0x100000));
  uint8_t* u = reinterpret_cast<uint8_t*>(p);

  // checkpoints
  zero_ckpt_t k = {u, u + 0x1000, 6, 70, 72, 5, ZERO_CKPT_E4M3};
  EXPECT(zero_ckpt_write(p + 2, ZERO_BF16, 71, &k, nullptr) == ZERO_OK && g_launches == 1);
  EXPECT(g_store.rows == 6 && g_store.cols == 70 && g_store.x == p + 2 && g_store.x_stride == 71 &&
         g_store.dtype == ZERO_BF16 && g_store.c.code_stride == 72 &&
         g_store.c.scale_stride == 5 && g_store.c.format == ZERO_CKPT_E4M3);
  EXPECT(zero_ckpt_read(&k, p, ZERO_F32, 70, nullptr) == ZERO_OK && g_launches == 2);
  k.code_stride = 69;
  EXPECT(zero_ckpt_write(p, ZERO_F16, 70, &k, nullptr) == ZERO_E_RANGE);
  k.rows = 1;  // a single row needs no stride
  EXPECT(zero_ckpt_write(p, ZERO_F16, 0, &k, nullptr) == ZERO_OK && g_launches == 3);
  k.rows = UINT64_MAX;
  k.code_stride = UINT64_MAX;
  EXPECT(zero_ckpt_write(p, ZERO_F16, 70, &k, nullptr) == ZERO_E_RANGE);
  k.rows = 4;
  k.cols = (1ull << 31) + 1;
  k.code_stride = 1ull << 33;
  k.scale_stride = 1ull << 33;
  EXPECT(zero_ckpt_write(p, ZERO_F16, 1ull << 33, &k, nullptr) == ZERO_E_RANGE);
  k.rows = 0;
  k.codes = nullptr;
  EXPECT(zero_ckpt_read(&k, nullptr, ZERO_F16, 0, nullptr) == ZERO_OK && g_launches == 3);

  // the weight gradient
  zero_ckpt_t x = {u, u + 0x1000, 50, 70, 70, 3, ZERO_CKPT_INT8};
  EXPECT(zero_ckpt_weight_grad(&x, p, ZERO_F16, 9, 9, p, ZERO_F32, 70, 1, nullptr, 0, nullptr) ==
             ZERO_OK && g_launches == 4);
  EXPECT(g_weight.rows == 50 && g_weight.k == 70 && g_weight.n == 9 && g_weight.accumulate == 1 &&
         g_weight.dw_dtype == ZERO_F32);
  x.rows = 200;
  EXPECT(zero_ckpt_weight_grad(&x, p, ZERO_F16, 9, 9, p, ZERO_F16, 70, 0, nullptr, 0, nullptr) ==
         ZERO_E_INVAL);
  EXPECT(zero_ckpt_weight_grad(&x, p, ZERO_F16, 9, 9, p, ZERO_F16, 70, 0, p, 4095, nullptr) ==
         ZERO_E_RANGE);
  EXPECT(zero_ckpt_weight_grad(&x, p, ZERO_F16, 9, 9, p, ZERO_F16, 70, 0, p, 4096, nullptr) ==
             ZERO_OK && g_launches == 5);
  EXPECT(zero_ckpt_weight_grad_workspace(200, 70, 9) == 4096);
  EXPECT(zero_ckpt_weight_grad_workspace(200, 70, (1ull << 22) + 1) == 0);

  // norms
  zero_norm_t rms = {ZERO_NORM_RMS, 1e-5, p, nullptr}, none = {ZERO_NORM_NONE, 0, nullptr, nullptr};
  zero_ckpt_t c = {u, u + 0x1000, 5, 64, 64, 2, ZERO_CKPT_INT8};
  zero_block_norm_t f;
  memset(&f, 0, sizeof f);
  f.dtype = ZERO_F16;
  f.rows = 5;
  f.cols = 64;
  f.res = f.block = f.out = f.z = p;
  f.res_stride = f.block_stride = f.out_stride = f.z_stride = 64;
  f.scale = 0.5;
  f.post = f.pre = rms;
  f.ckpt_z = &c;
  EXPECT(zero_block_norm(&f, nullptr) == ZERO_OK && g_launches == 6);
  EXPECT(g_norm.scale == 0.5f && g_norm.c_z.codes == u && !g_norm.c_block.codes &&
         g_norm.gate.p == nullptr && g_norm.post.w.p && !g_norm.post.b.p);
  f.pre = none;
  EXPECT(zero_block_norm(&f, nullptr) == ZERO_E_INVAL);
  f.z = nullptr;
  EXPECT(zero_block_norm(&f, nullptr) == ZERO_E_INVAL);  // ckpt_z without a pre norm
  f.ckpt_z = nullptr;
  EXPECT(zero_block_norm(&f, nullptr) == ZERO_OK && g_launches == 7);
  f.rows = UINT64_MAX;
  EXPECT(zero_block_norm(&f, nullptr) == ZERO_E_RANGE);

  // their backward
  zero_block_norm_grad_t b;
  memset(&b, 0, sizeof b);
  b.dtype = b.grad_dtype = ZERO_F16;
  b.rows = 5;
  b.cols = 64;
  b.dz = b.dres = p;
  b.dz_stride = b.dres_stride = 64;
  b.scale = 1;
  b.pre = rms;
  b.post = none;
  b.ckpt_out = &c;
  b.stats = reinterpret_cast<const float*>(p);
  EXPECT(zero_block_norm_grad(&b, nullptr) == ZERO_OK && g_launches == 8);
  EXPECT(g_grad.block == 0 && g_grad.c_out.codes == u && !g_grad.c_block.codes);
  b.dw_pre = p;
  EXPECT(zero_block_norm_grad(&b, nullptr) == ZERO_E_INVAL);  // no workspace
  b.workspace = p;
  b.workspace_bytes = 5 * 64;
  EXPECT(zero_block_norm_grad(&b, nullptr) == ZERO_OK && g_launches == 9);
  zero_ckpt_t e = c;
  e.format = ZERO_CKPT_E4M3;
  b.post = rms;
  b.dblock = p;
  b.dblock_stride = 64;
  b.ckpt_block = &e;
  EXPECT(zero_block_norm_grad(&b, nullptr) == ZERO_E_INVAL);  // two formats
  b.ckpt_block = &c;
  EXPECT(zero_block_norm_grad(&b, nullptr) == ZERO_OK && g_grad.block == 1 && g_launches == 10);
  b.rows = c.rows = 0;
  b.accumulate = 1;
  EXPECT(zero_block_norm_grad(&b, nullptr) == ZERO_OK && g_launches == 10);

  if (g_fail) return 1;
  printf("act host check ok\n");
  return 0;
}
