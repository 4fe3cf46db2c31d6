// Launch interfaces of a layer's gated block and of the losses over the vocabulary
// (internal to libzero).  Every argument has been checked by the C entry points before
// these are filled.
#ifndef ZERO_ACT_LAYER_H_
#define ZERO_ACT_LAYER_H_

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act/launch.h"

namespace zero {
namespace act {

constexpr int kSilu = 0, kGelu = 1, kGeluTanh = 2;  // ZERO_ACT_*

struct GatedLaunch {
  int dtype, act;
  uint64_t rows, cols, width;
  Rows x, w, out;               // w: 2 width rows
  Ckpt c_gate, c_up, c_out;     // absent: codes == nullptr
  int format;                   // of those given
};

hipError_t launch_gated_ffn(const GatedLaunch& a, hipStream_t stream);

struct GatedGradLaunch {
  int dtype, act;
  uint64_t rows, cols, width;
  Rows dout, w, dx;             // dx.p == nullptr: not wanted
  Ckpt c_gate, c_up, c_x;
  int format;                   // of c_gate and c_up
  void* dw;                     // 2 width x cols, or nullptr
  uint64_t dw_stride;
  int dw_dtype, accumulate;
  uint8_t* workspace;           // gated_grad_workspace bytes
};

uint64_t gated_grad_workspace(uint64_t rows, uint64_t cols, uint64_t width);
// Whether the products of these sizes (dx: the backward's) fit one launch each.
bool gated_fits(uint64_t rows, uint64_t cols, uint64_t width, bool dx);
hipError_t launch_gated_ffn_grad(const GatedGradLaunch& a, hipStream_t stream);

struct VocabLaunch {
  int dtype;
  uint64_t rows, cols, vocab;
  Rows x, w, dx;                // dx.p == nullptr: not wanted
  const void* ids;              // rows x top, ids_stride apart
  int ids_64;                   // 64-bit ids, or 32-bit ones
  uint64_t ids_stride;
  uint32_t top;                 // 0: one target a row, without a temperature
  const void* logits;           // teacher's, rows x top
  int logits_dtype;
  uint64_t logits_stride;
  const float* weights;         // rows, or nullptr
  float tau;
  double scale;
  float* loss;
  void* dw;                     // vocab x cols, or nullptr
  uint64_t dw_stride;
  int dw_dtype, accumulate;
  uint8_t* workspace;           // vocab_workspace bytes
};

uint64_t vocab_workspace(uint64_t rows, uint64_t cols, uint64_t vocab, uint32_t top, bool dx,
                         bool dw);
bool vocab_fits(uint64_t rows, uint64_t cols, uint64_t vocab, bool dx, bool dw);
hipError_t launch_vocab_loss(const VocabLaunch& a, hipStream_t stream);

constexpr uint64_t kMaxTop = 1024;   // ZERO_DISTILL_MAX_TOP

}  // namespace act
}  // namespace zero

#endif  // ZERO_ACT_LAYER_H_
