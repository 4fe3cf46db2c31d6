// Host side of the gated block's and the losses' entry points: argument validation and
// launches.  Every check runs before the first HIP call, so a rejected call enqueues
// nothing.
#include <math.h>

#include "act/checks.h"
#include "act/launch.h"
#include "act/layer.h"
#include "zero.h"

namespace {

using namespace zero::act;
using zero::fail;
using zero::ok;

constexpr uint64_t kMostRows = 1ull << 25, kMostCols = 1ull << 22, kMostVocab = 1ull << 24;

int check_dtype(int dtype) {
  if (dtype != ZERO_F16 && dtype != ZERO_BF16)
    return fail(ZERO_E_INVAL, "dtype must be fp16 or bf16");
  return ZERO_OK;
}

int check_dim(const char* name, uint64_t n, uint64_t most) {
  if (n == 0) return fail(ZERO_E_INVAL, "%s must be > 0", name);
  if (n > most) return fail(ZERO_E_RANGE, "%s %llu exceeds %llu", name, (ull)n, (ull)most);
  return ZERO_OK;
}

// A 16-bit matrix; `needed` with rows that exist.
int check_16(const char* name, const void* p, uint64_t rows, uint64_t cols, uint64_t stride,
             bool needed) {
  if (!p) {
    if (needed && rows) return fail(ZERO_E_INVAL, "%s is NULL", name);
    return ZERO_OK;
  }
  int rc = check_matrix(name, rows, cols, stride);
  if (rc) return rc;
  if (!aligned(p, 2)) return fail(ZERO_E_ALIGN, "%s is not 2-byte aligned", name);
  return ZERO_OK;
}

int check_dw(const void* dw, int dw_dtype, int dtype, uint64_t rows, uint64_t cols,
             uint64_t stride, int accumulate) {
  if (accumulate != 0 && accumulate != 1)
    return fail(ZERO_E_INVAL, "accumulate must be 0 or 1");
  if (!dw) return ZERO_OK;
  if (dw_dtype != dtype && dw_dtype != ZERO_F32)
    return fail(ZERO_E_INVAL, "dw must have the call's type or fp32");
  int rc = check_matrix("dw", rows, cols, stride);
  if (rc) return rc;
  if (!aligned(dw, dw_dtype == ZERO_F32 ? 4 : 2))
    return fail(ZERO_E_ALIGN, "dw is not aligned to its elements");
  return ZERO_OK;
}

int check_workspace(const void* p, uint64_t bytes, uint64_t need) {
  if (need == 0) return ZERO_OK;
  if (!p) return fail(ZERO_E_INVAL, "workspace is NULL, needs %llu bytes", (ull)need);
  if (bytes < need)
    return fail(ZERO_E_RANGE, "workspace holds %llu bytes, needs %llu", (ull)bytes, (ull)need);
  if (!aligned(p, 16)) return fail(ZERO_E_ALIGN, "workspace is not 16-byte aligned");
  return ZERO_OK;
}

// A checkpoint that may be absent, of rows x cols and, if another came first, its format.
int check_held(const char* name, const zero_ckpt_t* c, uint64_t rows, uint64_t cols, int* format) {
  if (!c) return ZERO_OK;
  if (c->rows != rows || c->cols != cols)
    return fail(ZERO_E_RANGE, "%s is %llu x %llu, the call %llu x %llu", name, (ull)c->rows,
                (ull)c->cols, (ull)rows, (ull)cols);
  int rc = check_ckpt(name, c);
  if (rc) return rc;
  if (format && *format >= 0 && *format != c->format)
    return fail(ZERO_E_INVAL, "%s has another format than the call's other checkpoints", name);
  if (format) *format = c->format;
  return ZERO_OK;
}

int check_gated(int dtype, int act, uint64_t rows, uint64_t cols, uint64_t width) {
  int rc;
  if ((rc = check_dtype(dtype)) || (rc = check_dim("cols", cols, kMostCols)) ||
      (rc = check_dim("width", width, kMostCols)))
    return rc;
  if (act < ZERO_ACT_SILU || act > ZERO_ACT_GELU_TANH)
    return fail(ZERO_E_INVAL, "unknown activation %d", act);
  if (rows > kMostRows)
    return fail(ZERO_E_RANGE, "rows %llu exceeds %llu", (ull)rows, (ull)kMostRows);
  return ZERO_OK;
}

bool gated_sizes(uint64_t rows, uint64_t cols, uint64_t width) {
  return rows <= kMostRows && cols && cols <= kMostCols && width && width <= kMostCols;
}

bool loss_sizes(uint64_t rows, uint64_t cols, uint64_t vocab) {
  return rows <= kMostRows && cols && cols <= kMostCols && vocab && vocab <= kMostVocab;
}

// The checks that both losses share.
int check_loss(const zero_loss_t* a) {
  if (!a) return fail(ZERO_E_INVAL, "argument is NULL");
  int rc;
  if ((rc = check_dtype(a->dtype)) || (rc = check_dim("cols", a->cols, kMostCols)) ||
      (rc = check_dim("vocab", a->vocab, kMostVocab)))
    return rc;
  if (a->rows > kMostRows)
    return fail(ZERO_E_RANGE, "rows %llu exceeds %llu", (ull)a->rows, (ull)kMostRows);
  if (!isfinite(a->scale) || !isfinite(static_cast<float>(a->scale)))
    return fail(ZERO_E_INVAL, "scale must be finite in fp32");
  if ((rc = check_16("x", a->x, a->rows, a->cols, a->x_stride, true)) ||
      (rc = check_16("w", a->w, a->rows ? a->vocab : 0, a->cols, a->w_stride, true)) ||
      (rc = check_16("dx", a->dx, a->rows, a->cols, a->dx_stride, false)) ||
      (rc = check_dw(a->dw, a->dw_dtype, a->dtype, a->vocab, a->cols, a->dw_stride,
                     a->accumulate)))
    return rc;
  if (!aligned(a->weights, 4) || !aligned(a->loss, 4))
    return fail(ZERO_E_ALIGN, "weights or loss is not 4-byte aligned");
  if (a->rows && !a->loss) return fail(ZERO_E_INVAL, "loss is NULL");
  if (!vocab_fits(a->rows, a->cols, a->vocab, a->dx != nullptr, a->dw != nullptr))
    return fail(ZERO_E_RANGE, "a product of these sizes is too large for one launch");
  return ZERO_OK;
}

int check_ids(const char* name, const void* ids, int id_bytes, uint64_t rows) {
  if (id_bytes != 4 && id_bytes != 8) return fail(ZERO_E_INVAL, "id_bytes must be 4 or 8");
  if (!ids && rows) return fail(ZERO_E_INVAL, "%s is NULL", name);
  if (!aligned(ids, id_bytes))
    return fail(ZERO_E_ALIGN, "%s is not aligned to its elements", name);
  return ZERO_OK;
}

// The workspace check and the launch.
int run_loss(const zero_loss_t* a, VocabLaunch& L, void* hip_stream, const char* what) {
  if (a->rows == 0 && (!a->dw || a->accumulate)) return ok();
  const uint64_t need =
      vocab_workspace(a->rows, a->cols, a->vocab, L.top, a->dx != nullptr, a->dw != nullptr);
  const int rc = check_workspace(a->workspace, a->workspace_bytes, need);
  if (rc) return rc;
  L.dtype = a->dtype;
  L.rows = a->rows;
  L.cols = a->cols;
  L.vocab = a->vocab;
  L.x = rows_of(a->x, a->x_stride);
  L.w = rows_of(a->w, a->w_stride);
  L.dx = rows_of(a->dx, a->dx_stride);
  L.weights = a->weights;
  L.scale = a->scale;
  L.loss = a->loss;
  L.dw = a->dw;
  L.dw_stride = a->dw_stride;
  L.dw_dtype = a->dw_dtype;
  L.accumulate = a->accumulate;
  L.workspace = static_cast<uint8_t*>(a->workspace);
  return device(launch_vocab_loss(L, static_cast<hipStream_t>(hip_stream)), what);
}

}  // namespace

extern "C" {

int zero_gated_ffn(const zero_gated_ffn_t* a, void* hip_stream) {
  if (!a) return fail(ZERO_E_INVAL, "argument is NULL");
  int rc = check_gated(a->dtype, a->act, a->rows, a->cols, a->width);
  if (rc) return rc;
  int format = -1;
  if ((rc = check_16("x", a->x, a->rows, a->cols, a->x_stride, true)) ||
      (rc = check_16("w", a->w, a->rows ? 2 * a->width : 0, a->cols, a->w_stride, true)) ||
      (rc = check_16("out", a->out, a->rows, a->width, a->out_stride, false)) ||
      (rc = check_held("ckpt_gate", a->ckpt_gate, a->rows, a->width, &format)) ||
      (rc = check_held("ckpt_up", a->ckpt_up, a->rows, a->width, &format)) ||
      (rc = check_held("ckpt_out", a->ckpt_out, a->rows, a->width, &format)))
    return rc;
  if (a->rows == 0) return ok();
  if (!a->out && !a->ckpt_gate && !a->ckpt_up && !a->ckpt_out)
    return fail(ZERO_E_INVAL, "nothing to write");
  if (!gated_fits(a->rows, a->cols, a->width, false))
    return fail(ZERO_E_RANGE, "a product of these sizes is too large for one launch");
  GatedLaunch L;
  L.dtype = a->dtype;
  L.act = a->act;
  L.rows = a->rows;
  L.cols = a->cols;
  L.width = a->width;
  L.x = rows_of(a->x, a->x_stride);
  L.w = rows_of(a->w, a->w_stride);
  L.out = rows_of(a->out, a->out_stride);
  L.c_gate = ckpt_of(a->ckpt_gate);
  L.c_up = ckpt_of(a->ckpt_up);
  L.c_out = ckpt_of(a->ckpt_out);
  L.format = format < 0 ? ZERO_CKPT_INT8 : format;
  return device(launch_gated_ffn(L, static_cast<hipStream_t>(hip_stream)), "gated block");
}

uint64_t zero_gated_ffn_grad_workspace(uint64_t rows, uint64_t cols, uint64_t width) {
  if (!gated_sizes(rows, cols, width)) return 0;
  return gated_grad_workspace(rows, cols, width);
}

int zero_gated_ffn_grad(const zero_gated_ffn_grad_t* a, void* hip_stream) {
  if (!a) return fail(ZERO_E_INVAL, "argument is NULL");
  int rc = check_gated(a->dtype, a->act, a->rows, a->cols, a->width);
  if (rc) return rc;
  int format = -1;
  if ((rc = check_16("dout", a->dout, a->rows, a->width, a->dout_stride, true)) ||
      (rc = check_16("w", a->w, a->rows ? 2 * a->width : 0, a->cols, a->w_stride,
                     a->dx != nullptr)) ||
      (rc = check_16("dx", a->dx, a->rows, a->cols, a->dx_stride, false)) ||
      (rc = check_held("ckpt_gate", a->ckpt_gate, a->rows, a->width, &format)) ||
      (rc = check_held("ckpt_up", a->ckpt_up, a->rows, a->width, &format)) ||
      (rc = check_held("ckpt_x", a->ckpt_x, a->rows, a->cols, nullptr)) ||
      (rc = check_dw(a->dw, a->dw_dtype, a->dtype, 2 * a->width, a->cols, a->dw_stride,
                     a->accumulate)))
    return rc;
  if (a->rows == 0 && (!a->dw || a->accumulate)) return ok();
  if (!a->dx && !a->dw) return fail(ZERO_E_INVAL, "no output");
  if (a->rows && (!a->ckpt_gate || !a->ckpt_up))
    return fail(ZERO_E_INVAL, "ckpt_gate or ckpt_up is NULL");
  if (a->rows && a->dw && !a->ckpt_x) return fail(ZERO_E_INVAL, "dw needs ckpt_x");
  if (!gated_fits(a->rows, a->cols, a->width, true))
    return fail(ZERO_E_RANGE, "a product of these sizes is too large for one launch");
  const uint64_t need = gated_grad_workspace(a->rows, a->cols, a->width);
  if ((rc = check_workspace(a->workspace, a->workspace_bytes, need))) return rc;
  GatedGradLaunch L;
  L.dtype = a->dtype;
  L.act = a->act;
  L.rows = a->rows;
  L.cols = a->cols;
  L.width = a->width;
  L.dout = rows_of(a->dout, a->dout_stride);
  L.w = rows_of(a->w, a->w_stride);
  L.dx = rows_of(a->dx, a->dx_stride);
  L.c_gate = ckpt_of(a->ckpt_gate);
  L.c_up = ckpt_of(a->ckpt_up);
  L.c_x = ckpt_of(a->ckpt_x);
  L.format = format < 0 ? ZERO_CKPT_INT8 : format;
  L.dw = a->dw;
  L.dw_stride = a->dw_stride;
  L.dw_dtype = a->dw_dtype;
  L.accumulate = a->accumulate;
  L.workspace = static_cast<uint8_t*>(a->workspace);
  return device(launch_gated_ffn_grad(L, static_cast<hipStream_t>(hip_stream)),
                "gated block gradient");
}

uint64_t zero_loss_workspace(uint64_t rows, uint64_t cols, uint64_t vocab, uint32_t top,
                             int with_dx, int with_dw) {
  if (!loss_sizes(rows, cols, vocab) || top > ZERO_DISTILL_MAX_TOP) return 0;
  return vocab_workspace(rows, cols, vocab, top, with_dx != 0, with_dw != 0);
}

int zero_vocab_loss(const zero_loss_t* a, const void* targets, int id_bytes, void* hip_stream) {
  int rc;
  if ((rc = check_loss(a)) || (rc = check_ids("targets", targets, id_bytes, a->rows))) return rc;
  VocabLaunch L = {};
  L.ids = targets;
  L.ids_64 = id_bytes == 8;
  L.ids_stride = 1;
  L.tau = 1.0f;
  return run_loss(a, L, hip_stream, "vocabulary loss");
}

int zero_distill_loss(const zero_loss_t* a, const zero_top_logits_t* t, void* hip_stream) {
  int rc;
  if ((rc = check_loss(a))) return rc;
  if (!t) return fail(ZERO_E_INVAL, "argument is NULL");
  if (t->top == 0 || t->top > ZERO_DISTILL_MAX_TOP)
    return fail(ZERO_E_INVAL, "top must be 1 to %d", ZERO_DISTILL_MAX_TOP);
  const float tau = static_cast<float>(t->temperature);
  if (!isfinite(t->temperature) || !(tau > 0.f) || !isfinite(1.0f / tau) ||
      !isfinite(tau * tau) || !isfinite(static_cast<float>(a->scale * t->temperature)))
    return fail(ZERO_E_INVAL, "temperature must be > 0 and, with its square, finite in fp32");
  if (t->logits_dtype < ZERO_F16 || t->logits_dtype > ZERO_F32)
    return fail(ZERO_E_INVAL, "unknown dtype %d", t->logits_dtype);
  if ((rc = check_ids("ids", t->ids, t->id_bytes, a->rows))) return rc;
  if (!t->logits && a->rows) return fail(ZERO_E_INVAL, "logits is NULL");
  if (!aligned(t->logits, t->logits_dtype == ZERO_F32 ? 4 : 2))
    return fail(ZERO_E_ALIGN, "logits is not aligned to its elements");
  if ((rc = check_matrix("ids", a->rows, t->top, t->ids_stride)) ||
      (rc = check_matrix("logits", a->rows, t->top, t->logits_stride)))
    return rc;
  VocabLaunch L = {};
  L.ids = t->ids;
  L.ids_64 = t->id_bytes == 8;
  L.ids_stride = t->ids_stride;
  L.top = t->top;
  L.logits = t->logits;
  L.logits_dtype = t->logits_dtype;
  L.logits_stride = t->logits_stride;
  L.tau = tau;
  return run_loss(a, L, hip_stream, "distillation loss");
}

}  // extern "C"
