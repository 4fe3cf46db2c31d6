// Host side of the activation entry points: argument validation and launches.
// Every check runs before the first HIP call, so a rejected call enqueues
// nothing.
#include <math.h>

#include "act/launch.h"
#include "zero.h"

namespace {

using zero::fail;
using zero::ok;
using zero::act::Ckpt;
using zero::act::Rows;

typedef unsigned long long ull;

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// rows x cols elements with rows `stride` apart, of up to 4 bytes each: the last
// element's offset in bytes stays far inside 64 bits.
int check_matrix(const char* name, uint64_t rows, uint64_t cols, uint64_t stride) {
  if (rows > 1 && stride < cols)
    return fail(ZERO_E_RANGE, "%s: row stride %llu < %llu columns", name, (ull)stride, (ull)cols);
  constexpr uint64_t kMost = 1ull << 60;
  if (cols > kMost || (rows > 1 && stride > (kMost - cols) / (rows - 1)))
    return fail(ZERO_E_RANGE, "%s: size overflows", name);
  return ZERO_OK;
}

int check_ckpt(const char* name, const zero_ckpt_t* c) {
  if (!c) return fail(ZERO_E_INVAL, "%s is NULL", name);
  if (c->format != ZERO_CKPT_INT8 && c->format != ZERO_CKPT_E4M3)
    return fail(ZERO_E_INVAL, "%s: unknown format %d", name, c->format);
  if (c->rows == 0 || c->cols == 0) return ZERO_OK;
  if (!c->codes || !c->scales) return fail(ZERO_E_INVAL, "%s: codes or scales is NULL", name);
  if (c->cols > (1ull << 31)) return fail(ZERO_E_RANGE, "%s: more than 2^31 columns", name);
  int rc = check_matrix(name, c->rows, c->cols, c->code_stride);
  if (rc) return rc;
  return check_matrix(name, c->rows, (c->cols - 1) / ZERO_CKPT_BLOCK + 1, c->scale_stride);
}

Ckpt ckpt_of(const zero_ckpt_t* c) {
  Ckpt k;
  k.codes = c ? c->codes : nullptr;
  k.scales = c ? c->scales : nullptr;
  k.code_stride = c ? c->code_stride : 0;
  k.scale_stride = c ? c->scale_stride : 0;
  k.format = c ? c->format : ZERO_CKPT_INT8;
  return k;
}

Rows rows_of(const void* p, uint64_t stride) {
  Rows r;
  r.p = static_cast<uint16_t*>(const_cast<void*>(p));
  r.stride = stride;
  return r;
}

int device(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(ZERO_E_DEVICE, "%s launch: %s", what, hipGetErrorString(e));
  return ok();
}

int check_store(const void* x, int dtype, int most_dtype, uint64_t stride, const zero_ckpt_t* c) {
  int rc = check_ckpt("checkpoint", c);
  if (rc) return rc;
  if (dtype < ZERO_F16 || dtype > most_dtype) return fail(ZERO_E_INVAL, "unknown dtype %d", dtype);
  if (c->rows == 0 || c->cols == 0) return ZERO_OK;
  if (!x) return fail(ZERO_E_INVAL, "the matrix is NULL");
  if ((rc = check_matrix("matrix", c->rows, c->cols, stride))) return rc;
  if (!aligned(x, dtype == ZERO_F32 ? 4 : 2))
    return fail(ZERO_E_ALIGN, "the matrix is not aligned to its elements");
  return ZERO_OK;
}

zero::act::StoreLaunch store_of(const void* x, int dtype, uint64_t stride, const zero_ckpt_t* c) {
  zero::act::StoreLaunch L;
  L.c = ckpt_of(c);
  L.x = const_cast<void*>(x);
  L.x_stride = stride;
  L.dtype = dtype;
  L.rows = c->rows;
  L.cols = c->cols;
  return L;
}

// The checks that the norms' forward and backward share.
struct NormCall {
  int dtype;
  uint64_t rows, cols;
};

int check_dims(const NormCall& n) {
  if (n.dtype != ZERO_F16 && n.dtype != ZERO_BF16)
    return fail(ZERO_E_INVAL, "dtype must be fp16 or bf16");
  if (n.cols == 0) return fail(ZERO_E_INVAL, "cols must be > 0");
  if (n.cols > ZERO_NORM_MAX_COLS)
    return fail(ZERO_E_RANGE, "cols %llu exceeds %d", (ull)n.cols, ZERO_NORM_MAX_COLS);
  return ZERO_OK;
}

int check_rows(const NormCall& n, const char* name, const void* p, uint64_t stride) {
  if (!p) return ZERO_OK;
  int rc = check_matrix(name, n.rows, n.cols, stride);
  if (rc) return rc;
  if (!aligned(p, 2)) return fail(ZERO_E_ALIGN, "%s is not 2-byte aligned", name);
  return ZERO_OK;
}

int check_norm(const char* name, const zero_norm_t& n) {
  if (n.kind < ZERO_NORM_NONE || n.kind > ZERO_NORM_LAYER)
    return fail(ZERO_E_INVAL, "%s: unknown norm %d", name, n.kind);
  if (n.kind == ZERO_NORM_NONE) {
    if (n.weight || n.bias)
      return fail(ZERO_E_INVAL, "%s: a weight or bias without a norm", name);
    return ZERO_OK;
  }
  // in fp32 too: a smaller eps would let a row of zeros divide by zero
  const float eps = static_cast<float>(n.eps);
  if (!isfinite(n.eps) || !(eps > 0.f) || !isfinite(eps))
    return fail(ZERO_E_INVAL, "%s: eps must be finite and > 0 in fp32", name);
  if (!aligned(n.weight, 2) || !aligned(n.bias, 2))
    return fail(ZERO_E_ALIGN, "%s: weight or bias is not 2-byte aligned", name);
  return ZERO_OK;
}

int check_norm_ckpt(const NormCall& n, const char* name, const zero_ckpt_t* c) {
  if (!c) return ZERO_OK;
  if (c->rows != n.rows || c->cols != n.cols)
    return fail(ZERO_E_RANGE, "%s is %llu x %llu, the call %llu x %llu", name, (ull)c->rows,
                (ull)c->cols, (ull)n.rows, (ull)n.cols);
  return check_ckpt(name, c);
}

int check_gate(const NormCall& n, const void* gate, uint64_t stride) {
  if (gate && stride == 0) {
    if (!aligned(gate, 2)) return fail(ZERO_E_ALIGN, "gate is not 2-byte aligned");
    return ZERO_OK;
  }
  return check_rows(n, "gate", gate, stride);
}

int check_scale(double s) {
  if (!isfinite(s) || !isfinite(static_cast<float>(s)))
    return fail(ZERO_E_INVAL, "scale must be finite in fp32");
  return ZERO_OK;
}

zero::act::NormArgs norm_of(const zero_norm_t& n) {
  zero::act::NormArgs a;
  a.kind = n.kind;
  a.eps = static_cast<float>(n.eps);
  a.w = rows_of(n.weight, 0);
  a.b = rows_of(n.bias, 0);
  return a;
}

}  // namespace

extern "C" {

int zero_ckpt_write(const void* x, int dtype, uint64_t x_stride, const zero_ckpt_t* c,
                    void* hip_stream) {
  int rc = check_store(x, dtype, ZERO_BF16, x_stride, c);
  if (rc) return rc;
  if (c->rows == 0 || c->cols == 0) return ok();
  return device(zero::act::launch_ckpt_write(store_of(x, dtype, x_stride, c),
                                             static_cast<hipStream_t>(hip_stream)),
                "checkpoint write");
}

int zero_ckpt_read(const zero_ckpt_t* c, void* out, int dtype, uint64_t out_stride,
                   void* hip_stream) {
  int rc = check_store(out, dtype, ZERO_F32, out_stride, c);
  if (rc) return rc;
  if (c->rows == 0 || c->cols == 0) return ok();
  return device(zero::act::launch_ckpt_read(store_of(out, dtype, out_stride, c),
                                            static_cast<hipStream_t>(hip_stream)),
                "checkpoint read");
}

uint64_t zero_ckpt_weight_grad_workspace(uint64_t rows, uint64_t cols, uint64_t n) {
  constexpr uint64_t kMost = 1ull << 22;
  if (cols == 0 || n == 0 || cols > kMost || n > kMost || rows > (1ull << 60)) return 0;
  return zero::act::weight_grad_workspace(rows, cols, n);
}

int zero_ckpt_weight_grad(const zero_ckpt_t* x, const void* dy, int dtype, uint64_t n,
                          uint64_t dy_stride, void* dw, int dw_dtype, uint64_t dw_stride,
                          int accumulate, void* workspace, uint64_t workspace_bytes,
                          void* hip_stream) {
  int rc = check_ckpt("checkpoint", x);
  if (rc) return rc;
  if (dtype != ZERO_F16 && dtype != ZERO_BF16)
    return fail(ZERO_E_INVAL, "dy must be fp16 or bf16");
  if (dw_dtype != dtype && dw_dtype != ZERO_F32)
    return fail(ZERO_E_INVAL, "dw must have dy's type or fp32");
  if (accumulate != 0 && accumulate != 1) return fail(ZERO_E_INVAL, "accumulate must be 0 or 1");
  constexpr uint64_t kMost = 1ull << 22;
  if (n > kMost || x->cols > kMost)
    return fail(ZERO_E_RANGE, "n %llu or cols %llu exceeds 2^22", (ull)n, (ull)x->cols);
  if (n == 0 || x->cols == 0) return ok();
  if (x->rows == 0 && accumulate) return ok();
  if (!dw || (x->rows && !dy)) return fail(ZERO_E_INVAL, "dy or dw is NULL");
  if ((rc = check_matrix("dy", x->rows, n, dy_stride))) return rc;
  if ((rc = check_matrix("dw", n, x->cols, dw_stride))) return rc;
  if (!aligned(dy, 2) || !aligned(dw, dw_dtype == ZERO_F32 ? 4 : 2))
    return fail(ZERO_E_ALIGN, "dy or dw is not aligned to its elements");
  const uint64_t need = zero::act::weight_grad_workspace(x->rows, x->cols, n);
  if (need) {
    if (!workspace) return fail(ZERO_E_INVAL, "workspace is NULL, needs %llu bytes", (ull)need);
    if (workspace_bytes < need)
      return fail(ZERO_E_RANGE, "workspace holds %llu bytes, needs %llu", (ull)workspace_bytes,
                  (ull)need);
    if (!aligned(workspace, 16)) return fail(ZERO_E_ALIGN, "workspace is not 16-byte aligned");
  }
  zero::act::WeightGradLaunch L;
  L.x = ckpt_of(x);
  L.rows = x->rows;
  L.k = x->cols;
  L.n = n;
  L.dy = static_cast<const uint16_t*>(dy);
  L.dy_stride = dy_stride;
  L.dtype = dtype;
  L.dw = dw;
  L.dw_stride = dw_stride;
  L.dw_dtype = dw_dtype;
  L.accumulate = accumulate;
  L.partial = static_cast<float*>(workspace);
  return device(zero::act::launch_weight_grad(L, static_cast<hipStream_t>(hip_stream)),
                "weight gradient");
}

int zero_block_norm(const zero_block_norm_t* a, void* hip_stream) {
  if (!a) return fail(ZERO_E_INVAL, "argument is NULL");
  const NormCall n = {a->dtype, a->rows, a->cols};
  int rc;
  if ((rc = check_dims(n)) || (rc = check_norm("post", a->post)) ||
      (rc = check_norm("pre", a->pre)) || (rc = check_scale(a->scale)))
    return rc;
  if (!a->block && (a->gate || a->post.kind != ZERO_NORM_NONE || a->ckpt_block))
    return fail(ZERO_E_INVAL, "a gate, post norm or ckpt_block without a block");
  if ((a->pre.kind != ZERO_NORM_NONE) != (a->z != nullptr) && (a->rows || a->z))
    return fail(ZERO_E_INVAL, "z is given if and only if pre is a norm");
  if (a->ckpt_z && a->pre.kind == ZERO_NORM_NONE)
    return fail(ZERO_E_INVAL, "ckpt_z without a pre norm");
  if ((rc = check_rows(n, "res", a->res, a->res_stride)) ||
      (rc = check_rows(n, "block", a->block, a->block_stride)) ||
      (rc = check_gate(n, a->gate, a->gate_stride)) ||
      (rc = check_rows(n, "out", a->out, a->out_stride)) ||
      (rc = check_rows(n, "z", a->z, a->z_stride)) ||
      (rc = check_norm_ckpt(n, "ckpt_block", a->ckpt_block)) ||
      (rc = check_norm_ckpt(n, "ckpt_out", a->ckpt_out)) ||
      (rc = check_norm_ckpt(n, "ckpt_z", a->ckpt_z)))
    return rc;
  if (a->stats && !aligned(a->stats, 16))
    return fail(ZERO_E_ALIGN, "stats is not 16-byte aligned");
  if (a->rows > (1ull << 56)) return fail(ZERO_E_RANGE, "too many rows");
  if (a->rows == 0) return ok();
  if (!a->res) return fail(ZERO_E_INVAL, "res is NULL");
  if (!a->out && !a->z && !a->stats && !a->ckpt_block && !a->ckpt_out)
    return fail(ZERO_E_INVAL, "nothing to write");
  zero::act::BlockNormLaunch L;
  L.dtype = a->dtype;
  L.rows = a->rows;
  L.cols = static_cast<uint32_t>(a->cols);
  L.res = rows_of(a->res, a->res_stride);
  L.block = rows_of(a->block, a->block_stride);
  L.gate = rows_of(a->gate, a->gate_stride);
  L.out = rows_of(a->out, a->out_stride);
  L.z = rows_of(a->z, a->z_stride);
  L.post = norm_of(a->post);
  L.pre = norm_of(a->pre);
  L.scale = static_cast<float>(a->scale);
  L.stats = a->stats;
  L.c_block = ckpt_of(a->ckpt_block);
  L.c_out = ckpt_of(a->ckpt_out);
  L.c_z = ckpt_of(a->ckpt_z);
  return device(zero::act::launch_block_norm(L, static_cast<hipStream_t>(hip_stream)),
                "block norm");
}

uint64_t zero_block_norm_grad_workspace(uint64_t rows, uint64_t cols) {
  if (cols == 0 || cols > ZERO_NORM_MAX_COLS || rows > (1ull << 56)) return 0;
  return zero::act::norm_grad_workspace(rows, cols);
}

int zero_block_norm_grad(const zero_block_norm_grad_t* a, void* hip_stream) {
  if (!a) return fail(ZERO_E_INVAL, "argument is NULL");
  const NormCall n = {a->dtype, a->rows, a->cols};
  int rc;
  if ((rc = check_dims(n)) || (rc = check_norm("post", a->post)) ||
      (rc = check_norm("pre", a->pre)) || (rc = check_scale(a->scale)))
    return rc;
  const bool pre = a->pre.kind != ZERO_NORM_NONE, post = a->post.kind != ZERO_NORM_NONE;
  if (!pre && (a->dz || a->dw_pre || a->db_pre))
    return fail(ZERO_E_INVAL, "dz, dw_pre or db_pre without a pre norm");
  if (!post && (a->dw_post || a->db_post))
    return fail(ZERO_E_INVAL, "dw_post or db_post without a post norm");
  if (a->dgate && !a->gate) return fail(ZERO_E_INVAL, "dgate without a gate");
  if (a->grad_dtype != a->dtype && a->grad_dtype != ZERO_F32)
    return fail(ZERO_E_INVAL, "grad_dtype must be dtype or fp32");
  if (a->accumulate != 0 && a->accumulate != 1)
    return fail(ZERO_E_INVAL, "accumulate must be 0 or 1");
  const bool gate_row = a->gate_stride == 0;
  const bool block = a->dblock || a->dgate || a->dw_post || a->db_post;
  const bool need_block = block && (post || a->dgate);
  if (a->rows && !a->dres && !block && !a->dw_pre && !a->db_pre)
    return fail(ZERO_E_INVAL, "no output");
  if ((rc = check_rows(n, "dout", a->dout, a->dout_stride)) ||
      (rc = check_rows(n, "dz", a->dz, a->dz_stride)) ||
      (rc = check_gate(n, a->gate, a->gate_stride)) ||
      (rc = check_rows(n, "dres", a->dres, a->dres_stride)) ||
      (rc = check_rows(n, "dblock", a->dblock, a->dblock_stride)) ||
      (rc = gate_row ? ZERO_OK : check_rows(n, "dgate", a->dgate, a->dgate_stride)) ||
      (rc = check_norm_ckpt(n, "ckpt_out", a->ckpt_out)) ||
      (rc = check_norm_ckpt(n, "ckpt_block", a->ckpt_block)))
    return rc;
  void* sums[zero::act::kSums];
  sums[zero::act::kDwPre] = a->dw_pre;
  sums[zero::act::kDwPost] = a->dw_post;
  sums[zero::act::kDbPre] = a->db_pre;
  sums[zero::act::kDbPost] = a->db_post;
  sums[zero::act::kDgate] = gate_row ? a->dgate : nullptr;
  bool any = false;
  for (void* p : sums) {
    any = any || p;
    if (!aligned(p, a->grad_dtype == ZERO_F32 ? 4 : 2))
      return fail(ZERO_E_ALIGN, "a parameter's gradient is not aligned to its elements");
  }
  if (a->stats && !aligned(a->stats, 16))
    return fail(ZERO_E_ALIGN, "stats is not 16-byte aligned");
  if (a->rows > (1ull << 56)) return fail(ZERO_E_RANGE, "too many rows");
  if (a->rows == 0 && (!any || a->accumulate)) return ok();
  if (a->rows) {
    if (pre && (!a->dz || !a->ckpt_out))
      return fail(ZERO_E_INVAL, "a pre norm needs dz and ckpt_out");
    if (need_block && !a->ckpt_block)
      return fail(ZERO_E_INVAL, "a post norm or dgate needs ckpt_block");
    if (pre && need_block && a->ckpt_out->format != a->ckpt_block->format)
      return fail(ZERO_E_INVAL, "ckpt_out and ckpt_block have different formats");
    if ((pre || (block && post)) && !a->stats) return fail(ZERO_E_INVAL, "a norm needs stats");
  }
  const uint64_t need = any ? zero::act::norm_grad_workspace(a->rows, a->cols) : 0;
  if (need) {
    if (!a->workspace)
      return fail(ZERO_E_INVAL, "workspace is NULL, needs %llu bytes", (ull)need);
    if (a->workspace_bytes < need)
      return fail(ZERO_E_RANGE, "workspace holds %llu bytes, needs %llu",
                  (ull)a->workspace_bytes, (ull)need);
    if (!aligned(a->workspace, 16))
      return fail(ZERO_E_ALIGN, "workspace is not 16-byte aligned");
  }
  zero::act::BlockNormGradLaunch L;
  L.dtype = a->dtype;
  L.rows = a->rows;
  L.cols = static_cast<uint32_t>(a->cols);
  L.dout = rows_of(a->dout, a->dout_stride);
  L.dz = rows_of(a->dz, a->dz_stride);
  L.gate = rows_of(a->gate, a->gate_stride);
  L.dres = rows_of(a->dres, a->dres_stride);
  L.dblock = rows_of(a->dblock, a->dblock_stride);
  L.dgate = rows_of(gate_row ? nullptr : a->dgate, a->dgate_stride);
  L.c_out = ckpt_of(pre ? a->ckpt_out : nullptr);
  L.c_block = ckpt_of(need_block ? a->ckpt_block : nullptr);
  L.format = pre ? a->ckpt_out->format : need_block ? a->ckpt_block->format : ZERO_CKPT_INT8;
  L.block = block;
  L.stats = a->stats;
  L.post = norm_of(a->post);
  L.pre = norm_of(a->pre);
  L.scale = static_cast<float>(a->scale);
  for (int i = 0; i < zero::act::kSums; ++i) L.sums[i] = sums[i];
  L.grad_dtype = a->grad_dtype;
  L.accumulate = a->accumulate;
  L.partial = static_cast<float*>(a->workspace);
  return device(zero::act::launch_block_norm_grad(L, static_cast<hipStream_t>(hip_stream)),
                "block norm gradient");
}

}  // extern "C"
