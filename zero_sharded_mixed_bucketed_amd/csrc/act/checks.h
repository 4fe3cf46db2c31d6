// Argument checks and conversions that the activation-side entry points share
// (internal to libzero).
#ifndef ZERO_ACT_CHECKS_H_
#define ZERO_ACT_CHECKS_H_

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act/launch.h"
#include "zero.h"

namespace zero {
namespace act {

typedef unsigned long long ull;

inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// rows x cols elements with rows `stride` apart, of up to 4 bytes each: the last
// element's offset in bytes stays far inside 64 bits.
inline int check_matrix(const char* name, uint64_t rows, uint64_t cols, uint64_t stride) {
  if (rows > 1 && stride < cols)
    return fail(ZERO_E_RANGE, "%s: row stride %llu < %llu columns", name, (ull)stride, (ull)cols);
  constexpr uint64_t kMost = 1ull << 60;
  if (cols > kMost || (rows > 1 && stride > (kMost - cols) / (rows - 1)))
    return fail(ZERO_E_RANGE, "%s: size overflows", name);
  return ZERO_OK;
}

inline int check_ckpt(const char* name, const zero_ckpt_t* c) {
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

inline Ckpt ckpt_of(const zero_ckpt_t* c) {
  Ckpt k;
  k.codes = c ? c->codes : nullptr;
  k.scales = c ? c->scales : nullptr;
  k.code_stride = c ? c->code_stride : 0;
  k.scale_stride = c ? c->scale_stride : 0;
  k.format = c ? c->format : ZERO_CKPT_INT8;
  return k;
}

inline Rows rows_of(const void* p, uint64_t stride) {
  Rows r;
  r.p = static_cast<uint16_t*>(const_cast<void*>(p));
  r.stride = stride;
  return r;
}

inline int device(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(ZERO_E_DEVICE, "%s launch: %s", what, hipGetErrorString(e));
  return ok();
}

}  // namespace act
}  // namespace zero

#endif  // ZERO_ACT_CHECKS_H_
