// Launch interfaces of the activation-side kernels (internal to libzero).  Every
// argument has been checked by the C entry points before these are filled.
#ifndef ZERO_ACT_LAUNCH_H_
#define ZERO_ACT_LAUNCH_H_

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace zero {

// The error message of the calling thread (zero_last_error) and its status.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int ok();

namespace act {

// Workgroups of one launch, at most: HIP takes fewer than 2^32 threads in a grid's
// dimension.
constexpr uint64_t most_workgroups(uint32_t threads) { return 0xFFFFFFFFull / threads; }

// 8-bit checkpoint rows in device memory; codes == nullptr: none.
struct Ckpt {
  uint8_t* codes;
  uint8_t* scales;
  uint64_t code_stride, scale_stride;
  int format;
};

struct StoreLaunch {  // write: x -> c; read: c -> x
  Ckpt c;
  void* x;
  uint64_t x_stride;
  int dtype;
  uint64_t rows, cols;
};

hipError_t launch_ckpt_write(const StoreLaunch& a, hipStream_t stream);
hipError_t launch_ckpt_read(const StoreLaunch& a, hipStream_t stream);

// One 16-bit matrix of a row-wise kernel; p == nullptr: absent.
struct Rows {
  uint16_t* p;
  uint64_t stride;  // 0: the same row for every token
};

struct NormArgs {
  int kind;                     // ZERO_NORM_*
  float eps;
  Rows w, b;                    // one row each; absent: ones, zeros
};

struct BlockNormLaunch {
  int dtype;
  uint64_t rows;
  uint32_t cols;
  Rows res, block, gate, out, z;
  NormArgs post, pre;
  float scale;
  float* stats;                 // rows x 4
  Ckpt c_block, c_out, c_z;
};

hipError_t launch_block_norm(const BlockNormLaunch& a, hipStream_t stream);

// The parameter gradients of the backward, in this order.
constexpr int kSums = 5;
enum { kDwPre, kDwPost, kDbPre, kDbPost, kDgate };

struct BlockNormGradLaunch {
  int dtype;
  uint64_t rows;
  uint32_t cols;
  Rows dout, dz, gate, dres, dblock, dgate;  // dgate: per token
  Ckpt c_out, c_block;          // absent where not needed; both of `format`
  int format;
  int block;                    // an output on the block's side is wanted
  const float* stats;
  NormArgs post, pre;
  float scale;
  void* sums[kSums];            // nullable
  int grad_dtype, accumulate;
  float* partial;               // norm_grad_workspace bytes, or nullptr
  float* means;                 // inside it: two of each wide row
};

// Bytes of partial sums that launch_block_norm_grad needs at these sizes.
uint64_t norm_grad_workspace(uint64_t rows, uint64_t cols);
hipError_t launch_block_norm_grad(const BlockNormGradLaunch& a, hipStream_t stream);

// The widest row that the norms take: forward four waves of eight chunks a thread.
constexpr uint64_t kMaxNormCols = 16384;

struct WeightGradLaunch {
  Ckpt x;
  uint64_t rows, k, n;          // dw is n x k
  const uint16_t* dy;
  uint64_t dy_stride;
  int dtype;
  void* dw;
  uint64_t dw_stride;
  int dw_dtype, accumulate;
  float* partial;               // weight_grad_workspace bytes
};

uint64_t weight_grad_workspace(uint64_t rows, uint64_t k, uint64_t n);
hipError_t launch_weight_grad(const WeightGradLaunch& a, hipStream_t stream);

}  // namespace act
}  // namespace zero

#endif  // ZERO_ACT_LAUNCH_H_
