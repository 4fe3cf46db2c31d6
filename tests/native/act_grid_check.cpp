// The launches of the activation entry points over long inputs, recorded by
// stand-ins for the HIP runtime's launch calls (nothing runs on a device): each is
// within what HIP takes (fewer than 2^32 threads in a grid's dimension), together
// they cover every row once and in order, and the first that fails ends the call.
// Prints "act grid check ok" when every expectation holds.
#include <hip/hip_runtime.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include <vector>

#include "act/launch.h"
#include "zero.h"

namespace {

int g_fail = 0;
#define EXPECT(c)                                                                  \
  do {                                                                             \
    if (!(c)) {                                                                    \
      fprintf(stderr, "%s:%d: expectation failed: %s\n", __FILE__, __LINE__, #c);  \
      g_fail = 1;                                                                  \
    }                                                                              \
  } while (0)

// The first fields of the store's second kernel argument; the norms' is row0 alone.
struct Place {
  uint64_t row0;
  uint32_t units, segments, lanes;
};

struct Launch {
  dim3 grid, block;
  Place at;
  bool stored;
};

std::vector<Launch> g_launches;
dim3 g_grid, g_block;
size_t g_shared;
hipStream_t g_stream;
bool g_stores = false;         // the call under test is a store's
int g_fail_at = -1;            // the launch that fails, if any
hipError_t g_last = hipSuccess;

}  // namespace

extern "C" {

hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t shared, hipStream_t s) {
  g_grid = grid;
  g_block = block;
  g_shared = shared;
  g_stream = s;
  return hipSuccess;
}

hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, hipStream_t* s) {
  *grid = g_grid;
  *block = g_block;
  *shared = g_shared;
  *s = g_stream;
  return hipSuccess;
}

hipError_t hipLaunchKernel(const void*, dim3 grid, dim3 block, void** args, size_t, hipStream_t) {
  Launch l = {grid, block, {}, g_stores};
  if (g_stores) l.at = *static_cast<const Place*>(args[1]);
  else l.at.row0 = *static_cast<const uint64_t*>(args[1]);
  const bool fails = static_cast<int>(g_launches.size()) == g_fail_at;
  g_launches.push_back(l);
  if (fails) g_last = hipErrorInvalidConfiguration;
  return fails ? g_last : hipSuccess;
}

hipError_t hipGetLastError() {
  const hipError_t e = g_last;
  g_last = hipSuccess;
  return e;
}

hipError_t hipExtGetLastError() { return hipGetLastError(); }
const char* hipGetErrorString(hipError_t) { return "an error"; }
void** __hipRegisterFatBinary(const void*) { return nullptr; }
void __hipRegisterFunction(void**, const void*, char*, const char*, unsigned, void*, void*, void*,
                           void*, int*) {}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
void __hipUnregisterFatBinary(void**) {}

}  // extern "C"

namespace zero {
int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vfprintf(stdout, fmt, ap);
  va_end(ap);
  fputc('\n', stdout);
  return code;
}
int ok() { return ZERO_OK; }
}  // namespace zero

namespace {

char* const kAt = reinterpret_cast<char*>(static_cast<uintptr_t>(1) << 40);  // never read

void within_hip() {
  for (const Launch& l : g_launches) {
    EXPECT(static_cast<uint64_t>(l.grid.x) * l.block.x < 1ull << 32);
    EXPECT(l.grid.x > 0 && l.grid.y == 1 && l.grid.z == 1 && l.block.y == 1 && l.block.z == 1);
  }
}

int norm(uint64_t rows, uint64_t cols) {
  g_launches.clear();
  g_stores = false;
  zero_block_norm_t a = {};
  a.dtype = ZERO_F16;
  a.rows = rows;
  a.cols = cols;
  a.res = kAt;
  a.res_stride = cols;
  a.pre.kind = ZERO_NORM_RMS;
  a.pre.eps = 1e-5;
  a.z = kAt;
  a.z_stride = cols;
  a.scale = 1.0;
  return zero_block_norm(&a, nullptr);
}

void norm_covers(uint64_t rows, uint64_t cols, size_t least) {
  EXPECT(norm(rows, cols) == ZERO_OK);
  within_hip();
  EXPECT(g_launches.size() >= least);
  uint64_t next = 0;
  for (const Launch& l : g_launches) {   // a workgroup a row
    EXPECT(l.at.row0 == next);
    next += l.grid.x;
  }
  EXPECT(next == rows);
}

int store(bool read, uint64_t rows, uint64_t cols) {
  g_launches.clear();
  g_stores = true;
  uint8_t* u = reinterpret_cast<uint8_t*>(kAt);
  const zero_ckpt_t c = {u, u, rows, cols, cols, (cols - 1) / 32 + 1, ZERO_CKPT_INT8};
  return read ? zero_ckpt_read(&c, kAt, ZERO_F32, cols, nullptr)
              : zero_ckpt_write(kAt, ZERO_BF16, cols, &c, nullptr);
}

void store_covers(uint64_t rows, uint64_t cols, size_t least) {
  for (const bool read : {false, true}) {
    EXPECT(store(read, rows, cols) == ZERO_OK);
    within_hip();
    EXPECT(g_launches.size() >= least);
    uint64_t next = 0;
    for (const Launch& l : g_launches) {   // 256 threads, four units of work a wave
      EXPECT(l.at.row0 == next);
      EXPECT(l.block.x == 256 && l.grid.x == (static_cast<uint64_t>(l.at.units) + 15) / 16);
      EXPECT(l.at.segments * 512ull >= cols || l.at.segments == 1);
      if (l.at.segments == 1 && l.at.lanes < 64) EXPECT(l.at.lanes * 8ull >= cols);
      EXPECT(l.at.units % l.at.segments == 0);
      next += static_cast<uint64_t>(l.at.units) / l.at.segments *
              (l.at.segments == 1 ? 64 / l.at.lanes : 1);
    }
    // a unit of narrow rows may end past the last one
    EXPECT(next >= rows && next < rows + 64);
  }
}

}  // namespace

int main() {
  // rows of one, two and four waves, at the most of one launch and beyond it
  for (const uint64_t cols : {1, 72, 512, 4096}) {
    norm_covers(1, cols, 1);
    norm_covers((1ull << 26) - 1, cols, 1);
    norm_covers(1ull << 26, cols, 1);
    norm_covers((1ull << 26) + 5, cols, 2);
    norm_covers((1ull << 31) + 7, cols, 33);
  }
  for (const uint64_t cols : {4097, 8192}) {
    norm_covers((1ull << 25) - 1, cols, 1);
    norm_covers((1ull << 25) + 3, cols, 2);
  }
  for (const uint64_t cols : {8193, 16384}) {
    norm_covers((1ull << 24) - 1, cols, 1);
    norm_covers((1ull << 24) + 1, cols, 2);
  }

  // 16 rows of up to 32 columns a unit, one row of 257 to 512, rows of many units
  store_covers(1, 1, 1);
  store_covers((1ull << 26) + 5, 72, 1);
  store_covers((1ull << 32) - 256, 1, 1);
  store_covers((1ull << 32) + 17, 1, 2);
  store_covers((1ull << 34) + 1, 32, 5);
  store_covers((1ull << 28) + 3, 257, 2);
  store_covers((1ull << 28) + 3, 512, 2);
  store_covers((1ull << 27) + 3, 513, 2);
  store_covers(600, 1ull << 31, 10);

  // the first launch that fails ends the call, with its error
  g_fail_at = 0;
  EXPECT(norm((1ull << 26) + 5, 72) == ZERO_E_DEVICE && g_launches.size() == 1);
  EXPECT(store(false, (1ull << 32) + 17, 1) == ZERO_E_DEVICE && g_launches.size() == 1);
  g_fail_at = 1;
  EXPECT(norm((1ull << 31) + 7, 72) == ZERO_E_DEVICE && g_launches.size() == 2);
  if (g_fail) return 1;
  printf("act grid check ok\n");
  return 0;
}
