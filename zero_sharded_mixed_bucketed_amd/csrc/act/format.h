// Device arithmetic shared by the activation-side kernels: 16-bit loads and
// stores of 8-element chunks, the 8-bit checkpoint format, and sums over a
// wavefront.
//
// The checkpoint format: rows of 8-bit codes in blocks of 32 columns, one scale
// byte b per block that stands for 2^(b - 127), or for NaN if b = 255.  A scale that
// is a power of two makes every held value exactly representable in the 16-bit type
// it came from (7 significant bits of an int8 code, 4 of an e4m3 code, against 11 of
// fp16 and 8 of bf16), so whatever reads a checkpoint back rounds nothing a second
// time.
#ifndef ZERO_ACT_FORMAT_H_
#define ZERO_ACT_FORMAT_H_

#include <hip/hip_runtime.h>
#include <stdint.h>

#pragma clang fp contract(fast)

namespace zero {
namespace act {

constexpr int kF16 = 0, kBf16 = 1, kF32 = 2;   // ZERO_F16, ZERO_BF16, ZERO_F32
constexpr int kInt8 = 0, kE4m3 = 1;            // ZERO_CKPT_INT8, ZERO_CKPT_E4M3
constexpr int kBlock = 32;                     // ZERO_CKPT_BLOCK
constexpr int kChunk = 8;                      // columns a thread handles together
constexpr int kQuad = kBlock / kChunk;         // neighbouring lanes that share a block

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// The same where memory is aligned to its elements only: rows may start anywhere
// (an odd row length does that to every other row), and the chip loads and stores
// 16 bytes from any address.
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef u32x2 u32x2_at1 __attribute__((aligned(1)));
typedef f32x4 f32x4_at4 __attribute__((aligned(4)));

struct F16 { static constexpr int kType = kF16; };
struct Bf16 { static constexpr int kType = kBf16; };

// ------------------------------------------------------------ 16-bit values

template <typename T>
__device__ __forceinline__ float lo16(uint32_t w) {
  if constexpr (T::kType == kF16)
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(w)));
  else
    return __builtin_bit_cast(float, w << 16);
}

template <typename T>
__device__ __forceinline__ float hi16(uint32_t w) {
  if constexpr (T::kType == kF16)
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(w >> 16)));
  else
    return __builtin_bit_cast(float, w & 0xFFFF0000u);
}

// One rounding to nearest even per value.
template <typename T>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  const f2 v = {a, b};
  if constexpr (T::kType == kF16) {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, h2));
  } else {
    typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf2));
  }
}

// Keeps the compiler from carrying what it made from a packed value past this
// point (unpacking again is cheaper than holding twice the registers), and from
// unpacking one before it, where that would wait for a load.
template <typename V>
__device__ __forceinline__ void forget(V& w) {
  asm volatile("" : "+v"(w));
}

template <typename T>
__device__ __forceinline__ void unpack8(u32x4 w, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = lo16<T>(w[i]);
    x[2 * i + 1] = hi16<T>(w[i]);
  }
}

template <typename T>
__device__ __forceinline__ u32x4 pack8(const float (&x)[8]) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack16<T>(x[2 * i], x[2 * i + 1]);
  return w;
}

// Eight 16-bit elements of a row from column c < cols on; those from `cols` on are
// 0, and their memory is not touched.
__device__ __forceinline__ u32x4 load8(const uint16_t* row, uint64_t c, uint64_t cols) {
  if (c + kChunk <= cols) return *reinterpret_cast<const u32x4_at2*>(row + c);
  uint32_t e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = row[c + i < cols ? c + i : cols - 1];
  u32x4 w = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i >> 1] |= (c + i < cols ? e[i] : 0u) << (16 * (i & 1));
  return w;
}

__device__ __forceinline__ u32x4 stream8(const uint16_t* row, uint64_t c, uint64_t cols) {
  if (c + kChunk <= cols)
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4_at2*>(row + c));
  return load8(row, c, cols);
}

// Stores of whole activations bypass the caches' keeping: what is written here is
// larger than they are, and rows come in faster for it (16384 x 4096 bf16: reading a
// checkpoint back that was just written 42 -> 31 us, the norms 111 -> 99 us).  Loads of what is read once
// do too, where that measured faster.
template <bool STREAM = true>
__device__ __forceinline__ void store8(uint16_t* row, uint64_t c, uint64_t cols, u32x4 w) {
  if (c + kChunk <= cols) {
    if constexpr (STREAM) __builtin_nontemporal_store(w, reinterpret_cast<u32x4_at2*>(row + c));
    else *reinterpret_cast<u32x4_at2*>(row + c) = w;
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < cols) row[c + i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
}

// Eight codes, likewise.
__device__ __forceinline__ u32x2 load_codes(const uint8_t* row, uint64_t c, uint64_t cols) {
  if (c + kChunk <= cols) return *reinterpret_cast<const u32x2_at1*>(row + c);
  uint32_t e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = row[c + i < cols ? c + i : cols - 1];
  u32x2 w = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i >> 2] |= (c + i < cols ? e[i] : 0u) << (8 * (i & 3));
  return w;
}

__device__ __forceinline__ void store_codes(uint8_t* row, uint64_t c, uint64_t cols, u32x2 w) {
  if (c + kChunk <= cols) {
    __builtin_nontemporal_store(w, reinterpret_cast<u32x2_at1*>(row + c));
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < cols) row[c + i] = static_cast<uint8_t>(w[i >> 2] >> (8 * (i & 3)));
}

// The same for kernels that issue the loads of many chunks before they use them:
// every lane loads its chunk without a branch, or, past the last whole chunk, the
// row's last eight elements; mend8 then shifts those into place, or puts 0 where
// the row has ended.  Rows of fewer than eight elements are loaded by mend8.
// FULL: every chunk is whole.
template <bool FULL>
__device__ __forceinline__ uint32_t early(uint32_t c, uint32_t cols) {
  if constexpr (FULL) return c;
  return c + kChunk <= cols ? c : cols - kChunk;
}

template <bool FULL>
__device__ __forceinline__ u32x4 load8_early(const uint16_t* row, uint32_t c, uint32_t cols) {
  if (!FULL && cols < kChunk) return u32x4{0, 0, 0, 0};
  return *reinterpret_cast<const u32x4_at2*>(row + early<FULL>(c, cols));
}

// Read once (see store8); STREAM == false: as load8_early.
template <bool FULL, bool STREAM = true>
__device__ __forceinline__ u32x4 stream8_early(const uint16_t* row, uint32_t c, uint32_t cols) {
  if (!FULL && cols < kChunk) return u32x4{0, 0, 0, 0};
  if (!STREAM) return load8_early<FULL>(row, c, cols);
  return __builtin_nontemporal_load(
      reinterpret_cast<const u32x4_at2*>(row + early<FULL>(c, cols)));
}

template <bool FULL, bool STREAM = true>
__device__ __forceinline__ u32x2 stream_codes_early(const uint8_t* row, uint32_t c,
                                                    uint32_t cols) {
  if (!FULL && cols < kChunk) return u32x2{0, 0};
  if (!STREAM) return *reinterpret_cast<const u32x2_at1*>(row + early<FULL>(c, cols));
  return __builtin_nontemporal_load(
      reinterpret_cast<const u32x2_at1*>(row + early<FULL>(c, cols)));
}

template <bool FULL>
__device__ __forceinline__ void mend8(u32x4& w, const uint16_t* row, uint32_t c, uint32_t cols) {
  if (FULL || c + kChunk <= cols) return;
  if (c >= cols) {
    w = u32x4{0, 0, 0, 0};
  } else if (cols < kChunk) {
    w = load8(row, c, cols);
  } else {
    const uint32_t by = c + kChunk - cols;   // elements to drop, 1 .. 7
    if (by & 4) w = u32x4{w[2], w[3], 0, 0};
    if (by & 2) w = u32x4{w[1], w[2], w[3], 0};
    if (by & 1)
      w = u32x4{__builtin_amdgcn_alignbit(w[1], w[0], 16), __builtin_amdgcn_alignbit(w[2], w[1], 16),
                __builtin_amdgcn_alignbit(w[3], w[2], 16), w[3] >> 16};
  }
}

// Both at once, for rows that lie in the caches.
template <bool FULL>
__device__ __forceinline__ u32x4 load8_row(const uint16_t* row, uint32_t c, uint32_t cols) {
  u32x4 w = load8_early<FULL>(row, c, cols);
  mend8<FULL>(w, row, c, cols);
  return w;
}

template <bool FULL, bool STREAM = true>
__device__ __forceinline__ void store8_row(uint16_t* row, uint32_t c, uint32_t cols, u32x4 w) {
  if (FULL || c < cols) store8<STREAM>(row, c, FULL ? UINT64_MAX : cols, w);
}

template <bool FULL>
__device__ __forceinline__ void mend_codes(u32x2& w, const uint8_t* row, uint32_t c,
                                           uint32_t cols) {
  if (FULL || c + kChunk <= cols) return;
  if (c >= cols) {
    w = u32x2{0, 0};
  } else if (cols < kChunk) {
    w = load_codes(row, c, cols);
  } else {
    const uint32_t by = c + kChunk - cols;
    const uint64_t v = (static_cast<uint64_t>(w[1]) << 32 | w[0]) >> (8 * by);
    w = u32x2{static_cast<uint32_t>(v), static_cast<uint32_t>(v >> 32)};
  }
}

// ------------------------------------------------------------ the 8-bit format

// 2^(b - 127) of a scale byte: its exponent field (2^-127 is subnormal); 255: NaN.
__device__ __forceinline__ float scale_of(uint32_t b) {
  return __builtin_bit_cast(float, b == 255u ? 0x7FC00000u : b == 0 ? 0x00400000u : b << 23);
}

template <int FMT>
__device__ __forceinline__ void decode4(uint32_t w, float s, float* x) {
  if constexpr (FMT == kInt8) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = static_cast<float>(static_cast<int8_t>(w >> (8 * i))) * s;
  } else {
    typedef float f2 __attribute__((ext_vector_type(2)));
    const f2 a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false);
    const f2 b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
    x[0] = a[0] * s;
    x[1] = a[1] * s;
    x[2] = b[0] * s;
    x[3] = b[1] * s;
  }
}

template <int FMT>
__device__ __forceinline__ void decode8(u32x2 w, float s, float (&x)[8]) {
  decode4<FMT>(w[0], s, x);
  decode4<FMT>(w[1], s, x + 4);
}

// Codes straight to 16-bit values, each rounded to nearest even, two at a time, for
// kernels that feed the matrix instructions: Scale16 is made once a block, then
// pair<I> gives codes 2 I and 2 I + 1 of a chunk.
template <typename T, int FMT>
struct Scale16 {
  float s, off;

  __device__ __forceinline__ void set(uint32_t b) {
    if constexpr (FMT == kE4m3) {
      s = __builtin_bit_cast(float, b << 23);   // only its exponent field is read
    } else if constexpr (T::kType == kF16) {
      // 2^73 and more overflow alike, and 1152 * 2^73 is finite
      s = scale_of(b == 255u || b < 200u ? b : 200u);
      off = -1152.0f * s;
    } else {
      s = scale_of(b);
    }
  }

  template <int I>
  __device__ __forceinline__ uint32_t pair(u32x2 w) const {
    if constexpr (FMT == kE4m3) {
      if constexpr (T::kType == kF16)
        return __builtin_bit_cast(
            uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[I / 2], s, I % 2 != 0));
      else
        return __builtin_bit_cast(
            uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[I / 2], s, I % 2 != 0));
    } else if constexpr (T::kType == kF16) {
      // 0x6400 | u is the half 1024 + u, u = code + 128: one fused multiply-add in
      // fp32 gives code * 2^e, rounded once to 16 bits
      typedef _Float16 h2 __attribute__((ext_vector_type(2)));
      const h2 c = __builtin_bit_cast(
          h2, __builtin_amdgcn_perm(0x64646464u, w[I / 2] ^ 0x80808080u,
                                    I % 2 ? 0x04030402u : 0x04010400u));
      const h2 v = {static_cast<_Float16>(__builtin_fmaf(static_cast<float>(c[0]), s, off)),
                    static_cast<_Float16>(__builtin_fmaf(static_cast<float>(c[1]), s, off))};
      return __builtin_bit_cast(uint32_t, v);
    } else {
      constexpr int kAt = I % 2 * 16;
      return pack16<T>(static_cast<float>(static_cast<int8_t>(w[I / 2] >> kAt)) * s,
                       static_cast<float>(static_cast<int8_t>(w[I / 2] >> (kAt + 8))) * s);
    }
  }
};

// The value of lane i ^ 1, i ^ 2 within each quad of lanes.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, true));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  typedef uint16_t us2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(us2, a),
                                                                __builtin_bit_cast(us2, b)));
}

// Encodes this lane's eight 16-bit elements of a block that four neighbouring
// lanes share (all four call this together).  The block's largest magnitude is
// found on the bit patterns, whose order as whole numbers is that of the
// magnitudes, with infinities and NaN above every finite value.
//   int8:  2^e = 2^(floor(log2 amax) - 6); codes rounded to nearest even and
//          held to +-127 (amax 2^-e lies in [64, 128)).
//   e4m3:  2^e is the least power of two with amax 2^-e <= 448; inputs are held
//          to 1.875 times the type's top power of two, which is the largest
//          value that 4 significant bits and the type both hold.
// A block with an infinity or NaN becomes NaN as a whole, so an overflow stays
// visible.  e is at least -126 (int8) or -117 (e4m3): every held value is a
// normal fp32 number or 0.
template <typename T, int FMT>
__device__ __forceinline__ u32x2 encode8(u32x4 w, uint32_t* scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max_u16x2(m, w[i] & 0x7FFF7FFFu);
  m = max_u16x2(m, dpp<kXor1>(m));
  m = max_u16x2(m, dpp<kXor2>(m));
  const uint32_t hi = m >> 16, lo = m & 0xFFFFu;
  const uint32_t top = hi > lo ? hi : lo;
  constexpr uint32_t kInf = T::kType == kF16 ? 0x7C00u : 0x7F80u;
  const uint32_t bits = __builtin_bit_cast(uint32_t, lo16<T>(top));
  int e;
  if constexpr (FMT == kInt8) {
    e = static_cast<int>(bits >> 23) - 127 - 6;
    e = e < -126 ? -126 : e;
  } else {
    constexpr float kTop = T::kType == kF16 ? 0x1.Ep15f : 0x1.Ep127f;
    const uint32_t held = bits < __builtin_bit_cast(uint32_t, kTop)
                              ? bits : __builtin_bit_cast(uint32_t, kTop);
    // the mantissa of 448 is 1.75: anything above it carries into the exponent
    e = static_cast<int>((held + 0x1FFFFFu) >> 23) - 127 - 8;
    e = e < -117 ? -117 : e;
  }
  const bool finite = top < kInf;
  *scale = finite ? static_cast<uint32_t>(e + 127) : 255u;
  const float inv = __builtin_bit_cast(float, static_cast<uint32_t>(127 - e) << 23);
  float x[8];
  unpack8<T>(w, x);
  u32x2 out;
  if constexpr (FMT == kInt8) {
    // adding 1.5 * 2^23 rounds to a whole number (nearest even) and leaves it in
    // the low mantissa bits in two's complement
    constexpr float kMagic = 0x1.8p23f;
    uint32_t q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = __builtin_fmaf(x[i], inv, kMagic);
      q[i] = __builtin_bit_cast(uint32_t,
                                __builtin_amdgcn_fmed3f(y, kMagic - 127.f, kMagic + 127.f));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t a = __builtin_amdgcn_perm(q[4 * i + 1], q[4 * i], 0x0C0C0400u);
      const uint32_t b = __builtin_amdgcn_perm(q[4 * i + 3], q[4 * i + 2], 0x04000C0Cu);
      out[i] = a | b;
    }
  } else {
    constexpr float kTop = T::kType == kF16 ? 0x1.Ep15f : 0x1.Ep127f;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __builtin_amdgcn_fmed3f(x[i], -kTop, kTop) * inv;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int p = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i], x[4 * i + 1], 0, false);
      p = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i + 2], x[4 * i + 3], p, true);
      out[i] = static_cast<uint32_t>(p);
    }
  }
  if (!finite) out = u32x2{0, 0};
  return out;
}

// ------------------------------------------------------------ sums

__device__ __forceinline__ float dpp_add(float v, uint32_t moved) {
  return v + __builtin_bit_cast(float, moved);
}

// The sum over the 64 lanes, in every lane; the order is fixed.
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add(v, dpp<kXor1>(__builtin_bit_cast(uint32_t, v)));
  v = dpp_add(v, dpp<kXor2>(__builtin_bit_cast(uint32_t, v)));
  v = dpp_add(v, dpp<kHalfMirror>(__builtin_bit_cast(uint32_t, v)));
  v = dpp_add(v, dpp<kMirror>(__builtin_bit_cast(uint32_t, v)));
  const int b = __builtin_bit_cast(int, v);
  const float r0 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 0));
  const float r1 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 16));
  const float r2 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 32));
  const float r3 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 48));
  return (r0 + r1) + (r2 + r3);
}

}  // namespace act
}  // namespace zero

#endif  // ZERO_ACT_FORMAT_H_
