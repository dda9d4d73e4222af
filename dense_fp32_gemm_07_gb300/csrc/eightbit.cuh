// eightbit.cuh -- the 8-bit form of matrix rows (b2g_quantize8 in include/b2g_train.h):
// e4m3 codes, and one power of two for each 32 columns of a row as an e8m0 byte (2^(byte -
// 127)).  The scale is the smallest power of two, 2^-110 at least, that brings the block's
// largest finite value to 448, e4m3's largest, or below: nothing saturates, and the one
// rounding, to nearest even, costs at most 2^-4 of a value (or 2^-10 of the scale).  Being
// powers of two, scales lose nothing when they are divided out or multiplied back, and a
// value read back has 4 significant bits: it is exact in BF16.
#pragma once
#include "train_common.cuh"

namespace b2g {

constexpr int kScaleBlock = 32;    // columns that share a scale
constexpr int kLeastScale = 17;    // byte of 2^-110: values read back stay normal BF16 numbers

inline __host__ __device__ long long scale_count(long long cols) {
  return (cols + kScaleBlock - 1) / kScaleBlock;
}

// The scale's byte from the largest finite magnitude: its exponent, one more where the
// mantissa is above 1.75 (448 = 1.75 * 2^8), less 8.
__device__ __forceinline__ uint32_t scale_byte(float largest) {
  const int e = (int)((__float_as_uint(largest) + 0x1FFFFFu) >> 23) - 8;
  return (uint32_t)max(e, kLeastScale);
}
// 1 / scale of a byte that scale_byte made.
__device__ __forceinline__ float scale_inverse(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}
// The scale of any byte: 0 is 2^-127 (subnormal), 255 NaN.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  const uint32_t bits = byte == 0u ? 0x00400000u : byte == 255u ? 0x7fc00000u : byte << 23;
  return __uint_as_float(bits);
}

// Two values to two codes, the first in the low byte; NaN becomes the code NaN.
__device__ __forceinline__ uint32_t encode2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void decode2(uint32_t codes, float& lo, float& hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  const __half2 v = *reinterpret_cast<const __half2*>(&h);
  lo = __low2float(v), hi = __high2float(v);
}

// One code as an element of a row.
struct E4m3 {
  unsigned char b;
};
__device__ __forceinline__ float to_f32(E4m3 x) {
  float v, none;
  decode2(x.b, v, none);
  return v;
}

// VEC consecutive codes as loaded or stored: VEC bytes on a boundary of their size.
template <int VEC>
struct Codes {
  uint32_t w[VEC / 4];
  __device__ __forceinline__ void load(const unsigned char* p) {
    if constexpr (VEC == 8) {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      w[0] = u.x, w[1] = u.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
  }
  __device__ __forceinline__ void store(unsigned char* p) const {
    if constexpr (VEC == 8)
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(p) = w[0];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void set(const float (&f)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i)
      w[i] = encode2(f[4 * i], f[4 * i + 1]) | encode2(f[4 * i + 2], f[4 * i + 3]) << 16;
  }
  __device__ __forceinline__ void get(float (&f)[VEC]) const {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      decode2(w[i] & 0xFFFFu, f[4 * i], f[4 * i + 1]);
      decode2(w[i] >> 16, f[4 * i + 2], f[4 * i + 3]);
    }
  }
};
template <>
struct Codes<1> {
  uint32_t w;
  __device__ __forceinline__ void load(const unsigned char* p) { w = *p; }
  __device__ __forceinline__ void store(unsigned char* p) const { *p = (unsigned char)w; }
  __device__ __forceinline__ void zero() { w = 0; }
  __device__ __forceinline__ void set(const float (&f)[1]) { w = encode2(f[0], 0.f) & 0xFFu; }
  __device__ __forceinline__ void get(float (&f)[1]) const {
    float none;
    decode2(w, f[0], none);
  }
};

// The largest finite magnitude of a block whose columns the 32 / VEC lanes of an aligned
// group hold, VEC each (zeros past the row).  Infinities become NaN, the code they get.
// The whole warp takes part.
template <int VEC>
__device__ __forceinline__ float block_largest(float (&f)[VEC]) {
  constexpr int lanes = kScaleBlock / VEC;
  // as whole numbers, magnitudes stand in the same order, infinity above all finite ones
  // and NaN above it
  auto largest = [&] {
    uint32_t m = __float_as_uint(f[0]) & 0x7fffffffu;
#pragma unroll
    for (int j = 1; j < VEC; ++j) m = max(m, __float_as_uint(f[j]) & 0x7fffffffu);
    if constexpr (lanes == 32) {
      m = __reduce_max_sync(0xffffffffu, m);
    } else {
#pragma unroll
      for (int o = lanes / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    return m;
  };
  uint32_t m = largest();
  if (__any_sync(0xffffffffu, m >= 0x7f800000u)) {  // rare: once more without those
    float g[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const bool bad = (__float_as_uint(f[j]) & 0x7fffffffu) >= 0x7f800000u;
      g[j] = bad ? __int_as_float(0x7fffffff) : f[j];
      f[j] = bad ? 0.f : f[j];
    }
    m = largest();
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = g[j];
  }
  return __uint_as_float(m);
}

// VEC columns of a row to their codes; the scale's byte is the same in all lanes of a block.
template <int VEC>
__device__ __forceinline__ uint32_t encode(float (&f)[VEC], Codes<VEC>& codes) {
  const uint32_t byte = scale_byte(block_largest<VEC>(f));
  const float inv = scale_inverse(byte);
  float g[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) g[j] = f[j] * inv;
  codes.set(g);
  return byte;
}

// Codes and scales of a matrix.
struct Rows8 {
  unsigned char* q;
  long long ldq;
  unsigned char* s;
  long long lds;
};
// Chunk c (VEC columns) of row `row`, of which `in` says whether it exists.
template <int VEC>
__device__ __forceinline__ void encode_to(const Rows8& to, long long row, int c, bool in,
                                          float (&f)[VEC]) {
  constexpr int lanes = kScaleBlock / VEC;
  Codes<VEC> k;
  const uint32_t byte = encode<VEC>(f, k);
  if (in) {
    k.store(to.q + row * to.ldq + (long long)c * VEC);
    if (c % lanes == 0) to.s[row * to.lds + c / lanes] = (unsigned char)byte;
  }
}
// Whether codes may be read and written VEC at a time (VEC a power of two).
inline bool codes_vec(const Rows8& r, int vec) {
  return !r.q || (reinterpret_cast<uintptr_t>(r.q) % vec == 0 && r.ldq % vec == 0);
}

}  // namespace b2g
