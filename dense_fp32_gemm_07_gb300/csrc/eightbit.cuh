// eightbit.cuh -- the 8-bit form of matrix rows (b2g_quantize8 in include/b2g_train.h):
// e4m3 codes, and one power of two for each 32 columns of a row as an e8m0 byte (2^(byte -
// 127)).  The scale is the smallest power of two, 2^-110 at least, that brings the block's
// largest finite value to 448, e4m3's largest, or below: nothing saturates, and the one
// rounding, to nearest even, costs at most 2^-4 of a value (or 2^-10 of the scale).  Being
// powers of two, scales lose nothing when they are divided out or multiplied back, and a
// value read back has 4 significant bits: it is exact in BF16.
#pragma once
#include "anyrow.cuh"

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
  // Those of [from, to), byte by byte.
  __device__ __forceinline__ void load(const unsigned char* p, int from, int to) {
    zero();
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (j >= from && j < to) w[j / 4] |= (uint32_t)p[j] << (8 * (j & 3));
  }
  __device__ __forceinline__ void store(unsigned char* p, int n) const {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (j < n) p[j] = (unsigned char)(w[j / 4] >> (8 * (j & 3)));
  }
  // Codes outside [from, to) become zero.
  __device__ __forceinline__ void keep(int from, int to) {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (j < from || j >= to) w[j / 4] &= ~(0xFFu << (8 * (j & 3)));
  }
  // From byte `off` of shared memory on 16-byte boundaries, which holds 4 more.
  __device__ __forceinline__ void load_shared(const unsigned char* base, uint32_t off) {
    const uint32_t* v = reinterpret_cast<const uint32_t*>(base + (off & ~3u));
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) w[i] = __funnelshift_r(v[i], v[i + 1], 8 * (off & 3u));
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
// The largest finite magnitudes of N blocks whose columns the 32 / VEC lanes of an aligned
// group hold, VEC each (zeros past the row).  Infinities become NaN, the code they get.
// The whole warp takes part.
template <int VEC, int N>
__device__ __forceinline__ void block_largest(float (&f)[N][VEC], float (&m)[N]) {
  constexpr int lanes = kScaleBlock / VEC;
  auto largest = [&] {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      m[i] = fabsf(f[i][0]);
#pragma unroll
      for (int j = 1; j < VEC; ++j) m[i] = fmaxf(m[i], fabsf(f[i][j]));  // a NaN is passed over
    }
#pragma unroll
    for (int o = lanes / 2; o; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
  };
  largest();
  bool fine = true;
#pragma unroll
  for (int i = 0; i < N; ++i) fine = fine && m[i] < INFINITY;
  if (__any_sync(0xffffffffu, !fine)) {  // rare: once more without those
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        f[i][j] = fabsf(f[i][j]) < INFINITY ? f[i][j] : __int_as_float(0x7fffffff);
    largest();
#pragma unroll
    for (int i = 0; i < N; ++i) m[i] = m[i] == m[i] ? m[i] : 0.f;  // nothing but NaN
  }
}

// N times VEC columns of rows to their codes; the bytes of the scales are the same in all
// lanes of a block.
template <int VEC, int N>
__device__ __forceinline__ void encode(float (&f)[N][VEC], Codes<VEC> (&codes)[N], uint32_t (&byte)[N]) {
  float m[N];
  block_largest<VEC, N>(f, m);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    byte[i] = scale_byte(m[i]);
    const float inv = scale_inverse(byte[i]);
    float g[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) g[j] = f[i][j] * inv;
    codes[i].set(g);
  }
}

// Codes and scales of a matrix.
struct Rows8 {
  unsigned char* q;
  long long ldq;
  unsigned char* s;
  long long lds;
  int vec;  // rows on boundaries of a chunk's codes
};
// Chunk c (VEC codes) of a row.  Without ANY it is whole and on its boundary.
template <int VEC, bool ANY>
__device__ __forceinline__ void load_codes(Codes<VEC>& k, const Rows8& from, long long row, int c, int cols) {
  const unsigned char* q = from.q + row * from.ldq + (long long)c * VEC;
  if (!ANY || (from.vec && (c + 1) * VEC <= cols))
    k.load(q);
  else
    k.load(q, 0, cols - c * VEC);
}
template <int VEC, bool ANY>
__device__ __forceinline__ void store_codes(const Codes<VEC>& k, const Rows8& to, long long row, int c,
                                            int cols) {
  unsigned char* q = to.q + row * to.ldq + (long long)c * VEC;
  if (!ANY || (to.vec && (c + 1) * VEC <= cols))
    k.store(q);
  else
    k.store(q, min(VEC, cols - c * VEC));
}
// Chunks c, c + step, ... (VEC columns each) of row `row`, those below `chunks`.
template <int VEC, int N, bool ANY>
__device__ __forceinline__ void encode_to(const Rows8& to, long long row, int c, int step, int chunks,
                                          int cols, float (&f)[N][VEC]) {
  constexpr int lanes = kScaleBlock / VEC;
  Codes<VEC> k[N];
  uint32_t byte[N];
  encode<VEC, N>(f, k, byte);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int at = c + i * step;
    if (at < chunks) {
      store_codes<VEC, ANY>(k[i], to, row, at, cols);
      if (at % lanes == 0) to.s[row * to.lds + at / lanes] = (unsigned char)byte[i];
    }
  }
}
// Whether codes may be read and written `vec` at a time (a power of two).
inline bool codes_vec(const Rows8& r, int vec) {
  return !r.q || (reinterpret_cast<uintptr_t>(r.q) % vec == 0 && r.ldq % vec == 0);
}

}  // namespace b2g
