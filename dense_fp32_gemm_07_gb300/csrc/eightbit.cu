// eightbit.cu -- rows to their 8-bit form and back (b2g_quantize8, b2g_dequantize8 in
// include/b2g_train.h; the form itself: eightbit.cuh).
#include "eightbit.cuh"

namespace b2g {
namespace {

struct Convert {
  long long rows;
  int cols;
  unsigned chunks, per;  // chunks of a row: those that exist, and with the last block filled up
  void* x;       // read by quantize, written by dequantize
  long long ldx;
  Rows8 k;
};

// A row counts as `per` chunks of VEC columns, whole blocks of 32 columns; a block takes
// 256 * U consecutive chunks of the matrix, so that a scale's block is in one warp and
// short rows fill it, and a thread has U of them on their way at a time.
struct Place {
  long long row;
  unsigned c;
};
template <int U>
struct Chunks {
  long long row0;
  unsigned c0, per;
  __device__ __forceinline__ Chunks(unsigned per_) : per(per_) {
    const long long first = (long long)blockIdx.x * (256 * U);
    row0 = first / per, c0 = (unsigned)(first - row0 * per);
  }
  __device__ __forceinline__ Place at(int u) const {
    const unsigned i = c0 + threadIdx.x + 256u * u, r = i / per;
    return Place{row0 + r, i - r * per};
  }
};

// Bound: bytes.
template <typename T, int VEC, int U>
__global__ void __launch_bounds__(256) quantize_kernel(const __grid_constant__ Convert p) {
  pdl_launch_dependents();
  pdl_wait();
  const Chunks<U> all(p.per);
  Pack<T, VEC> k[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const Place at = all.at(u);
    k[u].zero();
    if (at.row < p.rows && at.c < p.chunks)
      k[u].load(static_cast<const T*>(p.x) + at.row * p.ldx + (long long)at.c * VEC);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const Place at = all.at(u);
    float f[VEC];
    k[u].get(f);
    encode_to<VEC>(p.k, at.row, (int)at.c, at.row < p.rows && at.c < p.chunks, f);
  }
}

template <typename T, int VEC, int U>
__global__ void __launch_bounds__(256) dequantize_kernel(const __grid_constant__ Convert p) {
  pdl_launch_dependents();
  pdl_wait();
  const Chunks<U> all(p.per);
  Codes<VEC> k[U];
  uint32_t byte[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const Place at = all.at(u);
    if (at.row < p.rows && at.c < p.chunks) {
      k[u].load(p.k.q + at.row * p.k.ldq + (long long)at.c * VEC);
      byte[u] = p.k.s[at.row * p.k.lds + at.c / (kScaleBlock / VEC)];
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const Place at = all.at(u);
    if (at.row < p.rows && at.c < p.chunks) {
      const float scale = scale_value(byte[u]);
      float f[VEC];
      k[u].get(f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[j] *= scale;
      Pack<T, VEC> o;
      o.set(f);
      o.store(static_cast<T*>(p.x) + at.row * p.ldx + (long long)at.c * VEC);
    }
  }
}

int check(int dtype, long long rows, int cols, const void* x, long long ldx, const void* codes,
          long long ldq, const void* scales, long long lds) {
  if (!type_ok(dtype)) return B2G_ERR_INVALID_TYPE;
  if (rows < 0 || cols < 0 || rows > 0x7fffffffLL || cols > kMaxLength) return B2G_ERR_INVALID_DIM;
  const long long least = cols > 1 ? cols : 1;
  if (ldx < least || ldq < least || lds < scale_count(least)) return B2G_ERR_INVALID_LD;
  if (rows == 0 || cols == 0) return 0;
  return x && codes && scales ? 0 : B2G_ERR_NULL;
}

template <typename T, int VEC>
cudaError_t launch(bool back, Convert p, cudaStream_t st) {
  constexpr int U = VEC > 1 ? 4 : 8;
  p.chunks = (unsigned)(p.cols / VEC);
  p.per = (unsigned)(scale_count(p.cols) * (kScaleBlock / VEC));
  const long long blocks = ceil_div(p.rows * p.per, 256 * U);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_train(back ? dequantize_kernel<T, VEC, U> : quantize_kernel<T, VEC, U>,
                      dim3((unsigned)blocks), dim3(256), 0, st, p);
}

int convert(bool back, int dtype, const Convert& p, void* stream) {
  TrainDevice d;
  const int rc = train_device(&d);
  if (rc) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool f32 = dtype == B2G_F32;
  const bool v = vec16(p.x) && vec16_ld(p.ldx, dtype) && vec16_ld(p.cols, dtype) &&
                 codes_vec(p.k, f32 ? 4 : 8);
  if (f32) return launch_code(v ? launch<float, 4>(back, p, st) : launch<float, 1>(back, p, st));
  return launch_code(v ? launch<Bf16, 8>(back, p, st) : launch<Bf16, 1>(back, p, st));
}

}  // namespace
}  // namespace b2g

using namespace b2g;

extern "C" {

int b2g_quantize8(int dtype, long long rows, int cols, const void* x, long long ldx, void* codes,
                  long long ldq, void* scales, long long lds, void* stream) {
  const int rc = check(dtype, rows, cols, x, ldx, codes, ldq, scales, lds);
  if (rc || rows == 0 || cols == 0) return rc;
  return convert(false, dtype,
                 Convert{rows, cols, 0, 0, const_cast<void*>(x), ldx,
                         {static_cast<unsigned char*>(codes), ldq, static_cast<unsigned char*>(scales), lds}},
                 stream);
}

int b2g_dequantize8(int dtype, long long rows, int cols, const void* codes, long long ldq,
                    const void* scales, long long lds, void* y, long long ldy, void* stream) {
  const int rc = check(dtype, rows, cols, y, ldy, codes, ldq, scales, lds);
  if (rc || rows == 0 || cols == 0) return rc;
  return convert(true, dtype,
                 Convert{rows, cols, 0, 0, y, ldy,
                         {static_cast<unsigned char*>(const_cast<void*>(codes)), ldq,
                          static_cast<unsigned char*>(const_cast<void*>(scales)), lds}},
                 stream);
}

}  // extern "C"
