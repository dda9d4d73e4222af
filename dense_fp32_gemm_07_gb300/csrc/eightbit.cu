// eightbit.cu -- rows to their 8-bit form and back (b2g_quantize8, b2g_dequantize8 in
// include/b2g_train.h; the form itself: eightbit.cuh).
#include "eightbit.cuh"

namespace b2g {
namespace {

// A block of 32 columns stays within a pass of a warp.
struct Convert {
  Walk walk;
  int cols;
  void* x;  // read by quantize, written by dequantize
  long long ldx;
  Rows8 k;
};

// Four chunks a thread are on their way before the first is converted, and all four blocks'
// largest values are found together.  Bound: bytes.  BF16 16384 x 4096 33.8 us (6.0 TB/s),
// 8192 x 4096 18.3 (2.7 of them the launch), 8192 x 4095 30; FP32 4096 x 4096 14.5, 8192 x 4095 45.
template <typename T, bool ANY>
__global__ void __launch_bounds__(256) quantize_kernel(const __grid_constant__ Convert p) {
  constexpr int VEC = kVec<T>, U = kPasses, lanes = kScaleBlock / VEC;
  pdl_launch_dependents();
  const Places at(p.walk, blockIdx.x);
  pdl_wait();
  Pack<T, VEC> k[U];
  Fetched raw[ANY ? U : 1];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long row = at.row_of(u);
    const int c = at.chunk_of(u);
    const bool in = row < p.walk.rows && c < p.walk.chunks;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    if constexpr (ANY) {
      fetch<T>(raw[u], x, c * VEC, p.cols, in);
    } else {
      k[u].zero();
      if (in) k[u].load(x + (long long)c * VEC);
    }
  }
  float f[U][VEC];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if constexpr (ANY) {
      const long long row = at.row_of(u);
      const int c = at.chunk_of(u);
      finish<T>(k[u], raw[u], static_cast<const T*>(p.x) + row * p.ldx, c * VEC, p.cols,
                row < p.walk.rows && c < p.walk.chunks);
    }
    k[u].get(f[u]);
  }
  Codes<VEC> codes[U];
  uint32_t byte[U];
  encode<VEC, U>(f, codes, byte);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long row = at.row_of(u);
    const int c = at.chunk_of(u);
    if (row < p.walk.rows && c < p.walk.chunks) {
      store_codes<VEC, ANY>(codes[u], p.k, row, c, p.cols);
      if (c % lanes == 0) p.k.s[row * p.k.lds + c / lanes] = (unsigned char)byte[u];
    }
  }
}

// Bound: bytes.  BF16 16384 x 4096 31.2 us (6.5 TB/s), 8192 x 4096 16.8, 8192 x 4095 33; FP32
// 4096 x 4096 14.4, 8192 x 4095 45.
template <typename T, bool ANY>
__global__ void __launch_bounds__(256) dequantize_kernel(const __grid_constant__ Convert p) {
  constexpr int VEC = kVec<T>, U = kPasses;
  pdl_launch_dependents();
  const Places at(p.walk, blockIdx.x);
  pdl_wait();
  Codes<VEC> k[U];
  uint32_t byte[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long row = at.row_of(u);
    const int c = at.chunk_of(u);
    if (row < p.walk.rows && c < p.walk.chunks) {
      load_codes<VEC, ANY>(k[u], p.k, row, c, p.cols);
      byte[u] = p.k.s[row * p.k.lds + c / (kScaleBlock / VEC)];
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long row = at.row_of(u);
    const int c = at.chunk_of(u);
    const bool in = row < p.walk.rows && c < p.walk.chunks;
    Pack<T, VEC> o;
    o.zero();
    if (in) {
      const float scale = scale_value(byte[u]);
      float f[VEC];
      k[u].get(f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[j] *= scale;
      o.set(f);
    }
    store_chunk<T, ANY>(o, static_cast<T*>(p.x) + row * p.ldx, c, p.cols, in, at.lanes);
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

template <typename T, bool ANY>
cudaError_t launch(bool back, Convert p, cudaStream_t st) {
  p.walk = walk_of(p.walk.rows, (int)ceil_div(p.cols, kVec<T>), kScaleBlock / kVec<T>);
  if (p.walk.blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_train(back ? dequantize_kernel<T, ANY> : quantize_kernel<T, ANY>, dim3((unsigned)p.walk.blocks),
                      dim3(256), 0, st, p);
}

int convert(bool back, int dtype, Convert p, void* stream) {
  TrainDevice d;
  const int rc = train_device(&d);
  if (rc) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool f32 = dtype == B2G_F32;
  p.k.vec = codes_vec(p.k, f32 ? 4 : 8);
  const bool v = vec16(p.x) && vec16_ld(p.ldx, dtype) && vec16_ld(p.cols, dtype) && p.k.vec;
  if (f32) return launch_code(v ? launch<float, false>(back, p, st) : launch<float, true>(back, p, st));
  return launch_code(v ? launch<Bf16, false>(back, p, st) : launch<Bf16, true>(back, p, st));
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
                 Convert{{rows}, cols, const_cast<void*>(x), ldx,
                         {static_cast<unsigned char*>(codes), ldq, static_cast<unsigned char*>(scales), lds, 0}},
                 stream);
}

int b2g_dequantize8(int dtype, long long rows, int cols, const void* codes, long long ldq,
                    const void* scales, long long lds, void* y, long long ldy, void* stream) {
  const int rc = check(dtype, rows, cols, y, ldy, codes, ldq, scales, lds);
  if (rc || rows == 0 || cols == 0) return rc;
  return convert(true, dtype,
                 Convert{{rows}, cols, y, ldy,
                         {static_cast<unsigned char*>(const_cast<void*>(codes)), ldq,
                          static_cast<unsigned char*>(const_cast<void*>(scales)), lds, 0}},
                 stream);
}

}  // extern "C"
