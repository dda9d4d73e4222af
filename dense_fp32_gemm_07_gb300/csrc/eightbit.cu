// eightbit.cu -- rows to their 8-bit form and back (b2g_quantize8, b2g_dequantize8 in
// include/b2g_train.h; the form itself: eightbit.cuh).
#include "eightbit.cuh"

namespace b2g {
namespace {

struct Convert {
  long long rows;
  int cols;
  void* x;       // read by quantize, written by dequantize
  long long ldx;
  Rows8 k;
};

// A warp's lanes hold consecutive chunks of VEC columns of one row.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) quantize_kernel(const __grid_constant__ Convert p) {
  pdl_launch_dependents();
  pdl_wait();
  const int chunks = (p.cols + VEC - 1) / VEC, per = (chunks + 31) / 32;
  const long long total = p.rows * per;
  for (long long u = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); u < total;
       u += (long long)gridDim.x * 8) {
    const long long row = u / per;
    const int c = (int)(u - row * per) * 32 + (threadIdx.x & 31);
    Pack<T, VEC> k;
    k.zero();
    if (c < chunks) k.load(static_cast<const T*>(p.x) + row * p.ldx + (long long)c * VEC);
    float f[VEC];
    k.get(f);
    encode_to<VEC>(p.k, row, c, c < chunks, f);
  }
}

template <typename T, int VEC>
__global__ void __launch_bounds__(256) dequantize_kernel(const __grid_constant__ Convert p) {
  pdl_launch_dependents();
  pdl_wait();
  const int chunks = p.cols / VEC;
  const long long total = p.rows * chunks;
  for (long long u = (long long)blockIdx.x * 256 + threadIdx.x; u < total;
       u += (long long)gridDim.x * 256) {
    const long long row = u / chunks;
    const int c = (int)(u - row * chunks);
    Codes<VEC> k;
    k.load(p.k.q + row * p.k.ldq + (long long)c * VEC);
    const float scale = scale_value(p.k.s[row * p.k.lds + c / (kScaleBlock / VEC)]);
    float f[VEC];
    k.get(f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] *= scale;
    Pack<T, VEC> o;
    o.set(f);
    o.store(static_cast<T*>(p.x) + row * p.ldx + (long long)c * VEC);
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
cudaError_t launch(bool back, const Convert& p, int sms, cudaStream_t st) {
  const long long warps = p.rows * ceil_div(ceil_div(p.cols, VEC), 32);
  const long long blocks = ceil_div(warps, 8), most = 16LL * sms;
  const dim3 grid((unsigned)(blocks < most ? blocks : most));
  return launch_train(back ? dequantize_kernel<T, VEC> : quantize_kernel<T, VEC>, grid, dim3(256), 0,
                      st, p);
}

int convert(bool back, int dtype, const Convert& p, void* stream) {
  TrainDevice d;
  const int rc = train_device(&d);
  if (rc) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool f32 = dtype == B2G_F32;
  const bool v = vec16(p.x) && vec16_ld(p.ldx, dtype) && vec16_ld(p.cols, dtype) &&
                 codes_vec(p.k, f32 ? 4 : 8);
  if (f32) return launch_code(v ? launch<float, 4>(back, p, d.sms, st) : launch<float, 1>(back, p, d.sms, st));
  return launch_code(v ? launch<Bf16, 8>(back, p, d.sms, st) : launch<Bf16, 1>(back, p, d.sms, st));
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
                 Convert{rows, cols, const_cast<void*>(x), ldx,
                         {static_cast<unsigned char*>(codes), ldq, static_cast<unsigned char*>(scales), lds}},
                 stream);
}

int b2g_dequantize8(int dtype, long long rows, int cols, const void* codes, long long ldq,
                    const void* scales, long long lds, void* y, long long ldy, void* stream) {
  const int rc = check(dtype, rows, cols, y, ldy, codes, ldq, scales, lds);
  if (rc || rows == 0 || cols == 0) return rc;
  return convert(true, dtype,
                 Convert{rows, cols, y, ldy,
                         {static_cast<unsigned char*>(const_cast<void*>(codes)), ldq,
                          static_cast<unsigned char*>(const_cast<void*>(scales)), lds}},
                 stream);
}

}  // extern "C"
