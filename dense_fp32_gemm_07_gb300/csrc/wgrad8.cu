// wgrad8.cu -- a linear layer's weight gradient dw = dy^T x from an x kept in 8 bits
// (b2g_linear_dweight8 in include/b2g_train.h).
//
// Blocks of 64 x 64 results, 4 x 4 a thread, 16 tokens at a time through shared memory.
#include "eightbit.cuh"

namespace b2g {
namespace {

struct Dw8 {
  int tokens, outs, width;
  const void* dy;
  long long lddy;
  Rows8 x;
  int accumulate;
  void* dw;
  long long lddw;
};

template <typename T>
__global__ void __launch_bounds__(256) dw8_kernel(const __grid_constant__ Dw8 p) {
  __shared__ float a[16][64], b[16][64];
  pdl_launch_dependents();
  pdl_wait();
  const int n0 = blockIdx.x * 64, m0 = blockIdx.y * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < p.tokens; k0 += 16) {
    __syncthreads();
    for (int i = threadIdx.x; i < 1024; i += 256) {
      const int k = i >> 6, c = i & 63;
      const long long row = k0 + k;
      const bool in = row < p.tokens;
      a[k][c] = in && m0 + c < p.outs ? to_f32(static_cast<const T*>(p.dy)[row * p.lddy + m0 + c]) : 0.f;
      float v = 0.f, none;
      if (in && n0 + c < p.width) {
        decode2(p.x.q[row * p.x.ldq + n0 + c], v, none);
        v *= scale_value(p.x.s[row * p.x.lds + (n0 + c) / kScaleBlock]);
      }
      b[k][c] = v;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[k][ty * 4 + i], b[k][tx * 4 + j], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m < p.outs && n < p.width) {
        T* o = static_cast<T*>(p.dw) + m * p.lddw + n;
        *o = from_f32<T>(p.accumulate ? acc[i][j] + to_f32(*o) : acc[i][j]);
      }
    }
}

int check(int dtype, int tokens, int outs, int width) {
  if (!type_ok(dtype)) return B2G_ERR_INVALID_TYPE;
  if (tokens < 0 || outs < 0 || width < 0 || tokens > kMaxLength || outs > kMaxLength ||
      width > kMaxLength)
    return B2G_ERR_INVALID_DIM;
  return 0;
}

}  // namespace
}  // namespace b2g

using namespace b2g;

extern "C" {

int b2g_linear_dweight8_workspace_size(int dtype, int tokens, int outs, int width, const void* dy,
                                       long long lddy, size_t* bytes) {
  const int rc = check(dtype, tokens, outs, width);
  if (rc) return rc;
  if (!bytes) return B2G_ERR_NULL;
  *bytes = 0;
  return 0;
}

int b2g_linear_dweight8(int dtype, int tokens, int outs, int width, const void* dy, long long lddy,
                        const void* codes, long long ldq, const void* scales, long long lds,
                        int accumulate, void* dw, long long lddw, void* workspace,
                        size_t workspace_bytes, void* stream) {
  int rc = check(dtype, tokens, outs, width);
  if (rc) return rc;
  auto least = [](int n) { return n > 1 ? n : 1; };
  if (lddy < least(outs) || ldq < least(width) || lds < scale_count(least(width)) ||
      lddw < least(width))
    return B2G_ERR_INVALID_LD;
  if (outs == 0 || width == 0 || (tokens == 0 && accumulate)) return 0;
  if (!dw || (tokens > 0 && (!dy || !codes || !scales))) return B2G_ERR_NULL;
  TrainDevice d;
  rc = train_device(&d);
  if (rc) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Dw8 p{tokens, outs, width, dy, lddy,
        {static_cast<unsigned char*>(const_cast<void*>(codes)), ldq,
         static_cast<unsigned char*>(const_cast<void*>(scales)), lds},
        accumulate, dw, lddw};
  const dim3 grid((unsigned)ceil_div(width, 64), (unsigned)ceil_div(outs, 64));
  return launch_code(dtype == B2G_F32 ? launch_train(dw8_kernel<float>, grid, dim3(256), 0, st, p)
                                      : launch_train(dw8_kernel<Bf16>, grid, dim3(256), 0, st, p));
}

}  // extern "C"
