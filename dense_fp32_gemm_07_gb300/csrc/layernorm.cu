// layernorm.cu -- layer norm of matrix rows and its gradients
// (b2g_layernorm, b2g_layernorm_backward in include/b2g_train.h).
//
// Forward.  A row stays in registers between its one read and its one write:
// mean first, then the variance as the mean of (x - mean)^2, which loses no
// digits however large the mean is.  Bound: bytes (8 operations an element).
//
// Backward.  Persistent blocks walk the rows; each thread keeps the same
// columns throughout, so dy * xhat and dy add up in its registers, and a block
// leaves one FP32 partial row of each for a second kernel to add in block order
// (no atomics: the same bits every run).  x and dy are read once, dx written
// once.
#include "train_common.cuh"

namespace b2g {
namespace {

// ------------------------------------------------------------------- forward

struct LnFwd {
  long long rows;
  int cols, chunks;  // chunks = cols / VEC
  const void* x;
  long long ldx;
  const void* w;
  const void* b;
  float eps;
  void* y;
  long long ldy;
  float* mean;
  float* rstd;
};

// One row per blockDim.x threads (threadIdx.y picks the row of a one-warp-per-
// row block), NCH chunks of VEC columns per thread.  The weights are fetched
// with the row, ahead of the two sums, so that their latency is not added to
// the row's (one row of 4096: 5.0 us with, see below).
template <typename T, int VEC, int NCH>
__global__ void __launch_bounds__(512) ln_fwd_kernel(const __grid_constant__ LnFwd p) {
  __shared__ float red[2][32];
  pdl_launch_dependents();
  const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  const T* w = static_cast<const T*>(p.w);
  const T* b = static_cast<const T*>(p.b);
  pdl_wait();
  if (row >= p.rows) return;  // blockDim.y > 1 only with one warp per row: no barrier follows
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const int t = threadIdx.x, nt = blockDim.x;
  const int warps = nt >> 5;
  Pack<T, VEC> raw[NCH], wr[NCH], br[NCH];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = t + i * nt;
    raw[i].zero(), wr[i].zero(), br[i].zero();
    if (c < p.chunks) raw[i].load(x + c * VEC);
  }
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = t + i * nt;
    if (c < p.chunks) {
      if (w) wr[i].load(w + c * VEC);
      if (b) br[i].load(b + c * VEC);
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    float f[VEC];
    raw[i].get(f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) sum += f[j];
  }
  const float inv = 1.f / (float)p.cols;
  const float mean = block_sum(sum, red[0], warps) * inv;
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    float f[VEC];
    raw[i].get(f);
    if (t + i * nt < p.chunks) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) sq = fmaf(f[j] - mean, f[j] - mean, sq);
    }
  }
  const float rstd = 1.f / sqrtf(block_sum(sq, red[1], warps) * inv + p.eps);
  T* y = static_cast<T*>(p.y) + row * p.ldy;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = t + i * nt;
    if (c < p.chunks) {
      float f[VEC], wf[VEC], bf[VEC];
      raw[i].get(f), wr[i].get(wf), br[i].get(bf);
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        f[j] = fmaf((f[j] - mean) * rstd, w ? wf[j] : 1.f, bf[j]);
      Pack<T, VEC> o;
      o.set(f);
      o.store(y + c * VEC);
    }
  }
  if (t == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
}

// Rows wider than the registers of a block: three passes over the row (sum,
// squares, output), the later two from the caches.
template <typename T>
__global__ void __launch_bounds__(1024) ln_fwd_wide_kernel(const __grid_constant__ LnFwd p) {
  __shared__ float red[2][32];
  pdl_launch_dependents();
  pdl_wait();
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const T* w = static_cast<const T*>(p.w);
  const T* b = static_cast<const T*>(p.b);
  const int warps = blockDim.x >> 5;
  float sum = 0.f;
  for (int c = threadIdx.x; c < p.cols; c += blockDim.x) sum += to_f32(x[c]);
  const float inv = 1.f / (float)p.cols;
  const float mean = block_sum(sum, red[0], warps) * inv;
  float sq = 0.f;
  for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
    const float d = to_f32(x[c]) - mean;
    sq = fmaf(d, d, sq);
  }
  const float rstd = 1.f / sqrtf(block_sum(sq, red[1], warps) * inv + p.eps);
  T* y = static_cast<T*>(p.y) + row * p.ldy;
  for (int c = threadIdx.x; c < p.cols; c += blockDim.x)
    y[c] = from_f32<T>(fmaf((to_f32(x[c]) - mean) * rstd, w ? to_f32(w[c]) : 1.f,
                            b ? to_f32(b[c]) : 0.f));
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
}

// ------------------------------------------------------------------ backward

struct LnBwd {
  long long rows;
  int cols, chunks;
  const void* dy;
  long long lddy;
  const void* x;
  long long ldx;
  const void* w;
  const float* mean;
  const float* rstd;
  void* dx;
  long long lddx;
  float* part;  // [grid][2][cols]: partial dweight, then dbias; NULL: neither is wanted
};

// Block b takes rows b, b + grid, ...; thread t the chunks t + i * blockDim.x.
// The next row's x and dy are fetched before this row's two sums.
template <typename T, int VEC, int NCH>
__global__ void __launch_bounds__(512) ln_bwd_kernel(const __grid_constant__ LnBwd p) {
  __shared__ float red[2][64];
  pdl_launch_dependents();
  pdl_wait();
  const int t = threadIdx.x, nt = blockDim.x, warps = nt >> 5;
  const float inv = 1.f / (float)p.cols;
  float aw[NCH][VEC], ab[NCH][VEC];
  Pack<T, VEC> wr[NCH], xn[NCH], dn[NCH];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = t + i * nt;
    wr[i].zero(), xn[i].zero(), dn[i].zero();
    if (p.w && c < p.chunks) wr[i].load(static_cast<const T*>(p.w) + c * VEC);
#pragma unroll
    for (int j = 0; j < VEC; ++j) aw[i][j] = ab[i][j] = 0.f;
  }
  auto fetch = [&](long long row) {
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = t + i * nt;
      if (c < p.chunks) xn[i].load(x + c * VEC), dn[i].load(dy + c * VEC);
    }
  };
  long long row = blockIdx.x;
  float mean = 0.f, rstd = 0.f;
  if (row < p.rows) fetch(row), mean = p.mean[row], rstd = p.rstd[row];
  for (int it = 0; row < p.rows; row += gridDim.x, ++it) {
    float s1 = 0.f, s2 = 0.f;  // sums of g and of g * xhat
    Pack<T, VEC> xc[NCH], dc[NCH];
    const float m = mean, r = rstd;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      xc[i] = xn[i], dc[i] = dn[i];
      float xf[VEC], df[VEC], wf[VEC];
      xc[i].get(xf), dc[i].get(df), wr[i].get(wf);
      if (t + i * nt < p.chunks) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float xh = (xf[j] - m) * r, g = p.w ? df[j] * wf[j] : df[j];
          s1 += g, s2 = fmaf(g, xh, s2);
          aw[i][j] = fmaf(df[j], xh, aw[i][j]), ab[i][j] += df[j];
        }
      }
    }
    const long long next = row + gridDim.x;
    if (next < p.rows) fetch(next), mean = p.mean[next], rstd = p.rstd[next];
    const float2 s = block_sum2(s1, s2, red[it & 1], warps);
    const float c1 = s.x * inv, c2 = s.y * inv;
    T* dx = static_cast<T*>(p.dx) + row * p.lddx;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = t + i * nt;
      if (c < p.chunks) {
        float xf[VEC], df[VEC], wf[VEC], o[VEC];
        xc[i].get(xf), dc[i].get(df), wr[i].get(wf);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float xh = (xf[j] - m) * r, g = p.w ? df[j] * wf[j] : df[j];
          o[j] = r * (g - c1 - xh * c2);
        }
        Pack<T, VEC> v;
        v.set(o);
        v.store(dx + c * VEC);
      }
    }
  }
  if (p.part) {
    float* pw = p.part + (size_t)blockIdx.x * 2 * p.cols;
    float* pb = pw + p.cols;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = t + i * nt;
      if (c < p.chunks) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) pw[c * VEC + j] = aw[i][j], pb[c * VEC + j] = ab[i][j];
      }
    }
  }
}

// Rows wider than the registers of a block: dx in two passes over the row.
template <typename T>
__global__ void __launch_bounds__(1024) ln_bwd_wide_kernel(const __grid_constant__ LnBwd p) {
  __shared__ float red[64];
  pdl_launch_dependents();
  pdl_wait();
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
  const T* w = static_cast<const T*>(p.w);
  const float m = p.mean[row], r = p.rstd[row];
  float s1 = 0.f, s2 = 0.f;
  for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
    const float g = to_f32(dy[c]) * (w ? to_f32(w[c]) : 1.f);
    s1 += g, s2 = fmaf(g, (to_f32(x[c]) - m) * r, s2);
  }
  const float2 s = block_sum2(s1, s2, red, blockDim.x >> 5);
  const float inv = 1.f / (float)p.cols, c1 = s.x * inv, c2 = s.y * inv;
  T* dx = static_cast<T*>(p.dx) + row * p.lddx;
  for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
    const float g = to_f32(dy[c]) * (w ? to_f32(w[c]) : 1.f);
    const float xh = (to_f32(x[c]) - m) * r;
    dx[c] = from_f32<T>(r * (g - c1 - xh * c2));
  }
}

// The wide rows' dweight and dbias: block (x, y) adds rows y, y + gridDim.y, ...
// of its 256 columns into partial row y.  Runs before ln_bwd_wide_kernel, which
// may overwrite dy.
template <typename T>
__global__ void __launch_bounds__(256) ln_bwd_cols_kernel(const __grid_constant__ LnBwd p) {
  pdl_launch_dependents();
  pdl_wait();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= p.cols) return;
  float aw = 0.f, ab = 0.f;
  for (long long row = blockIdx.y; row < p.rows; row += gridDim.y) {
    const float d = to_f32(static_cast<const T*>(p.dy)[row * p.lddy + c]);
    const float xv = to_f32(static_cast<const T*>(p.x)[row * p.ldx + c]);
    aw = fmaf(d, (xv - p.mean[row]) * p.rstd[row], aw), ab += d;
  }
  float* pw = p.part + (size_t)blockIdx.y * 2 * p.cols;
  pw[c] = aw, pw[p.cols + c] = ab;
}

// dweight (blockIdx.y == 0) and dbias (1): the partial rows added in order, a
// quarter-interleaved set per warp, then the eight warps' sums in warp order.
template <typename T>
__global__ void __launch_bounds__(256) ln_bwd_reduce_kernel(const float* part, int parts, int cols,
                                                            T* dweight, T* dbias) {
  __shared__ float acc[8][32];
  pdl_launch_dependents();
  pdl_wait();
  T* out = blockIdx.y ? dbias : dweight;
  if (!out) return;
  const int c = blockIdx.x * 32 + threadIdx.x;
  float a = 0.f;
  if (c < cols) {
    const float* p0 = part + (size_t)blockIdx.y * cols + c;
#pragma unroll 4
    for (int i = threadIdx.y; i < parts; i += 8) a += p0[(size_t)i * 2 * cols];
  }
  acc[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  if (threadIdx.y == 0 && c < cols) {
#pragma unroll
    for (int i = 1; i < 8; ++i) a += acc[i][threadIdx.x];
    out[c] = from_f32<T>(a);
  }
}

// ----------------------------------------------------------------- host side

// Chunks a thread may hold (powers of two) without spilling at 512 threads.
template <int VEC>
constexpr int kMaxFwd = VEC == 1 ? 16 : 4;
template <int VEC>
constexpr int kMaxBwd = VEC == 1 ? 4 : 2;
constexpr int kMaxRowThreads = 512;

// Threads for one row of `chunks` chunks with at most `per` chunks a thread:
// the smallest power of two from 32 to kMaxRowThreads, or 0 when those are too few.
int row_threads(int chunks, int per) {
  for (int t = 32; t <= kMaxRowThreads; t *= 2)
    if ((long long)t * per >= chunks) return t;
  return 0;
}

template <typename T, int VEC, int NCH = 1>
cudaError_t fwd_kernel(int nch, dim3 grid, dim3 block, cudaStream_t st, const LnFwd& p) {
  if constexpr (NCH < kMaxFwd<VEC>) {
    if (nch > NCH) return fwd_kernel<T, VEC, 2 * NCH>(nch, grid, block, st, p);
  }
  return launch_train(ln_fwd_kernel<T, VEC, NCH>, grid, block, 0, st, p);
}

template <typename T, int VEC>
cudaError_t fwd_launch(LnFwd p, int sms, cudaStream_t st) {
  p.chunks = p.cols / VEC;
  // Few rows: one chunk a thread, for the shortest path; many: several, for the
  // fewest barriers per byte.
  int nt = p.rows <= 2 * sms ? row_threads(p.chunks, 1) : 0;
  if (!nt) nt = row_threads(p.chunks, kMaxFwd<VEC>);
  if (!nt)
    return launch_train(ln_fwd_wide_kernel<T>, dim3((unsigned)p.rows), dim3(1024), 0, st, p);
  const int ry = nt == 32 ? 4 : 1;
  const dim3 grid((unsigned)ceil_div(p.rows, ry)), block(nt, ry);
  return fwd_kernel<T, VEC>((int)ceil_div(p.chunks, nt), grid, block, st, p);
}

// Blocks of the backward kernel, each leaving one partial row of dweight and of
// dbias: about 1024 threads an SM, and few enough that the partial rows (two
// FP32 rows a block) stay a small share of the traffic.
int bwd_parts(long long rows, int cols, int sms) {
  const int nt = row_threads(cols, 16);
  const long long per_sm = nt == 0 || nt >= 512 ? 2 : 1024 / nt < 8 ? 1024 / nt : 8;
  const long long most = per_sm * sms, fair = ceil_div(rows, 4);
  return (int)(fair < most ? fair : most);
}

template <typename T, int VEC, int NCH = 1>
cudaError_t bwd_kernel(int nch, dim3 grid, dim3 block, cudaStream_t st, const LnBwd& p) {
  if constexpr (NCH < kMaxBwd<VEC>) {
    if (nch > NCH) return bwd_kernel<T, VEC, 2 * NCH>(nch, grid, block, st, p);
  }
  return launch_train(ln_bwd_kernel<T, VEC, NCH>, grid, block, 0, st, p);
}

template <typename T, int VEC>
cudaError_t bwd_launch(LnBwd p, T* dweight, T* dbias, int parts, cudaStream_t st) {
  p.chunks = p.cols / VEC;
  cudaError_t e = cudaSuccess;
  const int nt = row_threads(p.chunks, kMaxBwd<VEC>);
  if (nt) {
    e = bwd_kernel<T, VEC>((int)ceil_div(p.chunks, nt), dim3(parts), dim3(nt), st, p);
  } else {
    if (p.part)
      e = launch_train(ln_bwd_cols_kernel<T>, dim3((unsigned)ceil_div(p.cols, 256), parts),
                       dim3(256), 0, st, p);
    if (e == cudaSuccess)
      e = launch_train(ln_bwd_wide_kernel<T>, dim3((unsigned)p.rows), dim3(1024), 0, st, p);
  }
  if (e == cudaSuccess && p.part)
    e = launch_train(ln_bwd_reduce_kernel<T>, dim3((unsigned)ceil_div(p.cols, 32), 2),
                     dim3(32, 8), 0, st, (const float*)p.part, parts, p.cols, dweight, dbias);
  return e;
}

int check_rows(int dtype, long long rows, int cols) {
  if (!type_ok(dtype)) return B2G_ERR_INVALID_TYPE;
  if (rows < 0 || cols < 0 || rows > 0x7fffffffLL) return B2G_ERR_INVALID_DIM;
  return 0;
}

bool ld_ok(long long ld, int cols) { return ld >= (cols > 1 ? cols : 1); }

size_t bwd_bytes(long long rows, int cols, int sms) {
  return (size_t)bwd_parts(rows, cols, sms) * 2 * cols * sizeof(float);
}

}  // namespace
}  // namespace b2g

using namespace b2g;

extern "C" {

int b2g_layernorm(int dtype, long long rows, int cols, const void* x, long long ldx,
                  const void* weight, const void* bias, float eps, void* y, long long ldy,
                  float* mean, float* rstd, void* stream) {
  int rc = check_rows(dtype, rows, cols);
  if (rc) return rc;
  if (!(eps >= 0.f)) return B2G_ERR_INVALID_DIM;
  if (!ld_ok(ldx, cols) || !ld_ok(ldy, cols)) return B2G_ERR_INVALID_LD;
  if (rows == 0 || cols == 0) return 0;
  if (!x || !y) return B2G_ERR_NULL;
  TrainDevice d;
  rc = train_device(&d);
  if (rc) return rc;
  LnFwd p{rows, cols, 0, x, ldx, weight, bias, eps, y, ldy, mean, rstd};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool v = vec16(x) && vec16(y) && vec16(weight) && vec16(bias) && vec16_ld(ldx, dtype) &&
                 vec16_ld(ldy, dtype) && vec16_ld(cols, dtype);
  if (dtype == B2G_F32)
    return launch_code(v ? fwd_launch<float, 4>(p, d.sms, st) : fwd_launch<float, 1>(p, d.sms, st));
  return launch_code(v ? fwd_launch<Bf16, 8>(p, d.sms, st) : fwd_launch<Bf16, 1>(p, d.sms, st));
}

int b2g_layernorm_backward_workspace_size(int dtype, long long rows, int cols, size_t* bytes) {
  const int rc = check_rows(dtype, rows, cols);
  if (rc) return rc;
  if (!bytes) return B2G_ERR_NULL;
  TrainDevice d;
  const int sms = train_device(&d) ? 152 : d.sms;  // without a device: GB300's count
  *bytes = bwd_bytes(rows, cols, sms);
  return 0;
}

int b2g_layernorm_backward(int dtype, long long rows, int cols, const void* dy, long long lddy,
                           const void* x, long long ldx, const void* weight, const float* mean,
                           const float* rstd, void* dx, long long lddx, void* dweight, void* dbias,
                           void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_rows(dtype, rows, cols);
  if (rc) return rc;
  if (!ld_ok(lddy, cols) || !ld_ok(ldx, cols) || !ld_ok(lddx, cols)) return B2G_ERR_INVALID_LD;
  if (cols == 0) return 0;
  if (rows > 0 && (!dy || !x || !mean || !rstd || !dx)) return B2G_ERR_NULL;
  if (rows == 0 && !dweight && !dbias) return 0;
  TrainDevice d;
  rc = train_device(&d);
  if (rc) return rc;
  const bool sums = dweight || dbias;
  if (sums && rows > 0 &&
      (!workspace || !vec16(workspace) || workspace_bytes < bwd_bytes(rows, cols, d.sms)))
    return B2G_ERR_WORKSPACE;
  float* part = sums ? static_cast<float*>(workspace) : nullptr;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (rows == 0) {  // sums of nothing
    cudaError_t e = cudaSuccess;
    if (dweight) e = cudaMemsetAsync(dweight, 0, cols * type_size(dtype), st);
    if (dbias && e == cudaSuccess) e = cudaMemsetAsync(dbias, 0, cols * type_size(dtype), st);
    return e == cudaSuccess ? 0 : B2G_ERR_CUDA;
  }
  LnBwd p{rows, cols, 0, dy, lddy, x, ldx, weight, mean, rstd, dx, lddx, part};
  const int parts = bwd_parts(rows, cols, d.sms);
  const bool v = vec16(dy) && vec16(x) && vec16(weight) && vec16(dx) && vec16_ld(lddy, dtype) &&
                 vec16_ld(ldx, dtype) && vec16_ld(lddx, dtype) && vec16_ld(cols, dtype);
  if (dtype == B2G_F32) {
    float* dw = static_cast<float*>(dweight);
    float* db = static_cast<float*>(dbias);
    return launch_code(v ? bwd_launch<float, 4>(p, dw, db, parts, st)
                         : bwd_launch<float, 1>(p, dw, db, parts, st));
  }
  Bf16* dw = static_cast<Bf16*>(dweight);
  Bf16* db = static_cast<Bf16*>(dbias);
  return launch_code(v ? bwd_launch<Bf16, 8>(p, dw, db, parts, st)
                       : bwd_launch<Bf16, 1>(p, dw, db, parts, st));
}

}  // extern "C"
