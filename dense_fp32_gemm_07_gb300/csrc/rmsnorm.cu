// rmsnorm.cu -- root-mean-square norm of matrix rows with the residual's addition and
// 8-bit results, and its gradients (b2g_rmsnorm, b2g_rmsnorm_backward in
// include/b2g_train.h).
//
// Forward.  t = x + residual rounded to the type, rstd = 1 / sqrt(mean(t^2) + eps),
// y = t rstd weight.  A row stays in registers between its one read and its one write;
// t and y leave as they are, in 8 bits, or both.  Bound: bytes.
//
// Backward, with xhat = t rstd and g = dy weight:
//     dx = rstd (g - xhat mean(g xhat)) + dtotal,   dweight = sum over the rows of dy xhat.
// Persistent groups of threads walk the rows; a thread keeps the same columns throughout,
// so dweight adds up in its registers, and a block leaves one FP32 partial row for a second
// kernel to add in block order (no atomics: the same bits every run).
#include "eightbit.cuh"

namespace b2g {
namespace {

// ------------------------------------------------------------------- forward

struct RmsFwd {
  long long rows;
  int cols, chunks;  // chunks = cols / VEC
  const void* x;
  long long ldx;
  const void* res;
  long long ldr;
  const void* w;
  float eps;
  void* total;
  long long ldt;
  void* y;
  long long ldy;
  Rows8 y8, t8;
  float* rstd;
};

// A sum over the nt lanes (a power of two, up to 32, consecutive) that share a row, or
// over the nt threads of a block.
__device__ __forceinline__ float row_sum(float v, float* red, int nt) {
  if (nt > 32) return block_sum(v, red, nt >> 5);
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    if (o < nt) v += w;
  }
  return v;
}

// One row per blockDim.x threads (from 8 lanes of a warp up; threadIdx.y picks the row of
// a block that has several), NCH chunks of VEC columns a thread.
template <typename T, int VEC, int NCH>
__global__ void __launch_bounds__(512) rms_fwd_kernel(const __grid_constant__ RmsFwd p) {
  __shared__ float red[32];
  pdl_launch_dependents();
  pdl_wait();
  const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < p.rows;  // the others of the warp take part in its sums
  const int t = threadIdx.x, nt = blockDim.x, chunks = live ? p.chunks : 0;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const T* r = static_cast<const T*>(p.res) + row * p.ldr;
  const T* w = static_cast<const T*>(p.w);
  Pack<T, VEC> raw[NCH], add[NCH], wr[NCH];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = t + i * nt;
    raw[i].zero(), add[i].zero(), wr[i].zero();
    if (c < chunks) {
      raw[i].load(x + c * VEC);
      if (p.res) add[i].load(r + c * VEC);
      if (w) wr[i].load(w + c * VEC);
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = t + i * nt;
    float f[VEC];
    raw[i].get(f);
    if (p.res) {
      float g[VEC];
      add[i].get(g);
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[j] += g[j];
      raw[i].set(f);
      raw[i].get(f);
    }
    if (p.total && c < chunks) raw[i].store(static_cast<T*>(p.total) + row * p.ldt + c * VEC);
#pragma unroll
    for (int j = 0; j < VEC; ++j) sum = fmaf(f[j], f[j], sum);
    if (p.t8.q) encode_to<VEC>(p.t8, row, c, c < chunks, f);
  }
  const float rstd = 1.f / sqrtf(row_sum(sum, red, nt) / (float)p.cols + p.eps);
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = t + i * nt;
    float f[VEC], wf[VEC];
    raw[i].get(f), wr[i].get(wf);
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = f[j] * rstd * (w ? wf[j] : 1.f);
    if (p.y && c < chunks) {
      Pack<T, VEC> o;
      o.set(f);
      o.store(static_cast<T*>(p.y) + row * p.ldy + c * VEC);
    }
    if (p.y8.q) encode_to<VEC>(p.y8, row, c, c < chunks, f);
  }
  if (t == 0 && live && p.rstd) p.rstd[row] = rstd;
}

// Rows wider than the registers of a block: two passes, the second one from the caches.
template <typename T>
__global__ void __launch_bounds__(1024) rms_fwd_wide_kernel(const __grid_constant__ RmsFwd p) {
  __shared__ float red[32];
  pdl_launch_dependents();
  pdl_wait();
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const T* r = static_cast<const T*>(p.res) + row * p.ldr;
  const T* w = static_cast<const T*>(p.w);
  auto at = [&](int c) {
    return p.res ? to_f32(from_f32<T>(to_f32(x[c]) + to_f32(r[c]))) : to_f32(x[c]);
  };
  float sum = 0.f;
  for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
    const float v = at(c);
    sum = fmaf(v, v, sum);
  }
  const float rstd = 1.f / sqrtf(block_sum(sum, red, blockDim.x >> 5) / (float)p.cols + p.eps);
  // whole blocks of 32 columns, for the scales
  const int end = (int)(scale_count(p.cols) * kScaleBlock);
  for (int c = threadIdx.x; c < end; c += blockDim.x) {
    const bool in = c < p.cols;
    float f[1] = {in ? at(c) : 0.f};
    const float v = f[0] * rstd * (w && in ? to_f32(w[c]) : 1.f);
    if (in) {
      if (p.total) static_cast<T*>(p.total)[row * p.ldt + c] = from_f32<T>(f[0]);
      if (p.y) static_cast<T*>(p.y)[row * p.ldy + c] = from_f32<T>(v);
    }
    if (p.t8.q) encode_to<1>(p.t8, row, c, in, f);
    f[0] = v;
    if (p.y8.q) encode_to<1>(p.y8, row, c, in, f);
  }
  if (threadIdx.x == 0 && p.rstd) p.rstd[row] = rstd;
}

// ------------------------------------------------------------------ backward

struct RmsBwd {
  long long rows;
  int cols, chunks;
  const void* dy;
  long long lddy;
  const void* x;   // the rows, or NULL: k8
  long long ldx;
  Rows8 k8;
  const void* w;
  const float* rstd;
  const void* dtotal;
  long long lddt;
  void* dx;
  long long lddx;
  float* part;  // [grid][cols]: partial dweight; NULL: it is not wanted
};

constexpr int kBwdThreads = 512;  // 16 columns a thread

// VEC columns of a row of t, from the type or from 8 bits.
template <typename T, int VEC, bool Q8>
__device__ __forceinline__ void load_t(const RmsBwd& p, long long row, int c, float (&f)[VEC]) {
  if constexpr (Q8) {
    Codes<VEC> k;
    k.load(p.k8.q + row * p.k8.ldq + (long long)c * VEC);
    const float s = scale_value(p.k8.s[row * p.k8.lds + c / (kScaleBlock / VEC)]);
    k.get(f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] *= s;
  } else {
    Pack<T, VEC> k;
    k.load(static_cast<const T*>(p.x) + row * p.ldx + (long long)c * VEC);
    k.get(f);
  }
}

// Sum over a group's nt threads (whole warps); `ex` is one of two buffers used by turns.
__device__ __forceinline__ float group_sum(float v, float (&ex)[16], int group, int nt) {
  v = warp_sum(v);
  const int warps = nt >> 5, lane = threadIdx.x & 31;
  if (warps == 1) return v;
  if (lane == 0) ex[threadIdx.x >> 5] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(nt) : "memory");
  v = lane < warps ? ex[group * warps + lane] : 0.f;
#pragma unroll
  for (int o = 8; o; o >>= 1)
    if (o < warps) v += __shfl_xor_sync(0xffffffffu, v, o);
  return __shfl_sync(0xffffffffu, v, 0);
}

// Groups of nt threads with a row each, 16 columns a thread.
template <typename T, int VEC, bool Q8>
__global__ void __launch_bounds__(kBwdThreads, 1)
    rms_bwd_kernel(const __grid_constant__ RmsBwd p, int nt, int groups) {
  extern __shared__ float sums[];  // [groups][cols], at the end
  __shared__ float red[2][16];
  constexpr int NCH = 16 / VEC;
  pdl_launch_dependents();
  pdl_wait();
  const int group = threadIdx.x / nt, t = threadIdx.x - group * nt;
  const float inv = 1.f / (float)p.cols;
  const T* w = static_cast<const T*>(p.w);
  float aw[NCH][VEC], wf[NCH][VEC];
  auto weight = [&](int i) {
    const int c = t + i * nt;
#pragma unroll
    for (int j = 0; j < VEC; ++j) wf[i][j] = 1.f;
    if (w && c < p.chunks) {
      Pack<T, VEC> k;
      k.load(w + c * VEC);
      k.get(wf[i]);
    }
  };
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) aw[i][j] = 0.f;
    if (VEC > 1) weight(i);
  }
  int turn = 0;
  for (long long row = (long long)group * gridDim.x + blockIdx.x; row < p.rows;
       row += (long long)gridDim.x * groups) {
    if (VEC == 1) asm volatile("" ::: "memory");  // nothing that depends on the column stays
    const float rstd = p.rstd[row];
    float xh[NCH][VEC], g[NCH][VEC], along = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = t + i * nt;
      if (c < p.chunks) {
        Pack<T, VEC> k;
        k.load(static_cast<const T*>(p.dy) + row * p.lddy + (long long)c * VEC);
        k.get(g[i]);
        load_t<T, VEC, Q8>(p, row, c, xh[i]);
        if (VEC == 1) weight(i);  // single elements: no registers to keep them in
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          xh[i][j] *= rstd;
          aw[i][j] = fmaf(g[i][j], xh[i][j], aw[i][j]);
          g[i][j] *= wf[i][j];
          along = fmaf(g[i][j], xh[i][j], along);
        }
      }
    }
    const float mean = group_sum(along, red[turn], group, nt) * inv;
    turn ^= 1;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = t + i * nt;
      if (c < p.chunks) {
        Pack<T, VEC> k;
        float d[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) d[j] = 0.f;
        if (p.dtotal) {
          k.load(static_cast<const T*>(p.dtotal) + row * p.lddt + (long long)c * VEC);
          k.get(d);
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) d[j] = fmaf(rstd, g[i][j] - xh[i][j] * mean, d[j]);
        k.set(d);
        k.store(static_cast<T*>(p.dx) + row * p.lddx + (long long)c * VEC);
      }
    }
  }
  if (!p.part) return;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = t + i * nt;
    if (c < p.chunks) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) sums[(size_t)group * p.cols + c * VEC + j] = aw[i][j];
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < p.cols; c += kBwdThreads) {
    float a = sums[c];
    for (int i = 1; i < groups; ++i) a += sums[(size_t)i * p.cols + c];
    p.part[(size_t)blockIdx.x * p.cols + c] = a;
  }
}

// Rows wider than the registers of a block: dx in two passes over the row.
template <typename T, bool Q8>
__global__ void __launch_bounds__(1024) rms_bwd_wide_kernel(const __grid_constant__ RmsBwd p) {
  __shared__ float red[32];
  pdl_launch_dependents();
  pdl_wait();
  const long long row = blockIdx.x;
  const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
  const T* w = static_cast<const T*>(p.w);
  const float rstd = p.rstd[row];
  float along = 0.f, t[1];
  for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
    load_t<T, 1, Q8>(p, row, c, t);
    along = fmaf(to_f32(dy[c]) * (w ? to_f32(w[c]) : 1.f), t[0] * rstd, along);
  }
  const float mean = block_sum(along, red, blockDim.x >> 5) / (float)p.cols;
  for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
    load_t<T, 1, Q8>(p, row, c, t);
    const float g = to_f32(dy[c]) * (w ? to_f32(w[c]) : 1.f);
    const float d = p.dtotal ? to_f32(static_cast<const T*>(p.dtotal)[row * p.lddt + c]) : 0.f;
    static_cast<T*>(p.dx)[row * p.lddx + c] = from_f32<T>(fmaf(rstd, g - t[0] * rstd * mean, d));
  }
}

// The wide rows' dweight: block (x, y) adds rows y, y + gridDim.y, ... of its 256 columns
// into partial row y.  Runs before rms_bwd_wide_kernel, which may overwrite dy.
template <typename T, bool Q8>
__global__ void __launch_bounds__(256) rms_bwd_cols_kernel(const __grid_constant__ RmsBwd p) {
  pdl_launch_dependents();
  pdl_wait();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= p.cols) return;
  float a = 0.f, t[1];
  for (long long row = blockIdx.y; row < p.rows; row += gridDim.y) {
    load_t<T, 1, Q8>(p, row, c, t);
    a = fmaf(to_f32(static_cast<const T*>(p.dy)[row * p.lddy + c]), t[0] * p.rstd[row], a);
  }
  p.part[(size_t)blockIdx.y * p.cols + c] = a;
}

// dweight: warp y adds the partial rows y, y + 16, ... in order, then the warps' sums are
// added in warp order.
template <typename T>
__global__ void __launch_bounds__(512) rms_bwd_reduce_kernel(const float* part, int parts, int cols,
                                                             T* dweight) {
  __shared__ float acc[16][32];
  pdl_launch_dependents();
  pdl_wait();
  const int c = blockIdx.x * 32 + threadIdx.x;
  float a = 0.f;
  if (c < cols) {
#pragma unroll 10
    for (int i = threadIdx.y; i < parts; i += 16) a += part[(size_t)i * cols + c];
  }
  acc[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  if (threadIdx.y == 0 && c < cols) {
#pragma unroll
    for (int i = 1; i < 16; ++i) a += acc[i][threadIdx.x];
    dweight[c] = from_f32<T>(a);
  }
}

// ----------------------------------------------------------------- host side

// Chunks a thread may hold (powers of two).
template <int VEC>
constexpr int kMaxFwd = VEC == 1 ? 16 : 4;

// Threads for one row of `chunks` chunks with at most `per` chunks a thread: the smallest
// power of two from `least` to 512, or 0 when those are too few.
int row_threads(int chunks, int per, int least) {
  for (int t = least; t <= 512; t *= 2)
    if ((long long)t * per >= chunks) return t;
  return 0;
}

template <typename T, int VEC, int NCH = 1>
cudaError_t fwd_kernel(int nch, dim3 grid, dim3 block, cudaStream_t st, const RmsFwd& p) {
  if constexpr (NCH < kMaxFwd<VEC>) {
    if (nch > NCH) return fwd_kernel<T, VEC, 2 * NCH>(nch, grid, block, st, p);
  }
  return launch_train(rms_fwd_kernel<T, VEC, NCH>, grid, block, 0, st, p);
}

template <typename T, int VEC>
cudaError_t fwd_launch(RmsFwd p, int sms, cudaStream_t st) {
  p.chunks = p.cols / VEC;
  // a block of 32 columns stays within a warp: 8 lanes at 4 columns, 32 at single ones
  constexpr int least = VEC > 1 ? 8 : 32;
  int nt = p.rows <= 2 * sms ? row_threads(p.chunks, 1, least) : 0;
  if (!nt) nt = row_threads(p.chunks, kMaxFwd<VEC>, least);
  if (!nt)
    return launch_train(rms_fwd_wide_kernel<T>, dim3((unsigned)p.rows), dim3(1024), 0, st, p);
  const int ry = nt <= 32 ? 128 / nt : 1;
  const dim3 grid((unsigned)ceil_div(p.rows, ry)), block(nt, ry);
  return fwd_kernel<T, VEC>((int)ceil_div(p.chunks, nt), grid, block, st, p);
}

// Threads and groups of the backward kernel; groups == 0: the rows are too wide.
struct Groups {
  int nt, groups;
};
Groups groups_of(int cols) {
  Groups g{32, 0};
  while (g.nt < kBwdThreads && g.nt * 16 < cols) g.nt *= 2;
  if (g.nt * 16 >= cols) g.groups = kBwdThreads / g.nt;
  return g;
}

// Blocks of a backward kernel, each leaving one partial row of dweight.
int bwd_parts(long long rows, int cols, int sms) {
  const Groups g = groups_of(cols);
  const long long most = g.groups ? sms : 4LL * sms, fair = ceil_div(rows, g.groups ? g.groups : 4);
  return (int)(fair < most ? fair : most);
}

template <typename T, int VEC, bool Q8>
cudaError_t bwd_launch(RmsBwd p, T* dweight, int parts, cudaStream_t st) {
  p.chunks = p.cols / VEC;
  cudaError_t e = cudaSuccess;
  const Groups g = groups_of(p.cols);
  if (g.groups) {
    e = launch_train(rms_bwd_kernel<T, VEC, Q8>, dim3(parts), dim3(kBwdThreads),
                     (size_t)g.groups * p.cols * sizeof(float), st, p, g.nt, g.groups);
  } else {
    if (p.part)
      e = launch_train(rms_bwd_cols_kernel<T, Q8>, dim3((unsigned)ceil_div(p.cols, 256), parts),
                       dim3(256), 0, st, p);
    if (e == cudaSuccess)
      e = launch_train(rms_bwd_wide_kernel<T, Q8>, dim3((unsigned)p.rows), dim3(1024), 0, st, p);
  }
  if (e == cudaSuccess && p.part)
    e = launch_train(rms_bwd_reduce_kernel<T>, dim3((unsigned)ceil_div(p.cols, 32)), dim3(32, 16), 0,
                     st, (const float*)p.part, parts, p.cols, dweight);
  return e;
}

int check_rows(int dtype, long long rows, int cols) {
  if (!type_ok(dtype)) return B2G_ERR_INVALID_TYPE;
  if (rows < 0 || cols < 0 || rows > 0x7fffffffLL || cols > kMaxLength) return B2G_ERR_INVALID_DIM;
  return 0;
}

bool ld_ok(const void* p, long long ld, int cols) { return !p || ld >= (cols > 1 ? cols : 1); }
bool codes_ok(const Rows8& k, int cols) {
  return ld_ok(k.q, k.ldq, cols) && (!k.q || k.lds >= scale_count(cols > 1 ? cols : 1));
}

size_t bwd_bytes(long long rows, int cols, int sms) {
  return (size_t)bwd_parts(rows, cols, sms) * cols * sizeof(float);
}

Rows8 rows8(void* q, long long ldq, void* s, long long lds) {
  return Rows8{static_cast<unsigned char*>(q), ldq, static_cast<unsigned char*>(s), lds};
}

}  // namespace
}  // namespace b2g

using namespace b2g;

extern "C" {

int b2g_rmsnorm(int dtype, long long rows, int cols, const void* x, long long ldx,
                const void* residual, long long ldr, const void* weight, float eps, void* total,
                long long ldt, void* y, long long ldy, void* y_codes, long long ldyq, void* y_scales,
                long long ldys, void* total_codes, long long ldtq, void* total_scales,
                long long ldts, float* rstd, void* stream) {
  int rc = check_rows(dtype, rows, cols);
  if (rc) return rc;
  if (!(eps >= 0.f)) return B2G_ERR_INVALID_DIM;
  const Rows8 y8 = rows8(y_codes, ldyq, y_scales, ldys);
  const Rows8 t8 = rows8(total_codes, ldtq, total_scales, ldts);
  if (!ld_ok(&rc, ldx, cols) || !ld_ok(residual, ldr, cols) || !ld_ok(total, ldt, cols) ||
      !ld_ok(y, ldy, cols) || !codes_ok(y8, cols) || !codes_ok(t8, cols))
    return B2G_ERR_INVALID_LD;
  if (rows == 0 || cols == 0) return 0;
  if (!x || (!y8.q) != (!y8.s) || (!t8.q) != (!t8.s)) return B2G_ERR_NULL;
  TrainDevice d;
  rc = train_device(&d);
  if (rc) return rc;
  const RmsFwd p{rows, cols, 0,   x,  ldx, residual, ldr,  weight, eps,
                 total, ldt, y,   ldy, y8, t8,       rstd};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto row16 = [&](const void* q, long long ld) { return !q || (vec16(q) && vec16_ld(ld, dtype)); };
  const int vec = dtype == B2G_F32 ? 4 : 8;
  const bool v = row16(x, ldx) && row16(residual, ldr) && row16(total, ldt) && row16(y, ldy) &&
                 row16(weight, cols) && vec16_ld(cols, dtype) && codes_vec(y8, vec) &&
                 codes_vec(t8, vec);
  if (dtype == B2G_F32)
    return launch_code(v ? fwd_launch<float, 4>(p, d.sms, st) : fwd_launch<float, 1>(p, d.sms, st));
  return launch_code(v ? fwd_launch<Bf16, 8>(p, d.sms, st) : fwd_launch<Bf16, 1>(p, d.sms, st));
}

int b2g_rmsnorm_backward_workspace_size(int dtype, long long rows, int cols, size_t* bytes) {
  const int rc = check_rows(dtype, rows, cols);
  if (rc) return rc;
  if (!bytes) return B2G_ERR_NULL;
  TrainDevice d;
  const int sms = train_device(&d) ? 152 : d.sms;  // without a device: GB300's count
  *bytes = bwd_bytes(rows, cols, sms);
  return 0;
}

int b2g_rmsnorm_backward(int dtype, long long rows, int cols, const void* dy, long long lddy,
                         const void* total, long long ldt, const void* total_scales, long long ldts,
                         const void* weight, const float* rstd, const void* dtotal, long long lddt,
                         void* dx, long long lddx, void* dweight, void* workspace,
                         size_t workspace_bytes, void* stream) {
  int rc = check_rows(dtype, rows, cols);
  if (rc) return rc;
  const Rows8 k8 = total_scales ? rows8(const_cast<void*>(total), ldt, const_cast<void*>(total_scales), ldts)
                                : Rows8{};
  if (!ld_ok(&rc, lddy, cols) || !ld_ok(&rc, ldt, cols) || !codes_ok(k8, cols) ||
      !ld_ok(dtotal, lddt, cols) || !ld_ok(&rc, lddx, cols))
    return B2G_ERR_INVALID_LD;
  if (cols == 0 || (rows == 0 && !dweight)) return 0;
  if (rows > 0 && (!dy || !total || !rstd || !dx)) return B2G_ERR_NULL;
  TrainDevice d;
  rc = train_device(&d);
  if (rc) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (rows == 0)  // a sum of nothing
    return cudaMemsetAsync(dweight, 0, cols * type_size(dtype), st) == cudaSuccess ? 0 : B2G_ERR_CUDA;
  if (dweight &&
      (!workspace || !vec16(workspace) || workspace_bytes < bwd_bytes(rows, cols, d.sms)))
    return B2G_ERR_WORKSPACE;
  const RmsBwd p{rows,   cols,   0,    dy, lddy, total_scales ? nullptr : total, ldt, k8,
                 weight, rstd, dtotal, lddt, dx, lddx, dweight ? static_cast<float*>(workspace) : nullptr};
  auto row16 = [&](const void* q, long long ld) { return !q || (vec16(q) && vec16_ld(ld, dtype)); };
  const bool q8 = total_scales != nullptr;
  const bool v = row16(dy, lddy) && row16(p.x, ldt) && codes_vec(k8, dtype == B2G_F32 ? 4 : 8) &&
                 row16(dtotal, lddt) && row16(dx, lddx) && row16(weight, cols) &&
                 vec16_ld(cols, dtype);
  const int parts = bwd_parts(rows, cols, d.sms);
  if (dtype == B2G_F32) {
    float* dw = static_cast<float*>(dweight);
    return launch_code(v ? (q8 ? bwd_launch<float, 4, true>(p, dw, parts, st)
                               : bwd_launch<float, 4, false>(p, dw, parts, st))
                         : (q8 ? bwd_launch<float, 1, true>(p, dw, parts, st)
                               : bwd_launch<float, 1, false>(p, dw, parts, st)));
  }
  Bf16* dw = static_cast<Bf16*>(dweight);
  return launch_code(v ? (q8 ? bwd_launch<Bf16, 8, true>(p, dw, parts, st)
                             : bwd_launch<Bf16, 8, false>(p, dw, parts, st))
                       : (q8 ? bwd_launch<Bf16, 1, true>(p, dw, parts, st)
                             : bwd_launch<Bf16, 1, false>(p, dw, parts, st)));
}

}  // extern "C"
