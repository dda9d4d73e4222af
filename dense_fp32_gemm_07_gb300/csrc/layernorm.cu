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
//
// Rows on 16-byte boundaries run on kernels that keep the next rows on their way
// while one is worked on (registers in the forward pass, a ring of bulk copies in
// shared memory in the backward pass); other rows are read element by element.
#include <atomic>

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

// Many rows: 16 warps per SM, G warps per row, each thread with NCH chunks of the
// row at hand and the same chunks of its next row already on their way.  With two
// warps a row, 8192 rows of 4096 BF16 values keep 128 KB an SM in flight.
template <typename T, int VEC, int NCH, int G>
__global__ void __launch_bounds__(512, 1) ln_fwd_rows_kernel(const __grid_constant__ LnFwd p) {
  constexpr int NT = 32 * G, GROUPS = 16 / G;
  __shared__ float red[2][16];
  pdl_launch_dependents();
  pdl_wait();
  const int group = threadIdx.x / NT, t = threadIdx.x % NT;
  const T* w = static_cast<const T*>(p.w);
  const T* b = static_cast<const T*>(p.b);
  const float inv = 1.f / (float)p.cols;
  const long long step = (long long)gridDim.x * GROUPS;
  long long row = (long long)group * gridDim.x + blockIdx.x;
  Pack<T, VEC> next[NCH];
  auto fetch = [&](long long r) {
    const T* x = static_cast<const T*>(p.x) + r * p.ldx;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = t + i * NT;
      if (c < p.chunks) next[i].load(x + c * VEC);
    }
  };
  // Sum over the group's threads; `k` alternates the exchange buffers.
  auto total = [&](float v, int k) {
    v = warp_sum(v);
    if (G == 1) return v;
    float* mine = red[k] + group * G;
    if ((threadIdx.x & 31) == 0) mine[(threadIdx.x % NT) / 32] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(NT) : "memory");
    float s = mine[0];
#pragma unroll
    for (int i = 1; i < G; ++i) s += mine[i];
    return s;
  };
#pragma unroll
  for (int i = 0; i < NCH; ++i) next[i].zero();
  if (row < p.rows) fetch(row);
  for (; row < p.rows; row += step) {
    Pack<T, VEC> raw[NCH];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      raw[i] = next[i];
      float f[VEC];
      raw[i].get(f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) sum += f[j];
    }
    if (row + step < p.rows) fetch(row + step);
    const float mean = total(sum, 0) * inv;
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      float f[VEC];
      raw[i].get(f);
      if (t + i * NT < p.chunks) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) sq = fmaf(f[j] - mean, f[j] - mean, sq);
      }
    }
    const float rstd = 1.f / sqrtf(total(sq, 1) * inv + p.eps);
    T* y = static_cast<T*>(p.y) + row * p.ldy;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = t + i * NT;
      if (c < p.chunks) {
        Pack<T, VEC> k;
        float f[VEC], wf[VEC], bf[VEC];
        raw[i].get(f);
        k.zero();
        if (w) k.load(w + c * VEC);
        k.get(wf);
        k.zero();
        if (b) k.load(b + c * VEC);
        k.get(bf);
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[j] = fmaf((f[j] - mean) * rstd, w ? wf[j] : 1.f, bf[j]);
        k.set(f);
        k.store(y + c * VEC);
      }
    }
    if (t == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
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

// The same for rows on 16-byte boundaries: one block of 512 threads an SM in groups
// of NT threads, a row per group.  A group's first thread keeps `stages` rows of x
// and dy on their way into the group's ring in shared memory (bulk copies that
// arrive on a barrier per slot; 160 KB an SM), so the rows' latency is not waited
// for; a slot is refilled once the group's sums have been exchanged, when every
// thread has read it.  At the end the groups' column sums are added in shared
// memory in group order.
constexpr int kRingBytes = 160 * 1024;
constexpr int kRingStages = 16;  // at most

template <typename T, int VEC, int NCH>
__global__ void __launch_bounds__(512, 1)
    ln_bwd_ring_kernel(const __grid_constant__ LnBwd p, int nt, int stages,
                       unsigned int* status, unsigned long long wait_limit_ns) {
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ __align__(8) unsigned long long bars[512 / 32 * kRingStages];
  __shared__ float red[2][2][16];
  pdl_launch_dependents();
  const int group = threadIdx.x / nt, t = threadIdx.x - group * nt, groups = 512 / nt;
  const int warps = nt >> 5;
  const uint32_t bytes = (uint32_t)(p.cols * (int)sizeof(T));
  const uint32_t bar0 = smem_addr(bars) + 8u * (uint32_t)(group * kRingStages);
  unsigned char* mine = ring + (size_t)group * stages * 2 * bytes;
  if (t == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(bar0 + 8u * s, 1);
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  __syncthreads();
  pdl_wait();
  const float inv = 1.f / (float)p.cols;
  const long long step = (long long)gridDim.x * groups;
  const long long row0 = (long long)group * gridDim.x + blockIdx.x;
  auto issue = [&](long long row, int s) {
    const uint32_t bar = bar0 + 8u * s, dst = smem_addr(mine + (size_t)s * 2 * bytes);
    mbar_arrive_expect_tx(bar, 2 * bytes);
    bulk_load(dst, static_cast<const T*>(p.x) + row * p.ldx, bytes, bar);
    bulk_load(dst + bytes, static_cast<const T*>(p.dy) + row * p.lddy, bytes, bar);
  };
  if (t == 0) {
    long long row = row0;
    for (int s = 0; s < stages && row < p.rows; ++s, row += step) issue(row, s);
  }
  float aw[NCH][VEC], ab[NCH][VEC];
  Pack<T, VEC> wr[NCH];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = t + i * nt;
    wr[i].zero();
    if (p.w && c < p.chunks) wr[i].load(static_cast<const T*>(p.w) + c * VEC);
#pragma unroll
    for (int j = 0; j < VEC; ++j) aw[i][j] = ab[i][j] = 0.f;
  }
  float mean = 0.f, rstd = 0.f;
  if (row0 < p.rows) mean = p.mean[row0], rstd = p.rstd[row0];
  int s = 0, k = 0;
  uint32_t ph = 0;
  bool alive = true;  // false once a wait has run out: no more waits, no more copies
  for (long long row = row0; row < p.rows; row += step) {
    const float m = mean, r = rstd;
    if (row + step < p.rows) mean = p.mean[row + step], rstd = p.rstd[row + step];
    if (alive)
      alive = mbar_wait(bar0 + 8u * s, ph, wait_limit_ns, status, kStatusTimeoutFull);
    const T* xs = reinterpret_cast<const T*>(mine + (size_t)s * 2 * bytes);
    const T* ds = reinterpret_cast<const T*>(mine + (size_t)s * 2 * bytes + bytes);
    Pack<T, VEC> xc[NCH], dc[NCH];
    float s1 = 0.f, s2 = 0.f;  // sums of g and of g * xhat
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = t + i * nt;
      xc[i].zero(), dc[i].zero();
      if (c < p.chunks) {
        xc[i].load(xs + c * VEC), dc[i].load(ds + c * VEC);
        float xf[VEC], df[VEC], wf[VEC];
        xc[i].get(xf), dc[i].get(df), wr[i].get(wf);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float xh = (xf[j] - m) * r, g = p.w ? df[j] * wf[j] : df[j];
          s1 += g, s2 = fmaf(g, xh, s2);
          aw[i][j] = fmaf(df[j], xh, aw[i][j]), ab[i][j] += df[j];
        }
      }
    }
    s1 = warp_sum(s1), s2 = warp_sum(s2);
    if (warps > 1) {
      float(&ex)[2][16] = red[k];
      if ((threadIdx.x & 31) == 0) ex[0][threadIdx.x >> 5] = s1, ex[1][threadIdx.x >> 5] = s2;
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(nt) : "memory");
      s1 = s2 = 0.f;
      for (int i = 0; i < warps; ++i) s1 += ex[0][group * warps + i], s2 += ex[1][group * warps + i];
    }
    if (t == 0 && alive && row + (long long)stages * step < p.rows)
      issue(row + (long long)stages * step, s);
    const float c1 = s1 * inv, c2 = s2 * inv;
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
    k ^= 1;
    if (++s == stages) s = 0, ph ^= 1u;
  }
  if (!p.part) return;
  __syncthreads();  // every ring is drained: its memory now takes the groups' sums
  float* sums = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = t + i * nt;
    if (c < p.chunks) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        sums[(size_t)(2 * group) * p.cols + c * VEC + j] = aw[i][j];
        sums[(size_t)(2 * group + 1) * p.cols + c * VEC + j] = ab[i][j];
      }
    }
  }
  __syncthreads();
  float* out = p.part + (size_t)blockIdx.x * 2 * p.cols;
  for (int c = threadIdx.x; c < 2 * p.cols; c += 512) {
    float a = sums[c];
    for (int g = 1; g < groups; ++g) a += sums[(size_t)2 * g * p.cols + c];
    out[c] = a;
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

// Warps per row of the many-rows kernel (8 chunks a thread), 0 when 4 are too few.
template <typename T, int VEC>
cudaError_t fwd_rows(LnFwd p, int sms, cudaStream_t st) {
  const long long warps = ceil_div(p.chunks, 256);
  const int g = warps <= 1 ? 1 : warps <= 2 ? 2 : 4;
  const long long blocks = ceil_div(p.rows, 16 / g);
  const dim3 grid((unsigned)(blocks < sms ? blocks : sms)), block(512);
  const int nch = (int)ceil_div(p.chunks, 32 * g);
  if (g == 4) return launch_train(ln_fwd_rows_kernel<T, VEC, 8, 4>, grid, block, 0, st, p);
  if (g == 2) return launch_train(ln_fwd_rows_kernel<T, VEC, 8, 2>, grid, block, 0, st, p);
  if (nch <= 2) return launch_train(ln_fwd_rows_kernel<T, VEC, 2, 1>, grid, block, 0, st, p);
  if (nch <= 4) return launch_train(ln_fwd_rows_kernel<T, VEC, 4, 1>, grid, block, 0, st, p);
  return launch_train(ln_fwd_rows_kernel<T, VEC, 8, 1>, grid, block, 0, st, p);
}

template <typename T, int VEC>
cudaError_t fwd_launch(LnFwd p, int sms, cudaStream_t st) {
  p.chunks = p.cols / VEC;
  if constexpr (VEC > 1) {
    if (p.rows > 4 * sms && p.chunks <= 1024) return fwd_rows<T, VEC>(p, sms, st);
  }
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

// The ring kernel's groups: threads a row (16 columns each), rows in the ring;
// stages == 0 when a row is too wide for it.
struct Ring {
  int nt, groups, stages;
};
Ring ring_of(int cols, int dtype) {
  Ring r{32, 0, 0};
  while (r.nt < 512 && r.nt * 16 < cols) r.nt *= 2;
  r.groups = 512 / r.nt;
  if (r.nt * 16 < cols) return r;
  const long long pair = 2LL * cols * (long long)type_size(dtype);
  const long long s = kRingBytes / (pair * r.groups);
  r.stages = (int)(s < kRingStages ? s : kRingStages);
  return r;
}

// Blocks of a backward kernel, each leaving one partial row of dweight and of
// dbias: one an SM in the ring kernel, up to four rows a block otherwise, at most
// four blocks an SM (the partial rows stay a small share of the traffic).
int bwd_parts(long long rows, int cols, int dtype, int sms, bool vec) {
  const Ring r = ring_of(cols, dtype);
  const long long most = vec && r.stages >= 2 ? sms : 4LL * sms;
  const long long fair = ceil_div(rows, vec && r.stages >= 2 ? r.groups : 4);
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
cudaError_t bwd_ring(const LnBwd& p, const Ring& r, int parts, const TrainDevice& d,
                     cudaStream_t st) {
  static std::atomic<int> configured[64];
  constexpr int NCH = 16 / VEC;
  // the rings, and at the end the groups' column sums (64 KB at most)
  const size_t rings = (size_t)r.groups * r.stages * 2 * p.cols * sizeof(T);
  const size_t sums = (size_t)r.groups * 2 * p.cols * sizeof(float);
  const size_t smem = rings > sums ? rings : sums;
  if (d.dev < 0 || d.dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[d.dev].load(std::memory_order_acquire)) {
    const cudaError_t e =
        cudaFuncSetAttribute(ln_bwd_ring_kernel<T, VEC, NCH>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (e != cudaSuccess) return e;
    configured[d.dev].store(1, std::memory_order_release);
  }
  return launch_train(ln_bwd_ring_kernel<T, VEC, NCH>, dim3(parts), dim3(512), smem, st, p, r.nt,
                      r.stages, d.status, d.wait_limit_ns);
}

template <typename T, int VEC>
cudaError_t bwd_launch(LnBwd p, int dtype, T* dweight, T* dbias, int parts, const TrainDevice& d,
                       cudaStream_t st) {
  p.chunks = p.cols / VEC;
  cudaError_t e = cudaSuccess;
  const int nt = row_threads(p.chunks, kMaxBwd<VEC>);
  const Ring r = ring_of(p.cols, dtype);
  bool done = false;
  if constexpr (VEC > 1) {
    if (r.stages >= 2) e = bwd_ring<T, VEC>(p, r, parts, d, st), done = true;
  }
  if (done) {
  } else if (nt) {
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

// Partial rows of either kind of kernel: the query does not know the alignment.
size_t bwd_bytes(long long rows, int cols, int dtype, int sms) {
  const int a = bwd_parts(rows, cols, dtype, sms, true), b = bwd_parts(rows, cols, dtype, sms, false);
  return (size_t)(a > b ? a : b) * 2 * cols * sizeof(float);
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
  *bytes = bwd_bytes(rows, cols, dtype, sms);
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
      (!workspace || !vec16(workspace) || workspace_bytes < bwd_bytes(rows, cols, dtype, d.sms)))
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
  const bool v = vec16(dy) && vec16(x) && vec16(weight) && vec16(dx) && vec16_ld(lddy, dtype) &&
                 vec16_ld(ldx, dtype) && vec16_ld(lddx, dtype) && vec16_ld(cols, dtype);
  const int parts = bwd_parts(rows, cols, dtype, d.sms, v);
  if (dtype == B2G_F32) {
    float* dw = static_cast<float*>(dweight);
    float* db = static_cast<float*>(dbias);
    return launch_code(v ? bwd_launch<float, 4>(p, dtype, dw, db, parts, d, st)
                         : bwd_launch<float, 1>(p, dtype, dw, db, parts, d, st));
  }
  Bf16* dw = static_cast<Bf16*>(dweight);
  Bf16* db = static_cast<Bf16*>(dbias);
  return launch_code(v ? bwd_launch<Bf16, 8>(p, dtype, dw, db, parts, d, st)
                       : bwd_launch<Bf16, 1>(p, dtype, dw, db, parts, d, st));
}

}  // extern "C"
