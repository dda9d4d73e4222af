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
// With many rows, both keep the next ones on their way while one is worked on, in rings
// of bulk copies in shared memory; rows that do not fit there twice, or that are wider
// than 8192 columns, take kernels that read them several times.
#include "ring.cuh"

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

// One row per blockDim.x threads (from 8 lanes of a warp up; threadIdx.y picks the row
// of a block that has several), NCH chunks of VEC columns per thread.  The weights are
// fetched with the row, ahead of the two sums, so that their latency is not added to the
// row's; except where many single elements a thread would take the registers of blocks
// that hide it better (8192 x 4095: BF16 89 us so, 74 with the weights fetched at the end).
// Serves few or short rows (one row of 4096: 2.1 us, which is the latency of a launch,
// a read, two block sums and a write) and rows off the 16-byte boundaries, element by
// element (8192 x 4095: 74 us in BF16, 71 in FP32, 1.8 and 3.8 TB/s; the ring of the
// backward pass off the boundaries, tried here, took 87 and 82).
template <typename T, int VEC, int NCH>
__global__ void __launch_bounds__(512) ln_fwd_kernel(const __grid_constant__ LnFwd p) {
  constexpr bool kEarly = VEC > 1 || NCH <= 2;
  __shared__ float red[2][32];
  pdl_launch_dependents();
  const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  const T* w = static_cast<const T*>(p.w);
  const T* b = static_cast<const T*>(p.b);
  pdl_wait();
  const bool live = row < p.rows;  // the others of the warp take part in its sums
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const int t = threadIdx.x, nt = blockDim.x, chunks = live ? p.chunks : 0;
  Pack<T, VEC> raw[NCH], wr[NCH], br[NCH];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = t + i * nt;
    raw[i].zero(), wr[i].zero(), br[i].zero();
    if (c < chunks) raw[i].load(x + c * VEC);
  }
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = t + i * nt;
    if (kEarly && c < chunks) {
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
  const float mean = row_sum(sum, red[0], nt) * inv;
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    float f[VEC];
    raw[i].get(f);
    if (t + i * nt < chunks) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) sq = fmaf(f[j] - mean, f[j] - mean, sq);
    }
  }
  const float rstd = 1.f / sqrtf(row_sum(sq, red[1], nt) * inv + p.eps);
  T* y = static_cast<T*>(p.y) + row * p.ldy;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = t + i * nt;
    if (c < chunks) {
      if (!kEarly) {
        if (w) wr[i].load(w + c * VEC);
        if (b) br[i].load(b + c * VEC);
      }
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
  if (t == 0 && live) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
}

// Rows on 16-byte boundaries: one block an SM, in groups of `nt` threads with a row
// each.  A group's first thread keeps `stages` rows on their way
// into the group's ring in shared memory (bulk copies that arrive on a barrier per
// slot; up to 192 KB an SM), so a row's latency is not waited for; a slot is
// refilled once the group's first sum has been exchanged, when every thread has
// read it.
constexpr int kFwdThreads = 512;  // 32 columns a thread
constexpr int kBwdThreads = 512;  // 16

// Two sums over a group's nt threads at once; `ex` is one of two exchange buffers
// used by turns.
__device__ __forceinline__ F2 group_sum2(F2 v, F2 (&ex)[16], int group, int nt) {
  auto over = [&](F2 x, int o) {
    float a, b;
    f2_split(x, a, b);
    return add2(x, f2(__shfl_xor_sync(0xffffffffu, a, o), __shfl_xor_sync(0xffffffffu, b, o)));
  };
#pragma unroll
  for (int o = 16; o; o >>= 1) v = over(v, o);
  const int warps = nt >> 5, lane = threadIdx.x & 31;
  if (warps == 1) return v;
  if (lane == 0) ex[threadIdx.x >> 5] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(nt) : "memory");
  v = lane < warps ? ex[group * warps + lane] : f2(0.f, 0.f);
#pragma unroll
  for (int o = 8; o; o >>= 1)
    if (o < warps) v = over(v, o);  // lanes 0 .. warps - 1 hold the sum
  float a, b;
  f2_split(v, a, b);
  return f2(__shfl_sync(0xffffffffu, a, 0), __shfl_sync(0xffffffffu, b, 0));
}
// 32 columns a thread (FULL: every thread has all of them).  The weights stand in
// shared memory after the rings: next to rings of this size L1 is too small to keep
// them, and fetching them from L2 for every row took 43 us at 8192 x 4096 BF16, where this
// takes 24 (5.5 TB/s).
template <typename T, int VEC, bool FULL>
__global__ void __launch_bounds__(kFwdThreads, 1)
    ln_fwd_ring_kernel(const __grid_constant__ LnFwd p, const __grid_constant__ Ring g,
                       const __grid_constant__ RingWait wait) {
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ __align__(8) unsigned long long bars[kFwdThreads / 32 * kRingStages];
  __shared__ float red[2][16];
  constexpr int H = VEC / 2, NCH = 32 / VEC;
  pdl_launch_dependents();
  const int group = threadIdx.x / g.nt, t = threadIdx.x - group * g.nt;
  const uint32_t bytes = (uint32_t)(p.cols * (int)sizeof(T));
  const uint32_t bar0 = smem_addr(bars) + 8u * (uint32_t)(group * kRingStages);
  unsigned char* mine = ring + (size_t)group * g.stages * bytes;
  T* ws = reinterpret_cast<T*>(ring + (size_t)g.groups * g.stages * bytes);
  T* bs = ws + p.cols;
  if (t == 0) {
    for (int s = 0; s < g.stages; ++s) mbar_init(bar0 + 8u * s, 1);
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  __syncthreads();
  pdl_wait();
  const float inv = 1.f / (float)p.cols;
  const long long step = (long long)gridDim.x * g.groups;
  const long long row0 = (long long)group * gridDim.x + blockIdx.x;
  auto issue = [&](long long row, int s) {
    if (wait.debug_stop >= 0 && (row - row0) / step >= wait.debug_stop) return;
    mbar_arrive_expect_tx(bar0 + 8u * s, bytes);
    bulk_load(smem_addr(mine + (size_t)s * bytes), static_cast<const T*>(p.x) + row * p.ldx, bytes,
              bar0 + 8u * s);
  };
  if (t == 0) {
    long long row = row0;
    for (int s = 0; s < g.stages && row < p.rows; ++s, row += step) issue(row, s);
  }
  for (int c = threadIdx.x; c < p.cols; c += kFwdThreads) {
    ws[c] = p.w ? static_cast<const T*>(p.w)[c] : from_f32<T>(1.f);
    bs[c] = p.b ? static_cast<const T*>(p.b)[c] : from_f32<T>(0.f);
  }
  __syncthreads();
  RingPos at;
  bool alive = true;  // false once a wait has run out: no more waits, no more copies
  for (long long row = row0; row < p.rows; row += step) {
    if (alive) alive = wait_row(bar0, at, g.stages, row, step, p.rows, t == 0, wait);
    const T* xs = reinterpret_cast<const T*>(mine + (size_t)at.s * bytes);
    F2 x[NCH][H];
    F2 s0 = f2(0.f, 0.f), s1 = f2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = t + i * g.nt;
      if (FULL || c < p.chunks) {
        Pack<T, VEC> k;
        k.load(xs + c * VEC);
        k.get2(x[i]);
#pragma unroll
        for (int j = 0; j < H; j += 2) s0 = add2(s0, x[i][j]), s1 = add2(s1, x[i][j + 1]);
      }
    }
    const float mean = group_sum(f2_sum(add2(s0, s1)), red[0], group, g.nt) * inv;
    if (t == 0 && alive && row + (long long)g.stages * step < p.rows)
      issue(row + (long long)g.stages * step, at.s);
    const F2 minus = f2(-mean, -mean);
    s0 = s1 = f2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      if (FULL || t + i * g.nt < p.chunks) {
#pragma unroll
        for (int j = 0; j < H; j += 2) {
          x[i][j] = add2(x[i][j], minus), x[i][j + 1] = add2(x[i][j + 1], minus);
          s0 = fma2(x[i][j], x[i][j], s0), s1 = fma2(x[i][j + 1], x[i][j + 1], s1);
        }
      }
    }
    const float var = group_sum(f2_sum(add2(s0, s1)), red[1], group, g.nt) * inv;
    const float rstd = 1.f / sqrtf(var + p.eps);
    const F2 r2 = f2(rstd, rstd);
    T* y = static_cast<T*>(p.y) + row * p.ldy;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = t + i * g.nt;
      if (FULL || c < p.chunks) {
        Pack<T, VEC> k;
        F2 wf[H], bf[H];
        k.load(ws + c * VEC);
        k.get2(wf);
        k.load(bs + c * VEC);
        k.get2(bf);
#pragma unroll
        for (int j = 0; j < H; ++j) x[i][j] = fma2(mul2(x[i][j], r2), wf[j], bf[j]);
        k.set2(x[i]);
        k.store(y + c * VEC);
      }
    }
    if (t == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
    at.next(g.stages);
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

// Rows on 16-byte boundaries: the ring above with rows of x and dy together, 16
// columns a thread (FULL: every thread has all of them).  With t = x - mean,
//     dx = rstd g + (-rstd^3 mean(g t)) t - rstd mean(g),
// two operations an element once g and t are there.  At the end the groups' column
// sums are added in shared memory in group order.  8192 x 4096 BF16: 40 us with the
// reduction (5.0 TB/s; the ring alone 36, 5.6 TB/s); 65536 x 256 BF16 29 us, 41 with 32
// columns a thread in half the threads.
template <typename T, int VEC, bool FULL>
__global__ void __launch_bounds__(kBwdThreads, 1)
    ln_bwd_ring_kernel(const __grid_constant__ LnBwd p, const __grid_constant__ Ring g,
                       const __grid_constant__ RingWait wait) {
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ __align__(8) unsigned long long bars[kBwdThreads / 32 * kRingStages];
  __shared__ F2 red[2][16];
  constexpr int H = VEC / 2, NCH = 16 / VEC;
  pdl_launch_dependents();
  const int group = threadIdx.x / g.nt, t = threadIdx.x - group * g.nt;
  const uint32_t bytes = (uint32_t)(p.cols * (int)sizeof(T));
  const uint32_t bar0 = smem_addr(bars) + 8u * (uint32_t)(group * kRingStages);
  unsigned char* mine = ring + (size_t)group * g.stages * 2 * bytes;
  if (t == 0) {
    for (int s = 0; s < g.stages; ++s) mbar_init(bar0 + 8u * s, 1);
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  __syncthreads();
  pdl_wait();
  const float inv = 1.f / (float)p.cols;
  const long long step = (long long)gridDim.x * g.groups;
  const long long row0 = (long long)group * gridDim.x + blockIdx.x;
  auto issue = [&](long long row, int s) {
    if (wait.debug_stop >= 0 && (row - row0) / step >= wait.debug_stop) return;
    const uint32_t bar = bar0 + 8u * s, dst = smem_addr(mine + (size_t)s * 2 * bytes);
    mbar_arrive_expect_tx(bar, 2 * bytes);
    bulk_load(dst, static_cast<const T*>(p.x) + row * p.ldx, bytes, bar);
    bulk_load(dst + bytes, static_cast<const T*>(p.dy) + row * p.lddy, bytes, bar);
  };
  if (t == 0) {
    long long row = row0;
    for (int s = 0; s < g.stages && row < p.rows; ++s, row += step) issue(row, s);
  }
  F2 aw[NCH][H], ab[NCH][H], wf[NCH][H];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = t + i * g.nt;
#pragma unroll
    for (int j = 0; j < H; ++j) aw[i][j] = ab[i][j] = f2(0.f, 0.f), wf[i][j] = f2(1.f, 1.f);
    if (p.w && c < p.chunks) {
      Pack<T, VEC> k;
      k.load(static_cast<const T*>(p.w) + c * VEC);
      k.get2(wf[i]);
    }
  }
  float mean = 0.f, rstd = 0.f;
  if (row0 < p.rows) mean = p.mean[row0], rstd = p.rstd[row0];
  RingPos at;
  int turn = 0;
  bool alive = true;  // false once a wait has run out: no more waits, no more copies
  for (long long row = row0; row < p.rows; row += step) {
    const F2 m2 = f2(-mean, -mean), r2 = f2(rstd, rstd);
    if (row + step < p.rows) mean = p.mean[row + step], rstd = p.rstd[row + step];
    if (alive) alive = wait_row(bar0, at, g.stages, row, step, p.rows, t == 0, wait);
    const T* xs = reinterpret_cast<const T*>(mine + (size_t)at.s * 2 * bytes);
    const T* ds = reinterpret_cast<const T*>(mine + (size_t)at.s * 2 * bytes + bytes);
    F2 x[NCH][H], gr[NCH][H];  // x - mean and g = dy * weight
    F2 s1 = f2(0.f, 0.f), s2 = f2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = t + i * g.nt;
      if (FULL || c < p.chunks) {
        Pack<T, VEC> k;
        F2 d[H];
        k.load(xs + c * VEC);
        k.get2(x[i]);
        k.load(ds + c * VEC);
        k.get2(d);
#pragma unroll
        for (int j = 0; j < H; ++j) {
          x[i][j] = add2(x[i][j], m2);
          gr[i][j] = mul2(d[j], wf[i][j]);
          s1 = add2(s1, gr[i][j]), s2 = fma2(gr[i][j], x[i][j], s2);
          aw[i][j] = fma2(d[j], mul2(x[i][j], r2), aw[i][j]), ab[i][j] = add2(ab[i][j], d[j]);
        }
      }
    }
    const F2 sums2 = group_sum2(f2(f2_sum(s1), f2_sum(s2)), red[turn], group, g.nt);
    if (t == 0 && alive && row + (long long)g.stages * step < p.rows)
      issue(row + (long long)g.stages * step, at.s);
    float sg, sgt, r, unused;
    f2_split(sums2, sg, sgt), f2_split(r2, r, unused);
    const float c1 = -r * (sg * inv), c2 = -r * (r * (r * (sgt * inv)));
    const F2 k1 = f2(c1, c1), k2 = f2(c2, c2);
    T* dx = static_cast<T*>(p.dx) + row * p.lddx;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = t + i * g.nt;
      if (FULL || c < p.chunks) {
#pragma unroll
        for (int j = 0; j < H; ++j) gr[i][j] = fma2(gr[i][j], r2, fma2(x[i][j], k2, k1));
        Pack<T, VEC> k;
        k.set2(gr[i]);
        k.store(dx + c * VEC);
      }
    }
    turn ^= 1;
    at.next(g.stages);
  }
  if (!p.part) return;
  __syncthreads();  // no ring has a copy on its way: its memory now takes the groups' sums
  float* sums = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = t + i * g.nt;
    if (FULL || c < p.chunks) {
#pragma unroll
      for (int j = 0; j < H; ++j) {
        F2* q = reinterpret_cast<F2*>(sums + (size_t)2 * group * p.cols + c * VEC) + j;
        q[0] = aw[i][j];
        q[p.cols / 2] = ab[i][j];
      }
    }
  }
  __syncthreads();
  float* out = p.part + (size_t)blockIdx.x * 2 * p.cols;
  for (int c = threadIdx.x; c < 2 * p.cols; c += kBwdThreads) {
    float a = sums[c];
    for (int i = 1; i < g.groups; ++i) a += sums[(size_t)2 * i * p.cols + c];
    out[c] = a;
  }
}

// The same for rows off the 16-byte boundaries, each thread with the 16 columns
// t + i * nt and the weights in shared memory.  8192 x 4095:
// 91 us in BF16, 87 in FP32 (2.3 and 4.6 TB/s), against 182 and 197 with the rows read
// element by element from global memory; element by element it is still issue that
// bounds it, on the boundaries the same size takes 41 in BF16.
template <typename T>
__global__ void __launch_bounds__(kBwdThreads, 1)
    ln_bwd_any_kernel(const __grid_constant__ LnBwd p, const __grid_constant__ Ring g,
                      const __grid_constant__ RingWait wait) {
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ __align__(8) unsigned long long bars[kBwdThreads / 32 * kRingStages];
  __shared__ F2 red[2][16];
  constexpr int N = 16;
  pdl_launch_dependents();
  const int group = threadIdx.x / g.nt, t = threadIdx.x - group * g.nt;
  const size_t slot = any_slot(p.cols, sizeof(T));
  const uint32_t bar0 = smem_addr(bars) + 8u * (uint32_t)(group * kRingStages);
  unsigned char* mine = ring + (size_t)group * g.stages * 2 * slot;
  if (t == 0) {
    for (int s = 0; s < g.stages; ++s) mbar_init(bar0 + 8u * s, 1);
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  __syncthreads();
  pdl_wait();
  const float inv = 1.f / (float)p.cols;
  const long long step = (long long)gridDim.x * g.groups;
  const long long row0 = (long long)group * gridDim.x + blockIdx.x;
  auto x_row = [&](long long row) {
    return AnyRow<T>(static_cast<const T*>(p.x) + row * p.ldx, p.cols);
  };
  auto d_row = [&](long long row) {
    return AnyRow<T>(static_cast<const T*>(p.dy) + row * p.lddy, p.cols);
  };
  auto issue = [&](long long row, int s) {
    if (wait.debug_stop >= 0 && (row - row0) / step >= wait.debug_stop) return;
    const uint32_t bar = bar0 + 8u * s, dst = smem_addr(mine + (size_t)s * 2 * slot);
    const AnyRow<T> x = x_row(row), d = d_row(row);
    mbar_arrive_expect_tx(bar, x.bytes() + d.bytes());
    x.copy(dst, bar);
    d.copy(dst + (uint32_t)slot, bar);
  };
  if (t == 0) {
    long long row = row0;
    for (int s = 0; s < g.stages && row < p.rows; ++s, row += step) issue(row, s);
  }
  T* ws = reinterpret_cast<T*>(ring + (size_t)g.groups * g.stages * 2 * slot);
  for (int c = threadIdx.x; c < p.cols; c += kBwdThreads)
    ws[c] = p.w ? static_cast<const T*>(p.w)[c] : from_f32<T>(1.f);
  __syncthreads();
  float aw[N], ab[N];
#pragma unroll
  for (int i = 0; i < N; ++i) aw[i] = ab[i] = 0.f;
  float mean = 0.f, rstd = 0.f;
  if (row0 < p.rows) mean = p.mean[row0], rstd = p.rstd[row0];
  RingPos at;
  int turn = 0;
  bool alive = true;  // false once a wait has run out: no more waits, no more copies
  for (long long row = row0; row < p.rows; row += step) {
    const float m = mean, r = rstd;
    if (row + step < p.rows) mean = p.mean[row + step], rstd = p.rstd[row + step];
    if (alive) alive = wait_row(bar0, at, g.stages, row, step, p.rows, t == 0, wait);
    const unsigned char* here = mine + (size_t)at.s * 2 * slot;
    const AnyRow<T> xr = x_row(row), dr = d_row(row);
    const typename AnyRow<T>::Ends xe = xr.ends(t, g.nt, p.cols), de = dr.ends(t, g.nt, p.cols);
    float x[N], gr[N];  // x - mean and g = dy * weight
    float s1 = 0.f, s2 = 0.f;
    // The columns are computed anew in each of the two loops: kept for all rows, with
    // what depends on them, they would spill.
    int c0 = t, nt = g.nt;
    asm volatile("" : "+r"(c0), "+r"(nt));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = c0 + i * nt;
      x[i] = gr[i] = 0.f;
      if (c < p.cols) {
        x[i] = xe.pick(i, xr.at(here, c)) - m;
        const float d = de.pick(i, dr.at(here + slot, c));
        gr[i] = d * to_f32(ws[c]);
        s1 += gr[i], s2 = fmaf(gr[i], x[i], s2);
        aw[i] = fmaf(d, x[i] * r, aw[i]), ab[i] += d;
      }
      if (i % 4 == 3) asm volatile("" : "+r"(c0), "+r"(nt)::"memory");
    }
    const F2 sums2 = group_sum2(f2(s1, s2), red[turn], group, g.nt);
    if (t == 0 && alive && row + (long long)g.stages * step < p.rows)
      issue(row + (long long)g.stages * step, at.s);
    float sg, sgt;
    f2_split(sums2, sg, sgt);
    const float k1 = -r * (sg * inv), k2 = -r * (r * (r * (sgt * inv)));
    T* dx = static_cast<T*>(p.dx) + row * p.lddx;
    asm volatile("" : "+r"(c0), "+r"(nt));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = c0 + i * nt;
      if (c < p.cols) dx[c] = from_f32<T>(fmaf(gr[i], r, fmaf(x[i], k2, k1)));
    }
    turn ^= 1;
    at.next(g.stages);
  }
  if (!p.part) return;
  __syncthreads();  // no ring has a copy on its way: its memory now takes the groups' sums
  float* sums = reinterpret_cast<float*>(ring) + (size_t)2 * group * p.cols;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = t + i * g.nt;
    if (c < p.cols) sums[c] = aw[i], sums[p.cols + c] = ab[i];
  }
  __syncthreads();
  const float* all = reinterpret_cast<const float*>(ring);
  float* out = p.part + (size_t)blockIdx.x * 2 * p.cols;
  for (int c = threadIdx.x; c < 2 * p.cols; c += kBwdThreads) {
    float a = all[c];
    for (int i = 1; i < g.groups; ++i) a += all[(size_t)2 * i * p.cols + c];
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

// dweight (blockIdx.y == 0) and dbias (1): warp y adds the partial rows y, y + 16,
// ... in order, then the warps' sums are added in warp order.
template <typename T>
__global__ void __launch_bounds__(512) ln_bwd_reduce_kernel(const float* part, int parts, int cols,
                                                            T* dweight, T* dbias) {
  __shared__ float acc[16][32];
  pdl_launch_dependents();
  pdl_wait();
  T* out = blockIdx.y ? dbias : dweight;
  if (!out) return;
  const int c = blockIdx.x * 32 + threadIdx.x;
  float a = 0.f;
  if (c < cols) {
    const float* p0 = part + (size_t)blockIdx.y * cols + c;
#pragma unroll 10
    for (int i = threadIdx.y; i < parts; i += 16) a += p0[(size_t)i * 2 * cols];
  }
  acc[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  if (threadIdx.y == 0 && c < cols) {
#pragma unroll
    for (int i = 1; i < 16; ++i) a += acc[i][threadIdx.x];
    out[c] = from_f32<T>(a);
  }
}

// ----------------------------------------------------------------- host side

// Chunks a thread may hold (powers of two) without spilling at 512 threads.
template <int VEC>
constexpr int kMaxFwd = VEC == 1 ? 16 : 4;
template <typename T, int VEC, int NCH = 1>
cudaError_t fwd_kernel(int nch, dim3 grid, dim3 block, cudaStream_t st, const LnFwd& p) {
  if constexpr (NCH < kMaxFwd<VEC>) {
    if (nch > NCH) return fwd_kernel<T, VEC, 2 * NCH>(nch, grid, block, st, p);
  }
  return launch_train(ln_fwd_kernel<T, VEC, NCH>, grid, block, 0, st, p);
}

Ring fwd_ring_of(int cols, int dtype) {
  const size_t es = type_size(dtype);
  return ring_of(kFwdThreads, 32, cols, cols * es, 2 * es * cols);
}
// vec: rows on 16-byte boundaries.
Ring bwd_ring_of(int cols, int dtype, bool vec) {
  const size_t es = type_size(dtype);
  return vec ? ring_of(kBwdThreads, 16, cols, 2 * cols * es, 0)
             : ring_of(kBwdThreads, 16, cols, 2 * any_slot(cols, es), es * cols);
}

template <typename T, int VEC, bool FULL>
cudaError_t fwd_ring(const LnFwd& p, const Ring& r, const TrainDevice& d, cudaStream_t st) {
  static std::atomic<int> done[64];
  const cudaError_t e =
      allow_ring(reinterpret_cast<const void*>(&ln_fwd_ring_kernel<T, VEC, FULL>), done, d.dev);
  if (e != cudaSuccess) return e;
  const long long blocks = ceil_div(p.rows, r.groups);
  return launch_train(ln_fwd_ring_kernel<T, VEC, FULL>,
                      dim3((unsigned)(blocks < d.sms ? blocks : d.sms)), dim3(kFwdThreads),
                      ((size_t)r.groups * r.stages + 2) * p.cols * sizeof(T), st, p, r,
                      RingWait{d.status, d.wait_limit_ns, d.debug_stop});
}

template <typename T, int VEC>
cudaError_t fwd_launch(LnFwd p, int dtype, const TrainDevice& d, cudaStream_t st) {
  const int sms = d.sms;
  p.chunks = p.cols / VEC;
  if constexpr (VEC > 1) {
    const Ring r = fwd_ring_of(p.cols, dtype);
    // Few elements or short rows go faster a row (or four) a block, with more blocks an SM
    // and no second row to wait for.  BF16, us, the ring and the other: 608 x 4096 3.7 and
    // 3.7, 912 x 4096 4.7 and 5.3, 2432 x 4096 8.5 and 10.1; 2432 x 1024 3.6 and 3.4, 4864 x
    // 1024 5.1 and 5.2; 4864 x 512 4.0 and 3.3, 65536 x 256 24.0 and 18.3.
    if (p.cols >= 1024 && p.rows * p.cols > 16384LL * sms && r.stages >= 2)
      return p.cols == r.nt * 32 ? fwd_ring<T, VEC, true>(p, r, d, st)
                                 : fwd_ring<T, VEC, false>(p, r, d, st);
  }
  // Few rows: one chunk a thread, for the shortest path; many: several, for the
  // fewest barriers per byte (single elements: 8 rather than 16 where that is enough, 8.7 us
  // and 10.8 at 4000 x 777 BF16).
  constexpr int least = VEC > 1 ? 8 : 32;  // lanes a row: whole 128-byte lines
  int nt = p.rows <= 2 * sms ? row_threads(p.chunks, 1, least) : 0;
  if (!nt && VEC == 1) nt = row_threads(p.chunks, kMaxFwd<VEC> / 2, least);
  if (!nt) nt = row_threads(p.chunks, kMaxFwd<VEC>, least);
  if (!nt)
    return launch_train(ln_fwd_wide_kernel<T>, dim3((unsigned)p.rows), dim3(1024), 0, st, p);
  const int ry = nt <= 32 ? 128 / nt : 1;
  const dim3 grid((unsigned)ceil_div(p.rows, ry)), block(nt, ry);
  return fwd_kernel<T, VEC>((int)ceil_div(p.chunks, nt), grid, block, st, p);
}

// Blocks of a backward kernel, each leaving one partial row of dweight and of
// dbias: one an SM in the ring kernels, row slices of the wide one otherwise.
int bwd_parts(long long rows, int cols, int dtype, int sms, bool vec) {
  const Ring r = bwd_ring_of(cols, dtype, vec);
  const long long most = r.stages >= 2 ? sms : 4LL * sms;
  const long long fair = ceil_div(rows, r.stages >= 2 ? r.groups : 4);
  return (int)(fair < most ? fair : most);
}

template <typename T, int VEC, bool FULL>
cudaError_t bwd_ring(const LnBwd& p, const Ring& r, int parts, const TrainDevice& d,
                     cudaStream_t st) {
  static std::atomic<int> done[64];
  const cudaError_t e =
      allow_ring(reinterpret_cast<const void*>(&ln_bwd_ring_kernel<T, VEC, FULL>), done, d.dev);
  if (e != cudaSuccess) return e;
  // the rings, and at the end the groups' column sums (64 KB at most)
  const size_t rings = (size_t)r.groups * r.stages * 2 * p.cols * sizeof(T);
  const size_t sums = (size_t)r.groups * 2 * p.cols * sizeof(float);
  return launch_train(ln_bwd_ring_kernel<T, VEC, FULL>, dim3(parts), dim3(kBwdThreads),
                      rings > sums ? rings : sums, st, p, r, RingWait{d.status, d.wait_limit_ns, d.debug_stop});
}

template <typename T>
cudaError_t bwd_any(const LnBwd& p, const Ring& r, int parts, const TrainDevice& d,
                    cudaStream_t st) {
  static std::atomic<int> done[64];
  const cudaError_t e =
      allow_ring(reinterpret_cast<const void*>(&ln_bwd_any_kernel<T>), done, d.dev);
  if (e != cudaSuccess) return e;
  const size_t rings =
      (size_t)r.groups * r.stages * 2 * any_slot(p.cols, sizeof(T)) + p.cols * sizeof(T);
  const size_t sums = (size_t)r.groups * 2 * p.cols * sizeof(float);
  return launch_train(ln_bwd_any_kernel<T>, dim3(parts), dim3(kBwdThreads),
                      rings > sums ? rings : sums, st, p, r, RingWait{d.status, d.wait_limit_ns, d.debug_stop});
}

template <typename T, int VEC>
cudaError_t bwd_launch(LnBwd p, int dtype, T* dweight, T* dbias, int parts, const TrainDevice& d,
                       cudaStream_t st) {
  p.chunks = p.cols / VEC;
  cudaError_t e = cudaSuccess;
  const Ring r = bwd_ring_of(p.cols, dtype, VEC > 1);
  if (r.stages >= 2) {
    if constexpr (VEC > 1)
      e = r.nt * 16 == p.cols ? bwd_ring<T, VEC, true>(p, r, parts, d, st)
                              : bwd_ring<T, VEC, false>(p, r, parts, d, st);
    else
      e = bwd_any<T>(p, r, parts, d, st);
  } else {
    if (p.part)
      e = launch_train(ln_bwd_cols_kernel<T>, dim3((unsigned)ceil_div(p.cols, 256), parts),
                       dim3(256), 0, st, p);
    if (e == cudaSuccess)
      e = launch_train(ln_bwd_wide_kernel<T>, dim3((unsigned)p.rows), dim3(1024), 0, st, p);
  }
  if (e == cudaSuccess && p.part)
    e = launch_train(ln_bwd_reduce_kernel<T>, dim3((unsigned)ceil_div(p.cols, 32), 2),
                     dim3(32, 16), 0, st, (const float*)p.part, parts, p.cols, dweight, dbias);
  return e;
}

int check_rows(int dtype, long long rows, int cols) {
  if (!type_ok(dtype)) return B2G_ERR_INVALID_TYPE;
  if (rows < 0 || cols < 0 || rows > 0x7fffffffLL || cols > kMaxLength) return B2G_ERR_INVALID_DIM;
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
    return launch_code(v ? fwd_launch<float, 4>(p, dtype, d, st) : fwd_launch<float, 1>(p, dtype, d, st));
  return launch_code(v ? fwd_launch<Bf16, 8>(p, dtype, d, st) : fwd_launch<Bf16, 1>(p, dtype, d, st));
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
