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
// kernel to add in block order (no atomics: the same bits every run).  With many rows the
// next ones are on their way meanwhile, in rings of bulk copies in shared memory.
#include <type_traits>

#include "eightbit.cuh"
#include "ring.cuh"

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
    for (int j = 0; j < VEC; ++j) f[j] = f[j] * (w ? wf[j] : 1.f) * rstd;  // BF16: one rounding
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
    const float v = f[0] * (w && in ? to_f32(w[c]) : 1.f) * rstd;
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
  float* part;  // [grid][cols]: partial dweight
  void* dw;     // NULL: it is not wanted.  One block writes it, several their parts
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

// The end of a block: its groups' sums of dy xhat (sums: [groups][cols] in shared memory),
// added in group order.
template <typename T>
__device__ __forceinline__ void leave_sums(const RmsBwd& p, const float* sums, int groups) {
  for (int c = threadIdx.x; c < p.cols; c += kBwdThreads) {
    float a = sums[c];
    for (int i = 1; i < groups; ++i) a += sums[(size_t)i * p.cols + c];
    if (gridDim.x == 1)
      static_cast<T*>(p.dw)[c] = from_f32<T>(a);
    else
      p.part[(size_t)blockIdx.x * p.cols + c] = a;
  }
}

// Few or short rows, on 16-byte boundaries: groups of nt threads (from 4 lanes of a warp
// up) with a row each, 16 columns a thread, all of whose loads are on their way together.
template <typename T, int VEC, bool Q8>
__global__ void __launch_bounds__(kBwdThreads, 1)
    rms_bwd_kernel(const __grid_constant__ RmsBwd p, int nt, int groups) {
  extern __shared__ __align__(16) float sums[];  // [groups][cols], at the end
  __shared__ float red[2][16];
  constexpr int NCH = 16 / VEC;
  pdl_launch_dependents();
  pdl_wait();
  const int group = threadIdx.x / nt, t = threadIdx.x - group * nt;
  const float inv = 1.f / (float)p.cols;
  const T* w = static_cast<const T*>(p.w);
  float aw[NCH][VEC];
  Pack<T, VEC> wr[NCH];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = t + i * nt;
#pragma unroll
    for (int j = 0; j < VEC; ++j) aw[i][j] = 0.f;
    wr[i].zero();
    if (w && c < p.chunks) wr[i].load(w + c * VEC);
  }
  int turn = 0;
  // every group makes as many rounds: the lanes of a warp take part in one another's sums
  for (long long row0 = blockIdx.x; row0 < p.rows; row0 += (long long)gridDim.x * groups) {
    const long long row = row0 + (long long)group * gridDim.x;
    const int chunks = row < p.rows ? p.chunks : 0;
    const float rstd = chunks ? p.rstd[row] : 0.f;
    Pack<T, VEC> dy[NCH], x[NCH], dt[NCH];
    Codes<VEC> q[NCH];
    uint32_t byte[NCH];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = t + i * nt;
      dy[i].zero(), x[i].zero(), dt[i].zero(), q[i].zero(), byte[i] = 127;
      if (c < chunks) {
        dy[i].load(static_cast<const T*>(p.dy) + row * p.lddy + (long long)c * VEC);
        if constexpr (Q8) {
          q[i].load(p.k8.q + row * p.k8.ldq + (long long)c * VEC);
          byte[i] = p.k8.s[row * p.k8.lds + c / (kScaleBlock / VEC)];
        } else {
          x[i].load(static_cast<const T*>(p.x) + row * p.ldx + (long long)c * VEC);
        }
        if (p.dtotal) dt[i].load(static_cast<const T*>(p.dtotal) + row * p.lddt + (long long)c * VEC);
      }
    }
    float xh[NCH][VEC], g[NCH][VEC], along = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      float wf[VEC];
      float scale = rstd;
      if constexpr (Q8) {
        q[i].get(xh[i]);
        const float s = scale_value(byte[i]);
#pragma unroll
        for (int j = 0; j < VEC; ++j) xh[i][j] *= s;
      } else {
        x[i].get(xh[i]);
      }
      dy[i].get(g[i]), wr[i].get(wf);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        xh[i][j] *= scale;
        aw[i][j] = fmaf(g[i][j], xh[i][j], aw[i][j]);
        if (w) g[i][j] *= wf[j];
        along = fmaf(g[i][j], xh[i][j], along);
      }
    }
    const float mean = (nt < 32 ? row_sum(along, nullptr, nt) : group_sum(along, red[turn], group, nt)) * inv;
    turn ^= 1;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = t + i * nt;
      float d[VEC];
      dt[i].get(d);
#pragma unroll
      for (int j = 0; j < VEC; ++j) d[j] = fmaf(rstd, fmaf(-xh[i][j], mean, g[i][j]), d[j]);
      if (c < chunks) {
        Pack<T, VEC> k;
        k.set(d);
        k.store(static_cast<T*>(p.dx) + row * p.lddx + (long long)c * VEC);
      }
    }
  }
  if (!p.dw) return;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = t + i * nt;
    if (c < p.chunks) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) sums[(size_t)group * p.cols + c * VEC + j] = aw[i][j];
    }
  }
  __syncthreads();
  leave_sums<T>(p, sums, groups);
}

// Bytes of a slot's part for one row of the kept rows.
template <typename T, bool Q8>
__host__ __device__ constexpr int kept_bytes(int cols) {
  return cols * (Q8 ? 1 : (int)sizeof(T));
}

// Many rows on 16-byte boundaries: a ring (ring.cuh) of the rows of dy, of the kept rows and
// of dtotal together, 16 columns a thread (FULL: every thread has all of them); the scales
// of 8-bit rows are fetched a row ahead.
template <typename T, int VEC, bool FULL, bool Q8>
__global__ void __launch_bounds__(kBwdThreads, 1)
    rms_bwd_ring_kernel(const __grid_constant__ RmsBwd p, const __grid_constant__ Ring g,
                        const __grid_constant__ RingWait wait) {
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ __align__(8) unsigned long long bars[kBwdThreads / 32 * kRingStages];
  __shared__ float red[2][16];
  constexpr int H = VEC / 2, NCH = 16 / VEC;
  pdl_launch_dependents();
  const int group = threadIdx.x / g.nt, t = threadIdx.x - group * g.nt;
  const uint32_t bytes = (uint32_t)(p.cols * (int)sizeof(T)), kept = (uint32_t)kept_bytes<T, Q8>(p.cols);
  const uint32_t slot = kept + bytes * (p.dtotal ? 2 : 1);
  const uint32_t bar0 = smem_addr(bars) + 8u * (uint32_t)(group * kRingStages);
  unsigned char* mine = ring + (size_t)group * g.stages * slot;
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
    const uint32_t bar = bar0 + 8u * s, dst = smem_addr(mine + (size_t)s * slot);
    mbar_arrive_expect_tx(bar, slot);
    bulk_load(dst, static_cast<const T*>(p.dy) + row * p.lddy, bytes, bar);
    if constexpr (Q8)
      bulk_load(dst + bytes, p.k8.q + row * p.k8.ldq, kept, bar);
    else
      bulk_load(dst + bytes, static_cast<const T*>(p.x) + row * p.ldx, kept, bar);
    if (p.dtotal)
      bulk_load(dst + bytes + kept, static_cast<const T*>(p.dtotal) + row * p.lddt, bytes, bar);
  };
  if (t == 0) {
    long long row = row0;
    for (int s = 0; s < g.stages && row < p.rows; ++s, row += step) issue(row, s);
  }
  F2 aw[NCH][H], wf[NCH][H];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = t + i * g.nt;
#pragma unroll
    for (int j = 0; j < H; ++j) aw[i][j] = f2(0.f, 0.f), wf[i][j] = f2(1.f, 1.f);
    if (p.w && c < p.chunks) {
      Pack<T, VEC> k;
      k.load(static_cast<const T*>(p.w) + c * VEC);
      k.get2(wf[i]);
    }
  }
  float rstd = 0.f;
  uint32_t byte[NCH];
  auto ahead = [&](long long row) {  // what is fetched past the ring
    rstd = p.rstd[row];
    if constexpr (Q8) {
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        const int c = t + i * g.nt;
        byte[i] = FULL || c < p.chunks ? p.k8.s[row * p.k8.lds + c / (kScaleBlock / VEC)] : 127;
      }
    }
  };
  if (row0 < p.rows) ahead(row0);
  RingPos at;
  int turn = 0;
  bool alive = true;  // false once a wait has run out: no more waits, no more copies
  for (long long row = row0; row < p.rows; row += step) {
    const float r = rstd;
    const F2 r2 = f2(r, r);
    F2 scale[NCH];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      if constexpr (Q8) {
        const float s = scale_value(byte[i]);
        scale[i] = f2(s, s);
      }
    }
    if (row + step < p.rows) ahead(row + step);
    if (alive) alive = wait_row(bar0, at, g.stages, row, step, p.rows, t == 0, wait);
    const unsigned char* here = mine + (size_t)at.s * slot;
    F2 xh[NCH][H], gr[NCH][H];  // xhat, and g = dy weight
    Pack<T, VEC> past[NCH];
    F2 s0 = f2(0.f, 0.f), s1 = f2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = t + i * g.nt;
      past[i].zero();
      if (FULL || c < p.chunks) {
        Pack<T, VEC> k;
        F2 d[H];
        k.load(reinterpret_cast<const T*>(here) + c * VEC);
        k.get2(d);
        if constexpr (Q8) {
          Codes<VEC> q;
          float f[VEC];
          q.load(here + bytes + c * VEC);
          q.get(f);
#pragma unroll
          for (int j = 0; j < H; ++j) xh[i][j] = mul2(f2(f[2 * j], f[2 * j + 1]), scale[i]);
        } else {
          k.load(reinterpret_cast<const T*>(here + bytes) + c * VEC);
          k.get2(xh[i]);
        }
        if (p.dtotal) past[i].load(reinterpret_cast<const T*>(here + bytes + kept) + c * VEC);
#pragma unroll
        for (int j = 0; j < H; ++j) {
          xh[i][j] = mul2(xh[i][j], r2);
          gr[i][j] = mul2(d[j], wf[i][j]);
          aw[i][j] = fma2(d[j], xh[i][j], aw[i][j]);
          if (j & 1)
            s1 = fma2(gr[i][j], xh[i][j], s1);
          else
            s0 = fma2(gr[i][j], xh[i][j], s0);
        }
      }
    }
    const float mean = group_sum(f2_sum(add2(s0, s1)), red[turn], group, g.nt) * inv;
    if (t == 0 && alive && row + (long long)g.stages * step < p.rows)
      issue(row + (long long)g.stages * step, at.s);
    const F2 minus = f2(-mean, -mean);
    T* dx = static_cast<T*>(p.dx) + row * p.lddx;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = t + i * g.nt;
      if (FULL || c < p.chunks) {
        F2 d[H];
        past[i].get2(d);
#pragma unroll
        for (int j = 0; j < H; ++j) d[j] = fma2(r2, fma2(xh[i][j], minus, gr[i][j]), d[j]);
        Pack<T, VEC> k;
        k.set2(d);
        k.store(dx + c * VEC);
      }
    }
    turn ^= 1;
    at.next(g.stages);
  }
  if (!p.dw) return;
  __syncthreads();  // no ring has a copy on its way: its memory now takes the groups' sums
  float* sums = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = t + i * g.nt;
    if (FULL || c < p.chunks) {
#pragma unroll
      for (int j = 0; j < H; ++j)
        reinterpret_cast<F2*>(sums + (size_t)group * p.cols + c * VEC)[j] = aw[i][j];
    }
  }
  __syncthreads();
  leave_sums<T>(p, sums, g.groups);
}

// The same for rows off the 16-byte boundaries, each thread with the 16 columns t + i * nt
// and the weights in shared memory.  A block of 32 columns is a warp's; its scales are
// fetched a row ahead, lane i that of column t + i * nt.
template <typename T, bool Q8>
__global__ void __launch_bounds__(kBwdThreads, 1)
    rms_bwd_any_kernel(const __grid_constant__ RmsBwd p, const __grid_constant__ Ring g,
                       const __grid_constant__ RingWait wait) {
  using K = std::conditional_t<Q8, E4m3, T>;
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ __align__(8) unsigned long long bars[kBwdThreads / 32 * kRingStages];
  __shared__ float red[2][16];
  constexpr int N = 16;
  pdl_launch_dependents();
  const int group = threadIdx.x / g.nt, t = threadIdx.x - group * g.nt, lane = threadIdx.x & 31;
  const uint32_t dslot = (uint32_t)any_slot(p.cols, sizeof(T)), kslot = (uint32_t)any_slot(p.cols, sizeof(K));
  const uint32_t slot = kslot + dslot * (p.dtotal ? 2 : 1);
  const uint32_t bar0 = smem_addr(bars) + 8u * (uint32_t)(group * kRingStages);
  unsigned char* mine = ring + (size_t)group * g.stages * slot;
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
  auto d_row = [&](long long row) {
    return AnyRow<T>(static_cast<const T*>(p.dy) + row * p.lddy, p.cols);
  };
  auto k_row = [&](long long row) {
    if constexpr (Q8)
      return AnyRow<K>(reinterpret_cast<const E4m3*>(p.k8.q) + row * p.k8.ldq, p.cols);
    else
      return AnyRow<K>(static_cast<const T*>(p.x) + row * p.ldx, p.cols);
  };
  auto p_row = [&](long long row) {
    return AnyRow<T>(static_cast<const T*>(p.dtotal) + row * p.lddt, p.cols);
  };
  auto issue = [&](long long row, int s) {
    if (wait.debug_stop >= 0 && (row - row0) / step >= wait.debug_stop) return;
    const uint32_t bar = bar0 + 8u * s, dst = smem_addr(mine + (size_t)s * slot);
    const AnyRow<T> d = d_row(row);
    const AnyRow<K> k = k_row(row);
    uint32_t bytes = d.bytes() + k.bytes();
    if (p.dtotal) bytes += p_row(row).bytes();
    mbar_arrive_expect_tx(bar, bytes);
    d.copy(dst, bar);
    k.copy(dst + dslot, bar);
    if (p.dtotal) p_row(row).copy(dst + dslot + kslot, bar);
  };
  if (t == 0) {
    long long row = row0;
    for (int s = 0; s < g.stages && row < p.rows; ++s, row += step) issue(row, s);
  }
  T* ws = reinterpret_cast<T*>(ring + (size_t)g.groups * g.stages * slot);
  for (int c = threadIdx.x; c < p.cols; c += kBwdThreads)
    ws[c] = p.w ? static_cast<const T*>(p.w)[c] : from_f32<T>(1.f);
  __syncthreads();
  float aw[N];
#pragma unroll
  for (int i = 0; i < N; ++i) aw[i] = 0.f;
  float rstd = 0.f, next_scale = 1.f;
  auto ahead = [&](long long row) {
    rstd = p.rstd[row];
    if constexpr (Q8) {
      const int c = t - lane + lane * g.nt;
      next_scale = lane < N && c < p.cols ? scale_value(p.k8.s[row * p.k8.lds + c / kScaleBlock]) : 1.f;
    }
  };
  if (row0 < p.rows) ahead(row0);
  RingPos at;
  int turn = 0;
  bool alive = true;  // false once a wait has run out: no more waits, no more copies
  for (long long row = row0; row < p.rows; row += step) {
    const float r = rstd, scale = next_scale;
    if (row + step < p.rows) ahead(row + step);
    if (alive) alive = wait_row(bar0, at, g.stages, row, step, p.rows, t == 0, wait);
    const unsigned char* here = mine + (size_t)at.s * slot;
    float xh[N], gr[N];
    float along = 0.f;
    // The columns are computed anew in each loop: kept for all rows, with what depends on
    // them, they would spill.
    int c0 = t, nt = g.nt;
    asm volatile("" : "+r"(c0), "+r"(nt));
    {
      const AnyRow<T> dr = d_row(row);
      const AnyRow<K> kr = k_row(row);
      const typename AnyRow<T>::Ends de = dr.ends(t, g.nt, p.cols);
      const typename AnyRow<K>::Ends ke = kr.ends(t, g.nt, p.cols);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = c0 + i * nt;
        xh[i] = gr[i] = 0.f;
        float s = r;
        if constexpr (Q8) s = __shfl_sync(0xffffffffu, scale, i);
        if (c < p.cols) {
          const float k = ke.pick(i, kr.at(here + dslot, c));
          xh[i] = Q8 ? k * s * r : k * r;
          const float d = de.pick(i, dr.at(here, c));
          gr[i] = d * to_f32(ws[c]);
          along = fmaf(gr[i], xh[i], along);
          aw[i] = fmaf(d, xh[i], aw[i]);
        }
        if (i % 4 == 3) asm volatile("" : "+r"(c0), "+r"(nt)::"memory");
      }
    }
    const float mean = group_sum(along, red[turn], group, g.nt) * inv;
    T* dx = static_cast<T*>(p.dx) + row * p.lddx;
    asm volatile("" : "+r"(c0), "+r"(nt));
    if (p.dtotal) {
      const AnyRow<T> pr = p_row(row);
      const typename AnyRow<T>::Ends pe = pr.ends(t, g.nt, p.cols);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = c0 + i * nt;
        if (c < p.cols)
          dx[c] = from_f32<T>(fmaf(r, fmaf(-xh[i], mean, gr[i]), pe.pick(i, pr.at(here + dslot + kslot, c))));
        if (i % 4 == 3) asm volatile("" : "+r"(c0), "+r"(nt)::"memory");
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = c0 + i * nt;
        if (c < p.cols) dx[c] = from_f32<T>(r * fmaf(-xh[i], mean, gr[i]));
      }
    }
    // the slot has been read by all of the group
    if (g.nt > 32)
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(g.nt) : "memory");
    else
      __syncwarp();
    if (t == 0 && alive && row + (long long)g.stages * step < p.rows)
      issue(row + (long long)g.stages * step, at.s);
    turn ^= 1;
    at.next(g.stages);
  }
  if (!p.dw) return;
  __syncthreads();  // no ring has a copy on its way: its memory now takes the groups' sums
  float* sums = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = t + i * g.nt;
    if (c < p.cols) sums[(size_t)group * p.cols + c] = aw[i];
  }
  __syncthreads();
  leave_sums<T>(p, sums, g.groups);
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

// How the backward pass runs.
enum BwdKind { kDirect, kRing, kAny, kWide };
struct BwdPlan {
  BwdKind kind;
  Ring r;     // stages only where there is a ring
  int parts;  // blocks, each leaving one partial row of dweight
};

// vec: rows on 16-byte boundaries; past: a dtotal; q8: 8-bit rows.
BwdPlan bwd_plan(long long rows, int cols, int dtype, int sms, bool vec, bool past, bool q8) {
  const size_t es = type_size(dtype), ks = q8 ? 1 : es;
  BwdPlan b{kWide, {}, 0};
  if (vec) {
    b.r = ring_of(kBwdThreads, 16, cols, (size_t)cols * (ks + es * (past ? 2 : 1)), 0);
    if (b.r.nt * 16 >= cols) {
      if (rows <= (long long)b.r.groups * sms || cols <= 512 || b.r.stages < 2) {
        b.kind = kDirect;
        b.r.nt = 4;
        while (b.r.nt * 16 < cols) b.r.nt *= 2;
        b.r.groups = kBwdThreads / b.r.nt;
      } else {
        b.kind = kRing;
      }
    }
  } else {
    b.r = ring_of(kBwdThreads, 16, cols, any_slot(cols, ks) + any_slot(cols, es) * (past ? 2 : 1), es * cols);
    if (b.r.nt * 16 >= cols && b.r.stages >= 2) b.kind = kAny;
  }
  const long long most = b.kind != kWide ? sms : 4LL * sms, each = b.kind != kWide ? b.r.groups : 4;
  const long long fair = ceil_div(rows, each);
  b.parts = (int)(fair < most ? fair : most);
  return b;
}

template <typename T, bool Q8>
size_t ring_bytes(const RmsBwd& p, const BwdPlan& b) {
  const size_t d = p.dtotal ? 2 : 1;
  const size_t slot = b.kind == kRing
                          ? (size_t)p.cols * sizeof(T) * d + kept_bytes<T, Q8>(p.cols)
                          : any_slot(p.cols, sizeof(T)) * d + any_slot(p.cols, Q8 ? 1 : sizeof(T));
  const size_t rings = b.r.groups * b.r.stages * slot + (b.kind == kAny ? p.cols * sizeof(T) : 0);
  const size_t sums = (size_t)b.r.groups * p.cols * sizeof(float);
  return rings > sums ? rings : sums;
}

template <typename T, int VEC, bool FULL, bool Q8>
cudaError_t bwd_ring(const RmsBwd& p, const BwdPlan& b, const TrainDevice& d, cudaStream_t st) {
  static std::atomic<int> done[64];
  const cudaError_t e = allow_ring(
      reinterpret_cast<const void*>(&rms_bwd_ring_kernel<T, VEC, FULL, Q8>), done, d.dev);
  if (e != cudaSuccess) return e;
  return launch_train(rms_bwd_ring_kernel<T, VEC, FULL, Q8>, dim3(b.parts), dim3(kBwdThreads),
                      ring_bytes<T, Q8>(p, b), st, p, b.r,
                      RingWait{d.status, d.wait_limit_ns, d.debug_stop});
}
template <typename T, bool Q8>
cudaError_t bwd_any(const RmsBwd& p, const BwdPlan& b, const TrainDevice& d, cudaStream_t st) {
  static std::atomic<int> done[64];
  const cudaError_t e =
      allow_ring(reinterpret_cast<const void*>(&rms_bwd_any_kernel<T, Q8>), done, d.dev);
  if (e != cudaSuccess) return e;
  return launch_train(rms_bwd_any_kernel<T, Q8>, dim3(b.parts), dim3(kBwdThreads),
                      ring_bytes<T, Q8>(p, b), st, p, b.r,
                      RingWait{d.status, d.wait_limit_ns, d.debug_stop});
}

template <typename T, bool Q8>
cudaError_t bwd_launch(RmsBwd p, const BwdPlan& b, const TrainDevice& d, cudaStream_t st) {
  constexpr int VEC = 16 / sizeof(T);
  p.chunks = p.cols / VEC;
  cudaError_t e = cudaSuccess;
  switch (b.kind) {
    case kDirect:
      e = launch_train(rms_bwd_kernel<T, VEC, Q8>, dim3(b.parts), dim3(kBwdThreads),
                       (size_t)b.r.groups * p.cols * sizeof(float), st, p, b.r.nt, b.r.groups);
      break;
    case kRing:
      e = b.r.nt * 16 == p.cols ? bwd_ring<T, VEC, true, Q8>(p, b, d, st)
                                : bwd_ring<T, VEC, false, Q8>(p, b, d, st);
      break;
    case kAny:
      e = bwd_any<T, Q8>(p, b, d, st);
      break;
    case kWide:
      if (p.dw)
        e = launch_train(rms_bwd_cols_kernel<T, Q8>, dim3((unsigned)ceil_div(p.cols, 256), b.parts),
                         dim3(256), 0, st, p);
      if (e == cudaSuccess)
        e = launch_train(rms_bwd_wide_kernel<T, Q8>, dim3((unsigned)p.rows), dim3(1024), 0, st, p);
  }
  if (e == cudaSuccess && p.dw && (b.parts > 1 || b.kind == kWide))
    e = launch_train(rms_bwd_reduce_kernel<T>, dim3((unsigned)ceil_div(p.cols, 32)), dim3(32, 16), 0,
                     st, (const float*)p.part, b.parts, p.cols, static_cast<T*>(p.dw));
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

// Partial rows of whichever way the pass runs: the query does not know the operands.
size_t bwd_bytes(long long rows, int cols, int sms) {
  const long long most = 4LL * sms;
  return (size_t)(rows < most ? rows : most) * cols * sizeof(float);
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
  const bool q8 = total_scales != nullptr;
  const RmsBwd p{rows, cols,   0,    dy, lddy, q8 ? nullptr : total, ldt, k8, weight, rstd, dtotal,
                 lddt, dx,     lddx, static_cast<float*>(workspace), dweight};
  auto row16 = [&](const void* q, long long ld) { return !q || (vec16(q) && vec16_ld(ld, dtype)); };
  const bool v = row16(dy, lddy) && row16(p.x, ldt) && row16(dtotal, lddt) && row16(dx, lddx) &&
                 row16(weight, cols) && vec16_ld(cols, dtype) &&
                 (!q8 || (vec16(k8.q) && k8.ldq % 16 == 0 && cols % 16 == 0));
  const BwdPlan b = bwd_plan(rows, cols, dtype, d.sms, v, dtotal != nullptr, q8);
  if (dtype == B2G_F32)
    return launch_code(q8 ? bwd_launch<float, true>(p, b, d, st) : bwd_launch<float, false>(p, b, d, st));
  return launch_code(q8 ? bwd_launch<Bf16, true>(p, b, d, st) : bwd_launch<Bf16, false>(p, b, d, st));
}

}  // extern "C"
