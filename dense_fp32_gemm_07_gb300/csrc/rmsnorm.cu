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
#include "tcgen05.cuh"

namespace b2g {
namespace {

// ------------------------------------------------------------------- forward

struct RmsFwd {
  long long rows;
  int cols, chunks;  // chunks of 16 bytes of a row, the last one perhaps cut short
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

// total of one chunk of x and of the residual, rounded, and its values.
template <typename T>
__device__ __forceinline__ void add_residual(Pack<T, kVec<T>>& x, const Pack<T, kVec<T>>& res,
                                             float (&f)[kVec<T>]) {
  float g[kVec<T>];
  x.get(f), res.get(g);
#pragma unroll
  for (int j = 0; j < kVec<T>; ++j) f[j] += g[j];
  x.set(f);
  x.get(f);
}

// The sum of a chunk's squares, added in pairs: few roundings reach the row's sum.
template <int VEC>
__device__ __forceinline__ float squares(const float (&f)[VEC]) {
  float s[VEC / 2];
#pragma unroll
  for (int j = 0; j < VEC / 2; ++j) s[j] = fmaf(f[2 * j + 1], f[2 * j + 1], f[2 * j] * f[2 * j]);
#pragma unroll
  for (int n = VEC / 4; n; n /= 2)
#pragma unroll
    for (int j = 0; j < n; ++j) s[j] += s[j + n];
  return s[0];
}
__device__ __forceinline__ float rstd_of(float sum, int cols, float eps) {
  return __frsqrt_rn(sum / (float)cols + eps);
}

// How a call's rows stand in memory (anyrow.cuh): on 16-byte boundaries; all of its
// matrices' at the same places within a 16-byte unit; anyhow.
enum Rows { kAligned, kPhase, kAny };

// One row per blockDim.x threads (from 8 lanes of a warp up; threadIdx.y picks the row of
// a block that has several), NCH chunks a thread, the weights fetched with the row.  Rows
// anyhow take shifted vectors (anyrow.cuh) and so do all rows off the boundaries whose
// results leave in 8 bits, since a scale's 32 columns are counted from the row's first.
//
// Several blocks an SM, each with all of its row on its way, keep HBM busy by themselves: a
// ring as in the backward pass is not needed.  With a residual, BF16: 8192 x 4096 40.3 us
// (6.66 TB/s), to 8 bits 36.7 (6.4), to both with total kept in 8 bits 51.8 (6.5); 8192 x 4095
// 51 us, to 8 bits 72; FP32 90 and 124.  One row of 4096: 1.9 us, the latency of a launch, a
// read, a sum over the block and a write.
template <typename T, int NCH, Rows ROWS>
__global__ void __launch_bounds__(kMaxRowThreads) rms_fwd_kernel(const __grid_constant__ RmsFwd p) {
  constexpr int VEC = kVec<T>;
  constexpr bool ANY = ROWS != kAligned;
  __shared__ float red[32];
  pdl_launch_dependents();
  pdl_wait();
  const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < p.rows;  // the others of the warp take part in its sums
  const int t = threadIdx.x, nt = blockDim.x, seg = nt < 32 ? nt : 32;
  const T* w = static_cast<const T*>(p.w);
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const T* res = static_cast<const T*>(p.res) + row * p.ldr;
  const int pad = ROWS == kPhase ? (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T)) : 0;
  const int chunks = live ? ROWS == kPhase ? (p.cols + pad + VEC - 1) / VEC : p.chunks : 0;
  const int e0 = t * VEC - pad, step = nt * VEC;
  auto in = [&](int i) { return t + i * nt < chunks; };
  Pack<T, VEC> raw[NCH], add[NCH], wr[NCH];
  if constexpr (ROWS == kPhase) {
    start_at<T>(raw, x, e0, step, p.cols, in);
    if (p.res) start_at<T>(add, res, e0, step, p.cols, in);
    ends_at<T>(raw, x, e0, step, p.cols, in);
    if (p.res) ends_at<T>(add, res, e0, step, p.cols, in);
  } else {
    Fetched fx[ANY ? NCH : 1], fr[ANY ? NCH : 1];
    load_chunks<T, ANY>(raw, fx, x, e0, step, p.cols, in);
    if (p.res) load_chunks<T, ANY>(add, fr, res, e0, step, p.cols, in);
    finish_chunks<T, ANY>(raw, fx, x, e0, step, p.cols, in);
    if (p.res) finish_chunks<T, ANY>(add, fr, res, e0, step, p.cols, in);
  }
  {
    Fetched fw[ANY ? NCH : 1];
    if (w) load_chunks<T, ANY>(wr, fw, w, e0, step, p.cols, in);
    if (w) finish_chunks<T, ANY>(wr, fw, w, e0, step, p.cols, in);
  }
  auto put = [&](void* to, long long ld, const Pack<T, VEC>& k, int i) {
    T* o = static_cast<T*>(to) + row * ld;
    if constexpr (ROWS == kPhase) {
      if (in(i)) store_at<T>(k, o, e0 + i * step, p.cols);
    } else {
      store_chunk<T, ANY>(k, o, t + i * nt, p.cols, in(i), seg);
    }
  };
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    float f[1][VEC];
    if (p.res)
      add_residual<T>(raw[i], add[i], f[0]);
    else
      raw[i].get(f[0]);
    if (p.total) put(p.total, p.ldt, raw[i], i);
    sum += squares<VEC>(f[0]);
    if (ROWS != kPhase && p.t8.q) encode_to<VEC, 1, ANY>(p.t8, row, t + i * nt, 0, chunks, p.cols, f);
  }
  const float rstd = rstd_of(row_sum(sum, red, nt), p.cols, p.eps);
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    float f[1][VEC], wf[VEC];
    raw[i].get(f[0]), wr[i].get(wf);
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[0][j] = f[0][j] * (w ? wf[j] : 1.f) * rstd;  // BF16: one rounding
    if (p.y) {
      Pack<T, VEC> o;
      o.set(f[0]);
      put(p.y, p.ldy, o, i);
    }
    if (ROWS != kPhase && p.y8.q) encode_to<VEC, 1, ANY>(p.y8, row, t + i * nt, 0, chunks, p.cols, f);
  }
  if (t == 0 && live && p.rstd) p.rstd[row] = rstd;
}

// Rows wider than the registers of a block: two passes, the second one from the caches.
template <typename T>
__global__ void __launch_bounds__(1024) rms_fwd_wide_kernel(const __grid_constant__ RmsFwd p) {
  constexpr int VEC = kVec<T>;
  __shared__ float red[32];
  pdl_launch_dependents();
  pdl_wait();
  const long long row = blockIdx.x;
  const T* w = static_cast<const T*>(p.w);
  auto load = [&](int c, Pack<T, VEC>& k, float (&f)[1][VEC]) {
    k.zero();
    if (c < p.chunks) load_chunk<T, true>(k, static_cast<const T*>(p.x) + row * p.ldx, c, p.cols);
    if (p.res) {
      Pack<T, VEC> r;
      r.zero();
      if (c < p.chunks) load_chunk<T, true>(r, static_cast<const T*>(p.res) + row * p.ldr, c, p.cols);
      add_residual<T>(k, r, f[0]);
    } else {
      k.get(f[0]);
    }
  };
  Pack<T, VEC> k;
  float f[1][VEC], sum = 0.f;
  for (int c = threadIdx.x; c < p.chunks; c += blockDim.x) {
    load(c, k, f);
    sum += squares<VEC>(f[0]);
  }
  const float rstd = rstd_of(block_sum(sum, red, blockDim.x >> 5), p.cols, p.eps);
  for (int c0 = 0; c0 < p.chunks; c0 += blockDim.x) {  // whole warps, for the scales
    const int c = c0 + threadIdx.x;
    load(c, k, f);
    if (p.total) store_chunk<T, true>(k, static_cast<T*>(p.total) + row * p.ldt, c, p.cols, c < p.chunks, 32);
    if (p.t8.q) {
      encode_to<VEC, 1, true>(p.t8, row, c, 0, p.chunks, p.cols, f);
      k.get(f[0]);
    }
    Pack<T, VEC> o;
    float wf[VEC];
    o.zero();
    if (w && c < p.chunks) load_chunk<T, true>(o, w, c, p.cols);
    o.get(wf);
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[0][j] = f[0][j] * (w ? wf[j] : 1.f) * rstd;
    o.set(f[0]);
    if (p.y) store_chunk<T, true>(o, static_cast<T*>(p.y) + row * p.ldy, c, p.cols, c < p.chunks, 32);
    if (p.y8.q) encode_to<VEC, 1, true>(p.y8, row, c, 0, p.chunks, p.cols, f);
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
  int cluster;  // the direct kernel's blocks are one cluster, which writes it
};

constexpr int kBwdThreads = 512;  // 16 columns a thread
constexpr int kCluster = 8;       // blocks of a cluster, at most
// Rows off the 16-byte boundaries: 24 columns a thread and a third more registers, which their
// ends take.
constexpr int kPhaseThreads = 384, kPhaseCols = 24;

// Chunk c of the kept rows, from the type or from 8 bits.
template <typename T, bool Q8, bool ANY>
__device__ __forceinline__ void load_kept(const RmsBwd& p, long long row, int c, float (&f)[kVec<T>]) {
  if constexpr (Q8) {
    Codes<kVec<T>> k;
    load_codes<kVec<T>, ANY>(k, p.k8, row, c, p.cols);
    const float s = scale_value(p.k8.s[row * p.k8.lds + c / (kScaleBlock / kVec<T>)]);
    k.get(f);
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j) f[j] *= s;
  } else {
    Pack<T, kVec<T>> k;
    load_chunk<T, ANY>(k, static_cast<const T*>(p.x) + row * p.ldx, c, p.cols);
    k.get(f);
  }
}

// The end of a block: its groups' sums of dy xhat (sums: [groups][cols] in shared memory),
// added in group order.
template <typename T>
__device__ __forceinline__ void leave_sums(const RmsBwd& p, const float* sums, int groups) {
  for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
    float a = sums[c];
    for (int i = 1; i < groups; ++i) a += sums[(size_t)i * p.cols + c];
    if (gridDim.x == 1)
      static_cast<T*>(p.dw)[c] = from_f32<T>(a);
    else
      p.part[(size_t)blockIdx.x * p.cols + c] = a;
  }
}

// The same of a cluster that is the whole grid: block k adds its share of the columns over the
// blocks, in their order, from their shared memory.
template <typename T>
__device__ __forceinline__ void leave_cluster(const RmsBwd& p, float* sums, int groups) {
  for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
    float a = sums[c];
    for (int i = 1; i < groups; ++i) a += sums[(size_t)i * p.cols + c];
    sums[c] = a;
  }
  cluster_sync();
  for (int c = threadIdx.x + blockIdx.x * blockDim.x; c < p.cols; c += gridDim.x * blockDim.x) {
    float v[kCluster], a = 0.f;
#pragma unroll
    for (int k = 0; k < kCluster; ++k)
      v[k] = k < gridDim.x ? ld_shared_cluster_f32(mapa_shared(smem_addr(sums + c), k)) : 0.f;
#pragma unroll
    for (int k = 0; k < kCluster; ++k) a += v[k];
    static_cast<T*>(p.dw)[c] = from_f32<T>(a);
  }
  cluster_sync();  // nobody leaves while its sums are read
}

// Few or short rows: groups of nt threads (from 4 lanes of a warp up) with a row each, 16
// columns a thread, all of whose loads are on their way together.  Up to kCluster blocks are
// a cluster, which needs no second launch for dweight.  One row of 4096 BF16: 3.5 us; 16 rows
// 5.0 as a cluster; 128 rows 5.9 with the launch that adds 64 blocks'; 16384 x 64 FP32 7.8.
template <typename T, bool Q8, bool ANY>
__global__ void __launch_bounds__(kBwdThreads, 1)
    rms_bwd_kernel(const __grid_constant__ RmsBwd p, int nt, int groups) {
  extern __shared__ __align__(16) float sums[];  // [groups][cols], at the end
  __shared__ float red[2][16];
  constexpr int VEC = kVec<T>, NCH = 16 / VEC;
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
    if (!ANY && w && c < p.chunks) wr[i].load(w + c * VEC);
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
    const T* rd = static_cast<const T*>(p.dy) + row * p.lddy;
    const T* rx = static_cast<const T*>(p.x) + row * p.ldx;
    const T* rt = static_cast<const T*>(p.dtotal) + row * p.lddt;
    const int e0 = t * VEC, step = nt * VEC;
    auto in = [&](int i) { return t + i * nt < chunks; };
    // with ANY two chunks at a time: the vectors on their way take twice the registers
    auto load = [&](Pack<T, VEC>(&k)[NCH], const T* from) {
#pragma unroll
      for (int i = 0; i < NCH; i += 2) {
        if constexpr (ANY) {
          Fetched f[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) fetch<T>(f[j], from, e0 + (i + j) * step, p.cols, in(i + j));
#pragma unroll
          for (int j = 0; j < 2; ++j)
            finish<T>(k[i + j], f[j], from, e0 + (i + j) * step, p.cols, in(i + j));
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            k[i + j].zero();
            if (in(i + j)) k[i + j].load(from + e0 + (i + j) * step);
          }
        }
      }
    };
    load(dy, rd);
    if (!Q8) load(x, rx);
    if (!ANY && p.dtotal) load(dt, rt);
    if (ANY && w) load(wr, w);
    if constexpr (Q8) {
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        const int c = t + i * nt;
        q[i].zero(), byte[i] = 127;
        if (c < chunks) {
          load_codes<VEC, ANY>(q[i], p.k8, row, c, p.cols);
          byte[i] = p.k8.s[row * p.k8.lds + c / (kScaleBlock / VEC)];
        }
        if (ANY) asm volatile("" ::: "memory");  // one after another, for the registers
      }
    }
    float xh[NCH][VEC], g[NCH][VEC], along = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      float wf[VEC];
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
        xh[i][j] *= rstd;
        aw[i][j] = fmaf(g[i][j], xh[i][j], aw[i][j]);
        if (w) g[i][j] *= wf[j];
        along = fmaf(g[i][j], xh[i][j], along);
      }
    }
    const float mean = (nt < 32 ? row_sum(along, nullptr, nt) : group_sum(along, red[turn], group, nt)) * inv;
    turn ^= 1;
    if (ANY && p.dtotal) load(dt, rt);
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = t + i * nt;
      float d[VEC];
      if (!p.dtotal) dt[i].zero();
      dt[i].get(d);
#pragma unroll
      for (int j = 0; j < VEC; ++j) d[j] = fmaf(rstd, fmaf(-xh[i][j], mean, g[i][j]), d[j]);
      Pack<T, VEC> k;
      k.set(d);
      store_chunk<T, ANY>(k, static_cast<T*>(p.dx) + row * p.lddx, c, p.cols, c < chunks, nt < 32 ? nt : 32);
    }
  }
  if (!p.dw) return;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = (t + i * nt) * VEC;
    float* q = sums + (size_t)group * p.cols + c;
#pragma unroll
    for (int j = 0; j < VEC; j += 4) {
      if constexpr (!ANY) {
        if (c < p.cols)
          *reinterpret_cast<float4*>(q + j) = make_float4(aw[i][j], aw[i][j + 1], aw[i][j + 2], aw[i][j + 3]);
      } else {
#pragma unroll
        for (int e = j; e < j + 4; ++e)
          if (c + e < p.cols) q[e] = aw[i][e];
      }
    }
  }
  __syncthreads();
  if (p.cluster)
    leave_cluster<T>(p, sums, groups);
  else
    leave_sums<T>(p, sums, groups);
}

// Bytes of a ring's slot that one row of `cols` elements of `es` bytes takes: with PHASE, in
// the 16-byte units that it lies across, and one before them.
template <bool PHASE>
__host__ __device__ constexpr uint32_t row_slot(int cols, int es) {
  return PHASE ? (uint32_t)((cols * es + 15) / 16 * 16 + 32) : (uint32_t)(cols * es);
}

// The 16-byte units that a row lies across, and whether they are all of the matrix (not at its
// very ends).
struct RowUnits {
  const unsigned char* from;
  uint32_t bytes;
  bool inside;
  __device__ __forceinline__ RowUnits(const void* base, long long row, long long ld, long long rows, int cols,
                                      int es) {
    const uintptr_t first = reinterpret_cast<uintptr_t>(base), start = first + row * ld * es;
    const uintptr_t end = start + (uintptr_t)cols * es, last = first + ((rows - 1) * ld + cols) * es;
    const uintptr_t a = start & ~(uintptr_t)15, b = (end + 15) & ~(uintptr_t)15;
    from = reinterpret_cast<const unsigned char*>(a), bytes = (uint32_t)(b - a);
    inside = a >= first && b <= last;
  }
};

// Many rows: a ring (ring.cuh) of the rows of dy, of the kept rows and of dtotal together, 16
// columns a thread; the scales of 8-bit rows are fetched a row ahead.  FULL: every thread has
// all of its columns.
// PHASE: rows off the 16-byte boundaries, all at the same place within a 16-byte unit (8-bit
// rows on the boundaries).  The step from row to row of a group is a multiple of 16 bytes, so
// that the place, and with it a thread's columns, stays; the slots hold whole units.  The
// first and last rows, whose units may begin before the matrix or end after it, are read where
// they are.
// BF16, with dtotal and the sums' reduction: 8192 x 4096 45.6 us (5.9 TB/s), from 8 bits 44.2;
// 16384 x 4096 81 (6.6 TB/s): a further row costs what its bytes do, the first ones 9 us.
// 8192 x 4095 60 us (FP32 87), from 8 bits 78 (104); read row by row into registers, as above,
// 8192 x 4096 took 88.
template <typename T, bool FULL, bool Q8, bool PHASE>
__global__ void __launch_bounds__(PHASE ? kPhaseThreads : kBwdThreads, 1)
    rms_bwd_ring_kernel(const __grid_constant__ RmsBwd p, const __grid_constant__ Ring g,
                        const __grid_constant__ RingWait wait) {
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ __align__(8) unsigned long long bars[kBwdThreads / 32 * kRingStages];
  __shared__ float red[2][16];
  constexpr int VEC = kVec<T>, H = VEC / 2, NCH = (PHASE ? kPhaseCols : 16) / VEC, ES = (int)sizeof(T);
  constexpr int KS = Q8 ? 1 : ES;
  constexpr uint32_t kBefore = PHASE ? 16 : 0;  // where a row's units begin in its part of a slot
  pdl_launch_dependents();
  const int group = threadIdx.x / g.nt, t = threadIdx.x - group * g.nt;
  const uint32_t dslot = row_slot<PHASE>(p.cols, ES), kslot = row_slot<PHASE>(p.cols, KS);
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
  const T* dy0 = static_cast<const T*>(p.dy) + row0 * p.lddy;
  const int pad = PHASE ? (int)((reinterpret_cast<uintptr_t>(dy0) & 15u) / ES) : 0;
  const int chunks = PHASE ? (p.cols + pad + VEC - 1) / VEC : p.chunks;
  // A chunk's first column; of 8-bit rows computed anew each time with PHASE, as keeping what
  // depends on it for all rows would spill.
  auto first_of = [&](int i) {
    int c = t + i * g.nt;
    if (PHASE && Q8) asm volatile("" : "+r"(c));
    return c * VEC - pad;
  };
  const void* kept = Q8 ? p.k8.q : p.x;
  const long long ldk = Q8 ? p.k8.ldq : p.ldx;
  auto issue = [&](long long row, int s) {
    if (wait.debug_stop >= 0 && (row - row0) / step >= wait.debug_stop) return;
    const uint32_t bar = bar0 + 8u * s, dst = smem_addr(mine + (size_t)s * slot) + kBefore;
    const RowUnits d(p.dy, row, p.lddy, p.rows, p.cols, ES), k(kept, row, ldk, p.rows, p.cols, KS);
    const RowUnits q(p.dtotal ? p.dtotal : p.dy, row, p.dtotal ? p.lddt : p.lddy, p.rows, p.cols, ES);
    if (PHASE && !(d.inside && k.inside && q.inside)) {
      mbar_arrive(bar);  // nothing to wait for
      return;
    }
    mbar_arrive_expect_tx(bar, d.bytes + k.bytes + (p.dtotal ? q.bytes : 0));
    bulk_load(dst, d.from, d.bytes, bar);
    bulk_load(dst + dslot, k.from, k.bytes, bar);
    if (p.dtotal) bulk_load(dst + dslot + kslot, q.from, q.bytes, bar);
  };
  auto in_slot = [&](long long row) {
    if (!PHASE) return true;
    return RowUnits(p.dy, row, p.lddy, p.rows, p.cols, ES).inside &&
           RowUnits(kept, row, ldk, p.rows, p.cols, KS).inside &&
           (!p.dtotal || RowUnits(p.dtotal, row, p.lddt, p.rows, p.cols, ES).inside);
  };
  auto direct = [&](Pack<T, VEC>& to, const void* m, long long ld, long long row, int e) {
    const T* from = static_cast<const T*>(m) + row * ld;
    Fetched f;
    fetch<T>(f, from, e, p.cols, true);
    finish<T>(to, f, from, e, p.cols, true);
  };
  if (t == 0) {
    long long row = row0;
    for (int s = 0; s < g.stages && row < p.rows; ++s, row += step) issue(row, s);
  }
  F2 aw[NCH][H];
  Pack<T, VEC> wr[NCH];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
#pragma unroll
    for (int j = 0; j < H; ++j) aw[i][j] = f2(0.f, 0.f);
    float one[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) one[j] = 1.f;
    wr[i].set(one);
    if (p.w && t + i * g.nt < chunks) {
      Fetched f;
      fetch<T>(f, static_cast<const T*>(p.w), first_of(i), p.cols, true);
      finish<T>(wr[i], f, static_cast<const T*>(p.w), first_of(i), p.cols, true);
    }
  }
  float rstd = 0.f;
  // The scales of a chunk's columns: one, or with PHASE those of both blocks it lies across
  // (the second in the upper byte).
  uint32_t byte[NCH];
  auto fetch_scales = [&](long long row) {
    if constexpr (Q8) {
      const unsigned char* s = p.k8.s + row * p.k8.lds;
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        byte[i] = 127;
        if (FULL || t + i * g.nt < chunks) {
          const int c = first_of(i);
          byte[i] = s[(PHASE ? max(c, 0) : c) / kScaleBlock];
          if (PHASE) byte[i] |= (uint32_t)s[min(c + VEC - 1, p.cols - 1) / kScaleBlock] << 8;
        }
      }
    }
  };
  // what is fetched past the ring, a row ahead (with PHASE, which is short of registers, the
  // scales of the row itself)
  if (row0 < p.rows) {
    rstd = p.rstd[row0];
    if (!PHASE) fetch_scales(row0);
  }
  RingPos at;
  int turn = 0;
  bool alive = true;  // false once a wait has run out: no more waits, no more copies
  for (long long row = row0; row < p.rows; row += step) {
    const float r = rstd;
    const F2 r2 = f2(r, r);
    if (PHASE) fetch_scales(row);
    uint32_t scales[NCH];
#pragma unroll
    for (int i = 0; i < NCH; ++i) scales[i] = Q8 ? byte[i] : 0;
    if (row + step < p.rows) {
      rstd = p.rstd[row + step];
      if (!PHASE) fetch_scales(row + step);
    }
    if (alive) alive = wait_row(bar0, at, g.stages, row, step, p.rows, t == 0, wait);
    const unsigned char* here = mine + (size_t)at.s * slot + kBefore;
    const bool there = in_slot(row);
    F2 xh[NCH][H], gr[NCH][H];  // xhat, and g = dy weight
    Pack<T, VEC> past[NCH];
    F2 s0 = f2(0.f, 0.f), s1 = f2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = t + i * g.nt, e = first_of(i);
      past[i].zero();
      if (FULL || c < chunks) {
        Pack<T, VEC> k, dk;
        Codes<VEC> q;
        F2 d[H], wf[H];
        if (!PHASE || there) {
          dk.load(reinterpret_cast<const T*>(here) + c * VEC);
          if constexpr (!Q8)
            k.load(reinterpret_cast<const T*>(here + dslot) + c * VEC);
          else if constexpr (PHASE)
            q.load_shared(here + dslot - kBefore, kBefore + e);  // the row begins on a boundary
          else
            q.load(here + dslot + c * VEC);
          if (!PHASE && p.dtotal) past[i].load(reinterpret_cast<const T*>(here + dslot + kslot) + c * VEC);
          if (PHASE && (e < 0 || e + VEC > p.cols)) {
            cut<T>(dk, -e, p.cols - e);
            if constexpr (Q8)
              q.keep(-e, p.cols - e);
            else
              cut<T>(k, -e, p.cols - e);
          }
        } else {
          direct(dk, p.dy, p.lddy, row, e);
          if constexpr (Q8)
            q.load(p.k8.q + row * p.k8.ldq + e, -e, p.cols - e);
          else
            direct(k, p.x, p.ldx, row, e);
        }
        dk.get2(d), wr[i].get2(wf);
        if constexpr (Q8) {
          float f[VEC];
          q.get(f);
          const float lo = scale_value(scales[i] & 255u);
          if constexpr (PHASE) {
            const float hi = scale_value(scales[i] >> 8);
            const int edge = kScaleBlock - (e & (kScaleBlock - 1));  // from here on the second block
#pragma unroll
            for (int j = 0; j < VEC; ++j) f[j] *= j < edge ? lo : hi;
          } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) f[j] *= lo;
          }
#pragma unroll
          for (int j = 0; j < H; ++j) xh[i][j] = f2(f[2 * j], f[2 * j + 1]);
        } else {
          k.get2(xh[i]);
        }
#pragma unroll
        for (int j = 0; j < H; ++j) {
          xh[i][j] = mul2(xh[i][j], r2);
          gr[i][j] = mul2(d[j], wf[j]);
          aw[i][j] = fma2(d[j], xh[i][j], aw[i][j]);
          if (j & 1)
            s1 = fma2(gr[i][j], xh[i][j], s1);
          else
            s0 = fma2(gr[i][j], xh[i][j], s0);
        }
      }
    }
    if (g.nt == 32) __syncwarp();  // no barrier in the sum: the warp's reads of the slot
    const float mean = group_sum(f2_sum(add2(s0, s1)), red[turn], group, g.nt) * inv;
    // the slot may be filled again: all of the group have read it (but for dtotal with PHASE)
    auto refill = [&] {
      if (t == 0 && alive && row + (long long)g.stages * step < p.rows)
        issue(row + (long long)g.stages * step, at.s);
    };
    if (!PHASE) refill();
    const F2 minus = f2(-mean, -mean);
    T* dx = static_cast<T*>(p.dx) + row * p.lddx;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = t + i * g.nt;
      if (FULL || c < chunks) {
        F2 d[H];
        if (PHASE && p.dtotal) {  // only now: no registers to keep it in
          if (there)
            past[i].load(reinterpret_cast<const T*>(here + dslot + kslot) + c * VEC);
          else
            direct(past[i], p.dtotal, p.lddt, row, first_of(i));
        }
        past[i].get2(d);
#pragma unroll
        for (int j = 0; j < H; ++j) d[j] = fma2(r2, fma2(xh[i][j], minus, gr[i][j]), d[j]);
        Pack<T, VEC> k;
        k.set2(d);
        if constexpr (PHASE)
          store_at<T>(k, dx, first_of(i), p.cols);
        else
          k.store(dx + c * VEC);
      }
    }
    if (PHASE) {
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(g.nt) : "memory");
      refill();
    }
    turn ^= 1;
    at.next(g.stages);
  }
  if (!p.dw) return;
  __syncthreads();  // no ring has a copy on its way: its memory now takes the groups' sums
  float* sums = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = first_of(i);
#pragma unroll
    for (int j = 0; j < H; j += 2) {
      float* q = sums + (size_t)group * p.cols + c + 2 * j;
      float4 v;
      f2_split(aw[i][j], v.x, v.y), f2_split(aw[i][j + 1], v.z, v.w);
      if constexpr (PHASE) {
        const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + 2 * j + e >= 0 && c + 2 * j + e < p.cols) q[e] = f[e];
      } else if (FULL || c < p.cols) {
        *reinterpret_cast<float4*>(q) = v;
      }
    }
  }
  __syncthreads();
  leave_sums<T>(p, sums, g.groups);
}

// Rows wider than the registers of a block: dx in two passes over the row.
template <typename T, bool Q8>
__global__ void __launch_bounds__(1024) rms_bwd_wide_kernel(const __grid_constant__ RmsBwd p) {
  constexpr int VEC = kVec<T>;
  __shared__ float red[32];
  pdl_launch_dependents();
  pdl_wait();
  const long long row = blockIdx.x;
  const T* w = static_cast<const T*>(p.w);
  const float rstd = p.rstd[row];
  // xhat and g of chunk c
  auto load = [&](int c, float (&xh)[VEC], float (&g)[VEC]) {
    load_kept<T, Q8, true>(p, row, c, xh);
    Pack<T, VEC> k;
    load_chunk<T, true>(k, static_cast<const T*>(p.dy) + row * p.lddy, c, p.cols);
    k.get(g);
    float wf[VEC];
    if (w) {
      load_chunk<T, true>(k, w, c, p.cols);
      k.get(wf);
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) xh[j] *= rstd, g[j] *= w ? wf[j] : 1.f;
  };
  float along = 0.f, xh[VEC], g[VEC];
  for (int c = threadIdx.x; c < p.chunks; c += blockDim.x) {
    load(c, xh, g);
#pragma unroll
    for (int j = 0; j < VEC; ++j) along = fmaf(g[j], xh[j], along);
  }
  const float mean = block_sum(along, red, blockDim.x >> 5) / (float)p.cols;
  for (int c0 = 0; c0 < p.chunks; c0 += blockDim.x) {
    const int c = c0 + threadIdx.x;
    Pack<T, VEC> k;
    k.zero();
    if (c < p.chunks) {
      float d[VEC];
      load(c, xh, g);
      if (p.dtotal) load_chunk<T, true>(k, static_cast<const T*>(p.dtotal) + row * p.lddt, c, p.cols);
      k.get(d);
#pragma unroll
      for (int j = 0; j < VEC; ++j) d[j] = fmaf(rstd, fmaf(-xh[j], mean, g[j]), d[j]);
      k.set(d);
    }
    store_chunk<T, true>(k, static_cast<T*>(p.dx) + row * p.lddx, c, p.cols, c < p.chunks, 32);
  }
}

// The wide rows' dweight: block (x, y) adds rows y, y + gridDim.y, ... of its 64 chunks into
// partial row y.  Runs before rms_bwd_wide_kernel, which may overwrite dy.
template <typename T, bool Q8>
__global__ void __launch_bounds__(64) rms_bwd_cols_kernel(const __grid_constant__ RmsBwd p) {
  constexpr int VEC = kVec<T>;
  pdl_launch_dependents();
  pdl_wait();
  const int c = blockIdx.x * 64 + threadIdx.x;
  if (c >= p.chunks) return;
  float a[VEC], xh[VEC], d[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) a[j] = 0.f;
  for (long long row = blockIdx.y; row < p.rows; row += gridDim.y) {
    load_kept<T, Q8, true>(p, row, c, xh);
    Pack<T, VEC> k;
    load_chunk<T, true>(k, static_cast<const T*>(p.dy) + row * p.lddy, c, p.cols);
    k.get(d);
    const float rstd = p.rstd[row];
#pragma unroll
    for (int j = 0; j < VEC; ++j) a[j] = fmaf(d[j], xh[j] * rstd, a[j]);
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j)
    if (c * VEC + j < p.cols) p.part[(size_t)blockIdx.y * p.cols + c * VEC + j] = a[j];
}

// dweight: warp y adds the partial rows y, y + 16, ... in order, then the warps' sums are
// added in warp order.  Bound: latency, about 3 us.
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

// Chunks a thread may hold; one more for the part of a unit before the row.
template <Rows ROWS>
constexpr int kMaxFwd = ROWS == kPhase ? 5 : 4;

template <typename T, Rows ROWS, int NCH = 1>
cudaError_t fwd_kernel(int nch, dim3 grid, dim3 block, cudaStream_t st, const RmsFwd& p) {
  if constexpr (NCH < kMaxFwd<ROWS>) {
    if (nch > NCH) return fwd_kernel<T, ROWS, NCH + 1>(nch, grid, block, st, p);
  }
  return launch_train(rms_fwd_kernel<T, NCH, ROWS>, grid, block, 0, st, p);
}

template <typename T, Rows ROWS>
cudaError_t fwd_launch(RmsFwd p, int sms, cudaStream_t st) {
  p.chunks = (int)ceil_div(p.cols, kVec<T>);
  const int most = (int)ceil_div(p.cols + (ROWS == kPhase ? kVec<T> - 1 : 0), kVec<T>);  // of any row
  constexpr int least = 8;  // lanes a row: a block of 32 columns stays within a warp
  // chunks a thread: one where there are few rows, for the shortest path; more otherwise, for
  // the fewest barriers a byte, but two where rows off the boundaries take twice the registers
  int nt = 0;
  for (int per = p.rows <= 2 * sms ? 1 : ROWS == kAligned ? 4 : 2; !nt && per <= kMaxFwd<ROWS>; ++per)
    nt = most <= 32 * per ? row_threads(most, per, least)
         : most <= kMaxRowThreads * per ? (int)round_up(ceil_div(most, per), 32) : 0;
  if (!nt)
    return launch_train(rms_fwd_wide_kernel<T>, dim3((unsigned)p.rows), dim3(1024), 0, st, p);
  const int ry = nt <= 32 ? 128 / nt : 1;
  const dim3 grid((unsigned)ceil_div(p.rows, ry)), block(nt, ry);
  return fwd_kernel<T, ROWS>((int)ceil_div(most, nt), grid, block, st, p);
}

// How the backward pass runs.
enum BwdKind { kDirect, kRing, kWide };
struct BwdPlan {
  BwdKind kind;
  Ring r;     // stages only where there is a ring
  int parts;  // blocks, each leaving one partial row of dweight
  bool cluster;
};

constexpr int kBwdRing = 224 * 1024;  // bytes of the rings
// Rows up to these lengths, of which a warp of the ring has too few columns for its lanes, go to
// the direct kernel.  BF16, us there and in the ring: 16384 x 128 8.1 and 11.5, x 256 11.5 and
// 12.7, x 512 17.0 and 17.3; off the boundaries x 101 15.8 and 18.6, x 201 27 and 20.
constexpr int kNarrow = 256, kNarrowPhase = 128;

uint32_t slot_of(int cols, size_t es, bool phase, bool past, bool q8) {
  const int e = (int)es, k = q8 ? 1 : e;
  return phase ? row_slot<true>(cols, k) + row_slot<true>(cols, e) * (past ? 2 : 1)
               : row_slot<false>(cols, k) + row_slot<false>(cols, e) * (past ? 2 : 1);
}

// past: a dtotal; q8: 8-bit rows.
BwdPlan bwd_plan(long long rows, int cols, int dtype, int sms, Rows how, bool past, bool q8) {
  BwdPlan b{kWide, {}, 0, false};
  const size_t es = type_size(dtype);
  // whole warps that hold a row with the part of a unit before it
  auto ring = [&](int threads, int per, bool phase) {
    const long long need = ceil_div(cols + (phase ? 16 / (int)es - 1 : 0), per);
    Ring r{(int)round_up(need, 32), 0, 0};
    if (r.nt > threads) return r;
    r.groups = threads / r.nt;
    const size_t s = kBwdRing / ((size_t)slot_of(cols, es, phase, past, q8) * r.groups);
    r.stages = (int)(s < (size_t)kRingStages ? s : (size_t)kRingStages);
    return r;
  };
  if (cols <= 16 * kBwdThreads) {
    b.r = how == kPhase ? ring(kPhaseThreads, kPhaseCols, true) : ring(kBwdThreads, 16, false);
    b.kind = kRing;
    // short rows, and one row a group: no second row to wait for
    if (how == kAny || (how == kPhase && sms < 8) || rows <= (long long)b.r.groups * sms ||
        cols <= (how == kPhase ? kNarrowPhase : kNarrow) || b.r.stages < 2) {
      b.kind = kDirect;
      b.r.nt = 4;
      while (b.r.nt * 16 < cols) b.r.nt *= 2;
      b.r.groups = kBwdThreads / b.r.nt;
    }
  }
  long long most = b.kind != kWide ? sms : 4LL * sms;
  const long long fair = ceil_div(rows, b.kind != kWide ? b.r.groups : 4);
  if (b.kind == kRing && how == kPhase) most = sms / 8 * 8;  // steps of whole 16-byte units
  b.parts = (int)(fair < most ? fair : most);
  // As fast as a second launch while groups have one row each (16 x 4096 BF16 5.0 us both ways,
  // 48 rows 7.4 in a cluster and 5.2), and a launch less for the host: calls one after another
  // 5.2 us each, 7.0 with two launches.
  b.cluster = b.kind == kDirect && fair > 1 && fair <= kCluster;
  return b;
}

// launch_train of blocks that are one cluster.
template <typename... P, typename... A>
cudaError_t launch_cluster(void (*kern)(P...), int blocks, dim3 block, size_t smem, cudaStream_t st, A... args) {
  return [&](P... typed) {
    void* ptrs[] = {const_cast<void*>(static_cast<const void*>(&typed))...};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks), cfg.blockDim = block, cfg.dynamicSmemBytes = smem, cfg.stream = st;
    cfg.attrs = attr, cfg.numAttrs = 2;
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(kern), ptrs);
  }(args...);
}

template <typename T, bool FULL, bool Q8, bool PHASE>
cudaError_t bwd_ring(const RmsBwd& p, const BwdPlan& b, const TrainDevice& d, cudaStream_t st) {
  static std::atomic<int> done[64];
  const cudaError_t e = allow_ring(
      reinterpret_cast<const void*>(&rms_bwd_ring_kernel<T, FULL, Q8, PHASE>), done, d.dev, kBwdRing);
  if (e != cudaSuccess) return e;
  // the rings, and at the end the groups' column sums
  const size_t rings = (size_t)b.r.groups * b.r.stages * slot_of(p.cols, sizeof(T), PHASE, p.dtotal, Q8);
  const size_t sums = (size_t)b.r.groups * p.cols * sizeof(float);
  return launch_train(rms_bwd_ring_kernel<T, FULL, Q8, PHASE>, dim3(b.parts), dim3(b.r.groups * b.r.nt),
                      rings > sums ? rings : sums, st, p, b.r,
                      RingWait{d.status, d.wait_limit_ns, d.debug_stop});
}

template <typename T, bool Q8, Rows ROWS>
cudaError_t bwd_launch(RmsBwd p, int dtype, const TrainDevice& d, cudaStream_t st) {
  p.chunks = (int)ceil_div(p.cols, kVec<T>);
  const BwdPlan b = bwd_plan(p.rows, p.cols, dtype, d.sms, ROWS, p.dtotal, Q8);
  cudaError_t e = cudaSuccess;
  if (b.kind == kDirect) {
    const size_t sums = (size_t)b.r.groups * p.cols * sizeof(float);
    p.cluster = b.cluster;
    e = b.cluster ? launch_cluster(rms_bwd_kernel<T, Q8, ROWS != kAligned>, b.parts, dim3(kBwdThreads), sums, st,
                                   p, b.r.nt, b.r.groups)
                  : launch_train(rms_bwd_kernel<T, Q8, ROWS != kAligned>, dim3(b.parts), dim3(kBwdThreads), sums,
                                 st, p, b.r.nt, b.r.groups);
  } else if (b.kind == kRing) {
    if constexpr (ROWS == kPhase)
      e = bwd_ring<T, false, Q8, true>(p, b, d, st);
    else if (b.r.nt * 16 == p.cols)
      e = bwd_ring<T, true, Q8, false>(p, b, d, st);
    else
      e = bwd_ring<T, false, Q8, false>(p, b, d, st);
  } else {
    if (p.dw)
      e = launch_train(rms_bwd_cols_kernel<T, Q8>, dim3((unsigned)ceil_div(p.chunks, 64), b.parts), dim3(64),
                       0, st, p);
    if (e == cudaSuccess)
      e = launch_train(rms_bwd_wide_kernel<T, Q8>, dim3((unsigned)p.rows), dim3(1024), 0, st, p);
  }
  if (e == cudaSuccess && p.dw && !b.cluster && (b.parts > 1 || b.kind == kWide))
    e = launch_train(rms_bwd_reduce_kernel<T>, dim3((unsigned)ceil_div(p.cols, 32)), dim3(32, 16), 0,
                     st, (const float*)p.part, b.parts, p.cols, static_cast<T*>(p.dw));
  return e;
}

// Whether matrices (those that are given) have their rows at the same places within a 16-byte
// unit.
struct Place16 {
  bool same = true;
  int at = -1;
  long long step = 0;
  void add(const void* q, long long ld, int dtype) {
    if (!q) return;
    const int a = (int)(reinterpret_cast<uintptr_t>(q) & 15u);
    const long long s = ld * (long long)type_size(dtype) % 16;
    if (at < 0) at = a, step = s;
    same = same && a == at && s == step;
  }
};

int check_rows(int dtype, long long rows, int cols) {
  if (!type_ok(dtype)) return B2G_ERR_INVALID_TYPE;
  if (rows < 0 || cols < 0 || rows > 0x7fffffffLL || cols > kMaxLength) return B2G_ERR_INVALID_DIM;
  return 0;
}

bool ld_ok(long long ld, int cols) { return ld >= (cols > 1 ? cols : 1); }
bool codes_ok(const Rows8& k, int cols) {  // where they are given
  return !k.q || (ld_ok(k.ldq, cols) && k.lds >= scale_count(cols > 1 ? cols : 1));
}

// Partial rows of whichever way the pass runs: the query does not know the operands.
size_t bwd_bytes(long long rows, int cols, int sms) {
  const long long most = 4LL * sms;
  return (size_t)(rows < most ? rows : most) * cols * sizeof(float);
}

// vec: codes that go at a time.
Rows8 rows8(void* q, long long ldq, void* s, long long lds, int vec) {
  Rows8 r{static_cast<unsigned char*>(q), ldq, static_cast<unsigned char*>(s), lds, 0};
  r.vec = codes_vec(r, vec);
  return r;
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
  const int vec = dtype == B2G_F32 ? 4 : 8;
  const Rows8 y8 = rows8(y_codes, ldyq, y_scales, ldys, vec);
  const Rows8 t8 = rows8(total_codes, ldtq, total_scales, ldts, vec);
  if (!ld_ok(ldx, cols) || (residual && !ld_ok(ldr, cols)) || (total && !ld_ok(ldt, cols)) ||
      (y && !ld_ok(ldy, cols)) || !codes_ok(y8, cols) || !codes_ok(t8, cols))
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
  const bool v = row16(x, ldx) && row16(residual, ldr) && row16(total, ldt) && row16(y, ldy) &&
                 row16(weight, cols) && vec16_ld(cols, dtype) && y8.vec && t8.vec;
  Place16 at;
  at.add(x, ldx, dtype), at.add(residual, ldr, dtype), at.add(total, ldt, dtype), at.add(y, ldy, dtype);
  const bool phase = at.same && !y8.q && !t8.q;  // a scale's columns are counted from the row's first
  if (dtype == B2G_F32)
    return launch_code(v       ? fwd_launch<float, kAligned>(p, d.sms, st)
                       : phase ? fwd_launch<float, kPhase>(p, d.sms, st)
                               : fwd_launch<float, kAny>(p, d.sms, st));
  return launch_code(v       ? fwd_launch<Bf16, kAligned>(p, d.sms, st)
                     : phase ? fwd_launch<Bf16, kPhase>(p, d.sms, st)
                             : fwd_launch<Bf16, kAny>(p, d.sms, st));
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
  const Rows8 k8 = total_scales ? rows8(const_cast<void*>(total), ldt, const_cast<void*>(total_scales), ldts,
                                       dtype == B2G_F32 ? 4 : 8)
                               : Rows8{};
  if (!ld_ok(lddy, cols) || !ld_ok(ldt, cols) || !codes_ok(k8, cols) || (dtotal && !ld_ok(lddt, cols)) ||
      !ld_ok(lddx, cols))
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
                 lddt, dx,     lddx, static_cast<float*>(workspace), dweight, 0};
  auto row16 = [&](const void* q, long long ld) { return !q || (vec16(q) && vec16_ld(ld, dtype)); };
  const bool v = row16(dy, lddy) && row16(p.x, ldt) && row16(dtotal, lddt) && row16(dx, lddx) &&
                 row16(weight, cols) && vec16_ld(cols, dtype) &&
                 (!q8 || (vec16(k8.q) && k8.ldq % 16 == 0 && cols % 16 == 0));
  Place16 at;
  at.add(dy, lddy, dtype), at.add(p.x, ldt, dtype), at.add(dtotal, lddt, dtype), at.add(dx, lddx, dtype);
  const bool phase = at.same && (!q8 || (vec16(k8.q) && k8.ldq % 16 == 0));
  auto run = [&](auto kept, auto how) {
    constexpr bool Q8 = decltype(kept)::value;
    constexpr Rows ROWS = decltype(how)::value;
    return launch_code(dtype == B2G_F32 ? bwd_launch<float, Q8, ROWS>(p, dtype, d, st)
                                        : bwd_launch<Bf16, Q8, ROWS>(p, dtype, d, st));
  };
  auto with = [&](auto kept) {
    return v       ? run(kept, std::integral_constant<Rows, kAligned>())
           : phase ? run(kept, std::integral_constant<Rows, kPhase>())
                   : run(kept, std::integral_constant<Rows, kAny>());
  };
  return q8 ? with(std::true_type()) : with(std::false_type());
}

}  // extern "C"
