// ring.cuh -- what the norms of matrix rows share (layernorm.cu, rmsnorm.cu): sums over the
// threads of a row, and rings of rows in shared memory that bulk copies fill ahead of use.
#pragma once
#include <atomic>

#include "train_common.cuh"

namespace b2g {

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

constexpr int kRingBytes = 192 * 1024;
constexpr int kRingStages = 16;  // at most

struct Ring {
  int nt, groups, stages;
};

struct RingPos {
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++s == stages) s = 0, ph ^= 1u;
  }
};

// A ring's waits, and where its copies stop in a test of them.
struct RingWait {
  unsigned int* status;
  unsigned long long limit_ns;
  int debug_stop;  // >= 0: rows a group starts to copy
};

// After a wait for `row` has run out: the group's copies still on their way, which are those
// of the next `stages` rows at most, land before its ring is used for anything else or left
// (one wait that runs out again ends this).
static __device__ __noinline__ void drain_ring(uint32_t bar0, int s, uint32_t ph, int stages, long long row,
                                        long long step, long long rows, const RingWait& w) {
  for (int i = 0; i < stages && row < rows; ++i, row += step) {
    if (!mbar_wait(bar0 + 8u * s, ph, w.limit_ns, w.status, kStatusTimeoutDrain)) return;
    if (++s == stages) s = 0, ph ^= 1u;
  }
}

// Wait for `row`'s copy; `first`: the thread that started it.  False when the wait ran out.
__device__ __forceinline__ bool wait_row(uint32_t bar0, const RingPos& at, int stages, long long row,
                                         long long step, long long rows, bool first,
                                         const RingWait& w) {
  if (mbar_wait(bar0 + 8u * at.s, at.ph, w.limit_ns, w.status, kStatusTimeoutFull)) return true;
  if (first) drain_ring(bar0, at.s, at.ph, stages, row, step, rows, w);
  return false;
}

// A sum over a group's nt threads (whole warps); `ex` is one of two exchange buffers used
// by turns.
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

// A row of any alignment on its way through a slot of the ring: a bulk copy moves the
// 16-byte units that lie inside the row, to the place they have within a 16-byte unit;
// the few elements before and after them are read where they are.
template <typename T>
struct AnyRow {
  const T* row;
  uint32_t off;    // of the row's first byte within its 16-byte unit
  int head, in;    // elements [head, head + in) are in the slot
  __device__ __forceinline__ AnyRow(const T* r, int cols) : row(r) {
    const uintptr_t start = reinterpret_cast<uintptr_t>(r), end = start + (size_t)cols * sizeof(T);
    off = (uint32_t)(start & 15u);
    const uintptr_t a = (start + 15u) & ~(uintptr_t)15u, b = end & ~(uintptr_t)15u;
    head = (int)((a - start) / sizeof(T));
    in = b > a ? (int)((b - a) / sizeof(T)) : 0;
  }
  __device__ __forceinline__ uint32_t bytes() const { return (uint32_t)(in * (int)sizeof(T)); }
  __device__ __forceinline__ void copy(uint32_t slot, uint32_t bar) const {
    if (in) bulk_load(slot + (off ? 16u : 0u), row + head, bytes(), bar);
  }
  // Element c as the slot has it: only the elements [head, head + in) are the row's.
  __device__ __forceinline__ float at(const unsigned char* slot, int c) const {
    return to_f32(reinterpret_cast<const T*>(slot + off)[c]);
  }
  // The others, at most 16 bytes' worth at either end: thread t of nt holds columns
  // t + i * nt, so at most one of each end, in i = 0 and in its last column.
  struct Ends {
    bool first, last;
    int i_last;
    float v_first, v_last;
    __device__ __forceinline__ float pick(int i, float v) const {
      if (i == 0 && first) v = v_first;
      return last && i == i_last ? v_last : v;
    }
  };
  __device__ __forceinline__ Ends ends(int t, int nt, int cols) const {
    Ends e;
    const int c = t < cols ? cols - 1 - (cols - 1 - t) % nt : 0;  // this thread's last column
    e.first = t < head && t < cols, e.last = t < cols && c >= head + in;
    e.i_last = c / nt;
    e.v_first = e.first ? to_f32(row[t]) : 0.f, e.v_last = e.last ? to_f32(row[c]) : 0.f;
    return e;
  }
};
// Bytes of a slot for one such row.
inline __host__ __device__ size_t any_slot(int cols, size_t es) {
  return ((size_t)cols * es + 15) / 16 * 16 + 16;
}

// ------------------------------------------------------------------ host side

constexpr int kMaxRowThreads = 512;

// Threads for one row of `chunks` chunks with at most `per` chunks a thread:
// the smallest power of two from `least` to kMaxRowThreads, or 0 when those are too few.
inline int row_threads(int chunks, int per, int least) {
  for (int t = least; t <= kMaxRowThreads; t *= 2)
    if ((long long)t * per >= chunks) return t;
  return 0;
}

// The ring of a block of `threads` for rows of `cols` columns in slots of `slot` bytes,
// `per` columns a thread, leaving `reserved` bytes; stages < 2 when they do not fit.
inline Ring ring_of(int threads, int per, int cols, size_t slot, size_t reserved) {
  Ring r{32, 0, 0};
  while (r.nt < threads && r.nt * per < cols) r.nt *= 2;
  r.groups = threads / r.nt;
  if (r.nt * per < cols || reserved >= kRingBytes) return r;
  const size_t s = (kRingBytes - reserved) / (slot * r.groups);
  r.stages = (int)(s < (size_t)kRingStages ? s : (size_t)kRingStages);
  return r;
}
// Opt in to the ring's shared memory, once per device and kernel.
inline cudaError_t allow_ring(const void* kern, std::atomic<int> (&done)[64], int dev,
                              int bytes = kRingBytes) {
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done[dev].store(1, std::memory_order_release);
  return e;
}

}  // namespace b2g
