// anyrow.cuh -- 16-byte chunks of matrix rows that begin anywhere: chunk c holds the
// elements from c * VEC on, wherever that is in memory.  A row off the 16-byte boundaries is
// read as the two aligned vectors a chunk lies across, shifted together, and written as
// aligned vectors with what the lane before holds; only what lies across the ends of a row
// or of a warp goes element by element.  Nothing outside the row is touched.
//
// Where all matrices of a call have their rows at the same places within a 16-byte unit (any
// contiguous ones of one width), chunks are counted from the unit that the row begins in
// instead: chunk c holds the elements from c * VEC - pad on, those of the row, and nothing
// has to be shifted.
#pragma once
#include "train_common.cuh"

namespace b2g {

template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

// 16 bytes from byte `off` (a multiple of T's size, below 16) of two vectors.
template <typename T>
__device__ __forceinline__ uint4 shift16(const uint4& a, const uint4& b, uint32_t off) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (off & 8u) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (off & 4u) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  if (sizeof(T) == 2 && (off & 2u)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T>
__device__ __forceinline__ uint32_t bits_of(T x) {
  if constexpr (sizeof(T) == 4)
    return __float_as_uint(x);
  else
    return (uint32_t)__bfloat16_as_ushort(x);
}
template <typename T>
__device__ __forceinline__ T element(const uint32_t (&w)[4], int j) {
  if constexpr (sizeof(T) == 4)
    return __uint_as_float(w[j]);
  else
    return __ushort_as_bfloat16((unsigned short)(w[j / 2] >> (16 * (j & 1))));
}

// Elements outside [from, to) become zero.
template <typename T>
__device__ __forceinline__ void cut(Pack<T, kVec<T>>& k, int from, int to) {
  uint32_t w[4] = {k.u.x, k.u.y, k.u.z, k.u.w};
  constexpr int per = 4 / (int)sizeof(T);
#pragma unroll
  for (int j = 0; j < kVec<T>; ++j)
    if (j < from || j >= to) w[j / per] &= per == 1 ? 0u : j % per ? 0x0000FFFFu : 0xFFFF0000u;
  k.u = make_uint4(w[0], w[1], w[2], w[3]);
}

// The aligned vectors that VEC elements lie across, on their way.  Loads of several chunks
// are started before the first one is finished: there is no branch between them.
struct Fetched {
  uint4 a, b;
};

// Starts the load of the elements from e0 on (e0 may be negative, and the last one past the
// row's end) of a row of `cols`, where `in`.
template <typename T>
__device__ __forceinline__ void fetch(Fetched& k, const T* row, int e0, int cols, bool in) {
  constexpr int es = (int)sizeof(T);
  const T* p = row + e0;
  const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u);
  const long long from = (long long)e0 * es - off, end = (long long)cols * es;
  const uint4* v = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) - off);
  k.a = k.b = make_uint4(0, 0, 0, 0);
  if (in && from >= 0 && from + 16 <= end) k.a = v[0];
  if (in && off && from >= -16 && from + 32 <= end) k.b = v[1];
}
// The elements, zeros outside the row.
template <typename T>
__device__ __forceinline__ void finish(Pack<T, kVec<T>>& k, const Fetched& f, const T* row, int e0, int cols,
                                       bool in) {
  constexpr int V = kVec<T>, es = (int)sizeof(T);
  const T* p = row + e0;
  const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u);
  const long long from = (long long)e0 * es - off, end = (long long)cols * es;
  k.u = off ? shift16<T>(f.a, f.b, off) : f.a;
  if (in && (from < 0 || from + (off ? 32 : 16) > end)) {  // across an end of the row
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (e0 + j >= 0 && e0 + j < cols) w[j * es / 4] |= bits_of<T>(p[j]) << (es == 2 ? 16 * (j & 1) : 0);
    k.u = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// N chunks at e0, e0 + step, ... of a row, those for which in(i).  Without ANY they are whole
// and on 16-byte boundaries.
template <typename T, bool ANY, int N, typename In>
__device__ __forceinline__ void load_chunks(Pack<T, kVec<T>> (&k)[N], Fetched (&f)[ANY ? N : 1], const T* row,
                                            int e0, int step, int cols, In in) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (ANY) {
      fetch<T>(f[i], row, e0 + i * step, cols, in(i));
    } else {
      k[i].zero();
      if (in(i)) k[i].load(row + e0 + i * step);
    }
  }
}
template <typename T, bool ANY, int N, typename In>
__device__ __forceinline__ void finish_chunks(Pack<T, kVec<T>> (&k)[N], const Fetched (&f)[ANY ? N : 1],
                                              const T* row, int e0, int step, int cols, In in) {
  if constexpr (ANY) {
#pragma unroll
    for (int i = 0; i < N; ++i) finish<T>(k[i], f[i], row, e0 + i * step, cols, in(i));
  }
}

// N chunks at e0, e0 + step, ... (row + e0 on a 16-byte boundary), zeros outside the row: those
// inside it are started first, then come the ones across its ends, element by element.
template <typename T, int N, typename In>
__device__ __forceinline__ void start_at(Pack<T, kVec<T>> (&k)[N], const T* row, int e0, int step, int cols,
                                         In in) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = e0 + i * step;
    k[i].zero();
    if (in(i) && e >= 0 && e + kVec<T> <= cols) k[i].load(row + e);
  }
}
template <typename T, int N, typename In>
__device__ __forceinline__ void ends_at(Pack<T, kVec<T>> (&k)[N], const T* row, int e0, int step, int cols,
                                        In in) {
  constexpr int per = 4 / (int)sizeof(T);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = e0 + i * step;
    if (in(i) && (e < 0 || e + kVec<T> > cols)) {
      uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < kVec<T>; ++j)
        if (e + j >= 0 && e + j < cols) w[j / per] |= bits_of<T>(row[e + j]) << (per == 2 ? 16 * (j & 1) : 0);
      k[i].u = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// Chunk c (it exists) of a row of `cols` elements, zeros past its end.
template <typename T, bool ANY>
__device__ __forceinline__ void load_chunk(Pack<T, kVec<T>>& k, const T* row, int c, int cols) {
  if constexpr (!ANY) {
    k.load(row + (long long)c * kVec<T>);
  } else {
    Fetched f;
    fetch<T>(f, row, c * kVec<T>, cols, true);
    finish<T>(k, f, row, c * kVec<T>, cols, true);
  }
}

// Stores the elements from e0 on, those of the row; row + e0 is on a 16-byte boundary.
template <typename T>
__device__ __forceinline__ void store_at(const Pack<T, kVec<T>>& k, T* row, int e0, int cols) {
  if (e0 >= 0 && e0 + kVec<T> <= cols) {
    k.store(row + e0);
  } else {
    const uint32_t w[4] = {k.u.x, k.u.y, k.u.z, k.u.w};
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j)
      if (e0 + j >= 0 && e0 + j < cols) row[e0 + j] = element<T>(w, j);
  }
}

// Stores chunk c (where `in`) of a row.  With ANY the whole warp takes part: consecutive lanes
// hold consecutive chunks, `seg` lanes (a power of two) of the same row.
template <typename T, bool ANY>
__device__ __forceinline__ void store_chunk(const Pack<T, kVec<T>>& k, T* row, int c, int cols, bool in,
                                            int seg) {
  constexpr int V = kVec<T>, es = (int)sizeof(T);
  T* p = row + (long long)c * V;
  if constexpr (!ANY) {
    if (in) k.store(p);
  } else {
    uint4 before;
    before.x = __shfl_up_sync(0xffffffffu, k.u.x, 1);
    before.y = __shfl_up_sync(0xffffffffu, k.u.y, 1);
    before.z = __shfl_up_sync(0xffffffffu, k.u.z, 1);
    before.w = __shfl_up_sync(0xffffffffu, k.u.w, 1);
    if (!in) return;
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u);
    const int at = threadIdx.x & (seg - 1);  // seg threads from a multiple of seg on
    const long long from = (long long)c * 16 - off, end = (long long)cols * es;
    // vector c holds the last `off` bytes of chunk c - 1 and the first ones of chunk c
    const bool mine = (off == 0 || at != 0) && from + 16 <= end;
    const bool next = off == 0 ? mine : at != seg - 1 && from + 32 <= end;
    if (mine)
      *reinterpret_cast<uint4*>(reinterpret_cast<uintptr_t>(p) - off) =
          off ? shift16<T>(before, k.u, 16u - off) : k.u;
    if (!mine || !next) {
      const uint32_t w[4] = {k.u.x, k.u.y, k.u.z, k.u.w};
      const int n = min(V, cols - c * V), head = V - (int)off / es;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (j < n && (j < head ? !mine : !next)) p[j] = element<T>(w, j);
    }
  }
}

// How blocks of 256 threads walk a matrix, four chunks a thread.  A warp's lanes stand in
// 2^lane_rows rows of consecutive chunks; its four passes are 2^pass_cols of them along the
// rows, the others down the matrix.  So long rows and short ones fill a warp, an aligned group
// of `least` lanes stays in one row and one pass, and places come without divisions but one by
// the pieces of a row.
constexpr int kPasses = 4;
struct Walk {
  long long rows;
  int chunks;       // of a row
  unsigned pieces;  // warps a row
  int lane_rows, pass_cols;
  long long blocks;
};
inline Walk walk_of(long long rows, int chunks, int least) {
  Walk w{rows, chunks, 1, 0, 0, 0};
  while ((32 >> w.lane_rows) / 2 >= least && (32 >> w.lane_rows) / 2 >= chunks) ++w.lane_rows;
  while ((1 << w.pass_cols) < kPasses && (32 << w.pass_cols) < chunks) ++w.pass_cols;
  w.pieces = (unsigned)ceil_div(chunks, 32 << w.pass_cols);
  w.blocks = ceil_div(ceil_div(rows, (long long)(kPasses >> w.pass_cols) << w.lane_rows) * w.pieces, 8);
  return w;
}
struct Places {
  long long row;
  int c, lanes, rows, mask, shift;
  __device__ __forceinline__ Places(const Walk& w, long long block) {
    const long long warp = block * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const long long line = w.pieces == 1 ? warp : warp / w.pieces;
    const int piece = (int)(warp - line * w.pieces);
    lanes = 32 >> w.lane_rows, rows = 1 << w.lane_rows;
    shift = w.pass_cols, mask = (1 << shift) - 1;
    row = line * ((kPasses >> shift) * rows) + lane / lanes;
    c = (piece << shift) * 32 + (lane & (lanes - 1));
  }
  __device__ __forceinline__ long long row_of(int u) const { return row + (u >> shift) * rows; }
  __device__ __forceinline__ int chunk_of(int u) const { return c + (u & mask) * 32; }
};

}  // namespace b2g
