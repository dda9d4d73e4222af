// embedding.cu -- embedding lookup and its gradient (b2g_embedding,
// b2g_embedding_backward in include/b2g_train.h).
//
// Forward: a gather, bound by bytes (each looked-up row read, each output row
// written): 32768 rows of 4096 BF16 take 54 us.
//
// Backward: dtable_v = scale * sum of dout_i over the tokens i with id v.  The
// tokens are first put in the order of their ids (a stable radix sort, so that
// equal ids keep their order and the sums their bits), then cut into windows of
// W consecutive sorted tokens:
//  1. emb_sort_kernel: one cluster sorts (id, token) pairs; the other blocks of
//     the same launch write the table's zeros meanwhile (that is most of the
//     traffic when the table is larger than the batch);
//  2. emb_window_kernel: each window adds the rows of each run of equal ids.  A
//     run that lies inside its window is final and goes to dtable; the first and
//     last run of a window may continue beyond it and go to FP32 partial rows;
//  3. emb_join_kernel: the block of the window in which a longer run begins adds
//     its partial rows in window order.
// Windows make the work even however often the most frequent token occurs.  The three
// launches follow one another: only the sort runs beside the clearing.
// 32768 tokens on 131072 rows of 4096 BF16: 260 us, of which the clearing (1 GB at 5.8 TB/s)
// takes 185, the windows 65 and the join 12; 4095 tokens on 50001 rows of 512 FP32: 27 us, 15
// for the table.
#include <atomic>

#include "tcgen05.cuh"
#include "train_common.cuh"

namespace b2g {
namespace {

__device__ __forceinline__ long long id_at(const void* ids, int bytes, long long i) {
  return bytes == 8 ? static_cast<const long long*>(ids)[i]
                    : (long long)static_cast<const int*>(ids)[i];
}

// Blocks of columns stand in the grid's y, and past its 65535 in z as well.
__device__ __forceinline__ int column_block() { return blockIdx.z * gridDim.y + blockIdx.y; }

// ------------------------------------------------------------------- forward

struct EmbFwd {
  long long tokens;
  int vocab, chunks;  // chunks = width / VEC
  const void* ids;
  int id_bytes;
  const void* table;
  long long ldt;
  float scale;
  void* out;
  long long ldo;
  unsigned int* status;
};

// blockDim.x threads per token, blockDim.y tokens per block; U chunks a thread
// (its loads are all in flight before the first store); column_block() covers wider
// rows.
template <typename T, int VEC, int U>
__global__ void __launch_bounds__(256) emb_fwd_kernel(const __grid_constant__ EmbFwd p) {
  pdl_launch_dependents();
  pdl_wait();
  const long long i = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  if (i >= p.tokens) return;
  const long long id = id_at(p.ids, p.id_bytes, i);
  const int c0 = column_block() * blockDim.x * U + threadIdx.x;
  T* o = static_cast<T*>(p.out) + i * p.ldo;
  const bool ok = id >= 0 && id < p.vocab;
  if (!ok && c0 == 0) atomicOr(p.status, kStatusIndex);
  const T* r = static_cast<const T*>(p.table) + (ok ? id : 0) * p.ldt;
  Pack<T, VEC> v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = c0 + u * blockDim.x;
    v[u].zero();
    if (ok && c < p.chunks) v[u].load(r + c * VEC);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = c0 + u * blockDim.x;
    if (c < p.chunks) {
      float f[VEC];
      v[u].get(f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[j] = ok ? f[j] * p.scale : __int_as_float(0x7fc00000);
      v[u].set(f);
      v[u].store(o + c * VEC);
    }
  }
}

// Rows off the 16-byte boundaries, in 4-byte words of the output row (BF16: two
// elements, from a word of the table or from two halves, with an element alone at either
// end of a row): U words a thread in flight, the row's threads striding over it.
// 20000 x 1111: BF16 18.8 us (4.7 TB/s), element by element 47; FP32 25 and 49.
template <typename T, int U>
__global__ void __launch_bounds__(256) emb_fwd_words_kernel(const __grid_constant__ EmbFwd p) {
  constexpr int E = 4 / (int)sizeof(T);  // elements a word; chunks counts elements
  pdl_launch_dependents();
  pdl_wait();
  const long long i = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  if (i >= p.tokens) return;
  const long long id = id_at(p.ids, p.id_bytes, i);
  T* o = static_cast<T*>(p.out) + i * p.ldo;
  const bool ok = id >= 0 && id < p.vocab;
  const T* r = static_cast<const T*>(p.table) + (ok ? id : 0) * p.ldt;
  const float scale = ok ? p.scale : __int_as_float(0x7fc00000);
  const int head = E == 2 ? (int)(reinterpret_cast<uintptr_t>(o) >> 1 & 1) : 0;
  const int words = (p.chunks - head) / E;
  if (threadIdx.x == 0) {
    if (!ok) atomicOr(p.status, kStatusIndex);
    const int last = p.chunks - 1;
    if (head) o[0] = from_f32<T>((ok ? to_f32(r[0]) : 0.f) * scale);
    if (E == 2 && head + 2 * words <= last)
      o[last] = from_f32<T>((ok ? to_f32(r[last]) : 0.f) * scale);
  }
  const T* src = r + head;
  uint32_t* dst = reinterpret_cast<uint32_t*>(o + head);
  const bool whole = E == 1 || (reinterpret_cast<uintptr_t>(src) & 3) == 0;
  for (int c0 = threadIdx.x; c0 < words; c0 += U * blockDim.x) {
    uint32_t v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * blockDim.x;
      v[u] = 0;
      if (ok && c < words) {
        if (whole) {
          v[u] = reinterpret_cast<const uint32_t*>(src)[c];
        } else {
          const unsigned short* h = reinterpret_cast<const unsigned short*>(src) + 2 * c;
          v[u] = h[0] | (uint32_t)h[1] << 16;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * blockDim.x;
      if (c < words) {
        if constexpr (E == 1) {
          v[u] = __float_as_uint(__uint_as_float(v[u]) * scale);
        } else {
          const __nv_bfloat162 h = __floats2bfloat162_rn(
              __uint_as_float(v[u] << 16) * scale, __uint_as_float(v[u] & 0xFFFF0000u) * scale);
          v[u] = *reinterpret_cast<const uint32_t*>(&h);
        }
        dst[c] = v[u];
      }
    }
  }
}

// ---------------------------------------------------------------------- sort

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortCtas = 8;              // most blocks of the sorting cluster (portable limit)
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;
constexpr int kSortSmem = (kSortWarps + 1) * kDigits * 4;

struct EmbSort {
  int tokens, vocab, passes, bits;  // bits a pass, at most kDigitBits
  const void* ids;
  int id_bytes;
  long long padding;
  unsigned* key[2];   // tokens ids each, unsorted / sorted by turns
  int* pos[2];        // the token each came from
  unsigned* totals;   // [blocks of the cluster][kDigits]
  unsigned int* status;
  // the table to clear; rows == 0: nothing to clear
  unsigned char* table;
  long long rows, row_bytes, ld_bytes;
};

// Zeros over the rows of the table, by blocks `b` of `nb`.
__device__ __noinline__ void clear_rows(const EmbSort& p, long long b, long long nb) {
  const bool flat = p.row_bytes == p.ld_bytes;
  const long long rows = flat ? 1 : p.rows, bytes = flat ? p.rows * p.row_bytes : p.row_bytes;
  if (flat) {  // one run of bytes: 16-byte stores between its ragged ends
    unsigned char* t = p.table;
    const long long head = (16 - (long long)(reinterpret_cast<uintptr_t>(t) & 15)) & 15;
    const long long h = head < bytes ? head : bytes, vecs = (bytes - h) / 16;
    uint4* v = reinterpret_cast<uint4*>(t + h);
    const long long step = nb * kSortThreads;
    long long i = b * kSortThreads + threadIdx.x;
    for (; i + 3 * step < vecs; i += 4 * step) {
#pragma unroll
      for (int u = 0; u < 4; ++u) v[i + u * step] = make_uint4(0, 0, 0, 0);
    }
    for (; i < vecs; i += step) v[i] = make_uint4(0, 0, 0, 0);
    if (b == 0) {
      for (long long j = threadIdx.x; j < h; j += kSortThreads) t[j] = 0;
      for (long long j = h + vecs * 16 + threadIdx.x; j < bytes; j += kSortThreads) t[j] = 0;
    }
  } else {
    for (long long r = b; r < rows; r += nb) {
      unsigned char* t = p.table + r * p.ld_bytes;
      if (((reinterpret_cast<uintptr_t>(t) | (uintptr_t)bytes) & 15) == 0) {
        for (long long i = threadIdx.x; i < bytes / 16; i += kSortThreads)
          reinterpret_cast<uint4*>(t)[i] = make_uint4(0, 0, 0, 0);
      } else {  // every element type has an even size
        for (long long i = threadIdx.x; i < bytes / 2; i += kSortThreads)
          reinterpret_cast<unsigned short*>(t)[i] = 0;
      }
    }
  }
}

constexpr int kRounds = 4;

// The keys of tokens i, i + 32, ... (kRounds of them, below hi): their ids, or
// `vocab` for one that takes part in no sum.
__device__ __forceinline__ void load_ids(const EmbSort& p, int i, int hi, unsigned (&k)[kRounds]) {
  long long id[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r)
    id[r] = i + 32 * r < hi ? id_at(p.ids, p.id_bytes, i + 32 * r) : 0;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const bool in = id[r] >= 0 && id[r] < p.vocab, pad = p.padding >= 0 && id[r] == p.padding;
    if (!in && !pad && i + 32 * r < hi) atomicOr(p.status, kStatusIndex);
    k[r] = in && !pad ? (unsigned)id[r] : (unsigned)p.vocab;
  }
}

// The first cluster sorts, the other ones clear the table.  The sort: `passes`
// stable passes over `bits` bits each (at most kDigitBits), lowest first.  Warp w of the cluster
// owns a contiguous range of the input.  It counts its digits; the block adds
// the counts up digit by digit and shares its totals with the cluster, so that
// each block knows where its pairs of a digit begin; and each warp then places its
// pairs in order, 32 at a time: a pair's place is its digit's next one plus the
// number of lower lanes with the same digit.  An id that takes part in no sum
// (padding, out of range) sorts last as `vocab`.  Bound: latency, a few
// microseconds a pass, behind the clearing of a table that is much larger than the
// batch.
__global__ void __launch_bounds__(kSortThreads)
    emb_sort_kernel(const __grid_constant__ EmbSort p, int ctas) {
  extern __shared__ unsigned counts[];  // [kSortWarps][kDigits], then [kDigits] first places
  __shared__ unsigned scan[kDigits / 32];
  pdl_launch_dependents();
  pdl_wait();
  if ((int)blockIdx.x >= ctas) {
    clear_rows(p, (long long)blockIdx.x - ctas, (long long)gridDim.x - ctas);
    return;
  }
  const int digits = 1 << p.bits;
  const unsigned mask = (unsigned)digits - 1u;
  unsigned* first = counts + kSortWarps * digits;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;
  const int W = ctas * kSortWarps;
  const int gw = cta * kSortWarps + warp;
  // ranges are whole multiples of 32 so that every warp runs full rounds
  const int per = ((p.tokens + W - 1) / W + 31) / 32 * 32;
  const long long lo64 = (long long)gw * per;
  const int lo = lo64 < p.tokens ? (int)lo64 : p.tokens;
  const int hi = lo + per < p.tokens ? lo + per : p.tokens;
  const unsigned below = (1u << lane) - 1u;

  unsigned* cnt = counts + warp * digits;
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.bits, src = pass & 1;
    // (the lists are read past L1: the other blocks of the cluster write them too)
    const unsigned* key = src ? p.key[1] : p.key[0];
    const int* pos = src ? p.pos[1] : p.pos[0];
    unsigned* key_out = src ? p.key[0] : p.key[1];
    int* pos_out = src ? p.pos[0] : p.pos[1];
    for (int d = lane; d < digits; d += 32) cnt[d] = 0;
    __syncwarp();
    // kRounds rounds of 32 pairs at a time, their loads together
    unsigned k[kRounds];
    for (int i0 = lo; i0 < hi; i0 += 32 * kRounds) {
      if (pass == 0) {
        load_ids(p, i0 + lane, hi, k);
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
          if (i0 + 32 * r + lane < hi) p.key[0][i0 + 32 * r + lane] = k[r];
      } else {
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
          k[r] = i0 + 32 * r + lane < hi ? __ldcg(key + i0 + 32 * r + lane) : 0u;
      }
#pragma unroll
      for (int r = 0; r < kRounds; ++r)
        if (i0 + 32 * r + lane < hi) atomicAdd(&cnt[(k[r] >> shift) & mask], 1u);
    }
    __syncthreads();
    // Two neighbouring threads per digit, 16 warps' counts each: counts become
    // offsets in the block.
    const int digit = threadIdx.x >> 1, half = threadIdx.x & 1;
    unsigned* col = counts + half * (kSortWarps / 2) * digits + digit;
    unsigned n[kSortWarps / 2], mine = 0;
    if (digit < digits) {
#pragma unroll
      for (int w = 0; w < kSortWarps / 2; ++w) mine += n[w] = col[w * digits];
    }
    const unsigned other = __shfl_xor_sync(0xffffffffu, mine, 1);
    if (!half && digit < digits) {
      if (ctas > 1)
        p.totals[cta * kDigits + digit] = mine + other;
      else
        first[digit] = mine + other;
    }
    if (ctas > 1)
      cluster_sync();
    else
      __syncthreads();
    // where the digit's pairs begin: lower digits anywhere, this digit in earlier blocks
    if (threadIdx.x < kDigits) {
      unsigned all = 0, earlier = 0;
      if ((int)threadIdx.x < digits) {
        if (ctas == 1) all = first[threadIdx.x];
        for (int c = 0; c < ctas && ctas > 1; ++c) {
          const unsigned t = __ldcg(p.totals + c * kDigits + threadIdx.x);
          all += t;
          earlier += c < cta ? t : 0u;
        }
      }
      unsigned incl = all;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      if (lane == 31) scan[warp] = incl;
      asm volatile("bar.sync 1, %0;" ::"n"(kDigits) : "memory");
      unsigned lower = 0;
#pragma unroll
      for (int w = 0; w < kDigits / 32; ++w) lower += w < warp ? scan[w] : 0u;
      if ((int)threadIdx.x < digits) first[threadIdx.x] = lower + incl - all + earlier;
    }
    __syncthreads();
    if (digit < digits) {
      unsigned at = first[digit] + (half ? other : 0u);
#pragma unroll
      for (int w = 0; w < kSortWarps / 2; ++w) {
        col[w * digits] = at;
        at += n[w];
      }
    }
    __syncthreads();
    const bool once = hi - lo <= 32 * kRounds;  // the keys are still in registers
    for (int i0 = lo; i0 < hi; i0 += 32 * kRounds) {
      int from[kRounds];
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        const int i = i0 + 32 * r + lane;
        if (!once) k[r] = i < hi ? __ldcg(key + i) : 0u;
        from[r] = pass == 0 ? i : i < hi ? __ldcg(pos + i) : 0;
      }
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        const bool in = i0 + 32 * r + lane < hi;
        const unsigned d = (k[r] >> shift) & mask;
        unsigned same = __ballot_sync(0xffffffffu, in);
#pragma unroll
        for (int b = 0; b < kDigitBits; ++b) {
          if (b < p.bits) {
            const unsigned one = __ballot_sync(0xffffffffu, (d >> b) & 1u);
            same &= (d >> b) & 1u ? one : ~one;
          }
        }
        unsigned to = 0;
        if (in) to = cnt[d] + __popc(same & below);
        __syncwarp();
        if (in) {
          if ((same & below) == 0) cnt[d] += __popc(same);
          key_out[to] = k[r], pos_out[to] = from[r];
        }
        __syncwarp();
      }
    }
    if (ctas > 1)
      cluster_sync();
    else
      __syncthreads();
  }
}

// ------------------------------------------------------------------- windows

struct EmbSum {
  int tokens, vocab, width, chunks, window;
  const unsigned* key;
  const int* pos;
  const void* dout;
  long long ldd;
  float scale;
  int accumulate;
  void* dtable;
  long long ldt;
  float* part;  // [windows][2][width]: the window's first run (0), its last run (1)
};

// VEC FP32 partial sums to a partial row.
template <int VEC>
__device__ __forceinline__ void put_part(float* q, const float (&a)[VEC]) {
  if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int j = 0; j < VEC; j += 4)
      *reinterpret_cast<float4*>(q + j) = make_float4(a[j], a[j + 1], a[j + 2], a[j + 3]);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) q[j] = a[j];
  }
}
// A sum of one run's columns, scaled and stored as one final row chunk; `old` is
// what was there, for accumulate.
template <typename T, int VEC>
__device__ __forceinline__ void put_row(const EmbSum& p, unsigned row, int c, const float (&a)[VEC],
                                        const Pack<T, VEC>& old) {
  float f[VEC];
  Pack<T, VEC> k;
  if (p.accumulate) {
    old.get(f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = fmaf(a[j], p.scale, f[j]);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = a[j] * p.scale;
  }
  k.set(f);
  k.store(static_cast<T*>(p.dtable) + (long long)row * p.ldt + c * VEC);
}

constexpr int kMaxWindow = 128;

// blockDim.x threads share a window's columns (one chunk each), blockDim.y
// windows per block; column_block() covers wider rows.  The window's ids and places are
// fetched into shared memory first, so that only the rows themselves are waited
// for, U at a time.  Runs that begin before the window or continue after it go
// to the window's partial rows.
template <typename T, int VEC, int U, bool ACC>
__global__ void __launch_bounds__(256) emb_window_kernel(const __grid_constant__ EmbSum p) {
  extern __shared__ unsigned keys[];  // blockDim.y windows' ids, then their places
  int* places = reinterpret_cast<int*>(keys + blockDim.y * p.window);
  pdl_launch_dependents();
  pdl_wait();
  const long long first_token = (long long)blockIdx.x * blockDim.y * p.window;
  const int tid = threadIdx.y * blockDim.x + threadIdx.x;
  for (int i = tid; i < (int)blockDim.y * p.window; i += 256) {
    const bool in = first_token + i < p.tokens;
    keys[i] = in ? p.key[first_token + i] : 0u;
    places[i] = in ? p.pos[first_token + i] : 0;
  }
  const int w = blockIdx.x * blockDim.y + threadIdx.y;
  const int c = column_block() * blockDim.x + threadIdx.x;
  const long long begin = (long long)w * p.window;
  const bool mine = begin < p.tokens && c < p.chunks;
  const int b = (int)begin, e = b + p.window < p.tokens ? b + p.window : p.tokens;
  const unsigned before = mine && b > 0 ? p.key[b - 1] : ~0u;  // no id is ~0
  const unsigned after = mine && e < p.tokens ? p.key[e] : ~0u;
  __syncthreads();
  if (!mine) return;
  const unsigned* key = keys + threadIdx.y * p.window - b;
  const int* pos = places + threadIdx.y * p.window - b;
  const unsigned vocab = (unsigned)p.vocab, key_b = key[b];
  const T* dout = static_cast<const T*>(p.dout) + c * VEC;
  const T* table = static_cast<const T*>(p.dtable) + c * VEC;
  if (key_b >= vocab) return;  // nothing but padding
  const bool from_before = before == key_b;
  float* part = p.part + (size_t)w * 2 * p.width + c * VEC;
  // The rows of U tokens at a time, and for accumulate the old values of the runs
  // that end among them.
  Pack<T, VEC> v[U], old[U], none, held;  // held: of the last token before these
  none.zero(), held.zero();
  float a[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) a[j] = 0.f;
  unsigned run = key_b;
  bool first = true;
  auto flush = [&](bool last, const Pack<T, VEC>& was) {
    if (run < vocab) {
      const bool head = first && from_before, tail = last && run == after;
      if (head || tail)
        put_part<VEC>(head ? part : part + p.width, a);
      else
        put_row<T, VEC>(p, run, c, a, was);
    }
  };
  for (int i0 = b; i0 < e; i0 += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = min(i0 + u, e - 1);
      v[u].load(dout + (long long)pos[i] * p.ldd);
      if (ACC) {  // what the run ending at i adds to
        old[u].zero();
        if (i < e && key[i] < vocab && (i + 1 == e || key[i + 1] != key[i]))
          old[u].load(table + (long long)key[i] * p.ldt);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const unsigned k = i0 + u < e ? key[i0 + u] : run;
      if (k != run) {
        flush(false, ACC ? (u ? old[u - 1] : held) : none);
        first = false, run = k;
#pragma unroll
        for (int j = 0; j < VEC; ++j) a[j] = 0.f;
      }
      float f[VEC];
      v[u].get(f);
      const bool in = i0 + u < e;
#pragma unroll
      for (int j = 0; j < VEC; ++j) a[j] = in ? a[j] + f[j] : a[j];
      if (ACC && i0 + u + 1 == e) held = old[u];
    }
    if (ACC && i0 + U < e) held = old[U - 1];
  }
  flush(true, ACC ? held : none);
}

// The run that begins in window w and continues past it: its last partial row,
// then the first partial rows of the windows after it up to where the run ends.  Bound:
// latency, of the most frequent token's windows: one column a thread and 16 windows at a
// time, with whether they begin with the run and their rows fetched together (past the
// run's end for nothing) and without branches, which would wait for each before the next
// one (30000 tokens of 129 columns, 2000 of them alike: 9 us, 24 in two steps of eight).
template <typename T>
__global__ void __launch_bounds__(256) emb_join_kernel(const __grid_constant__ EmbSum p) {
  pdl_launch_dependents();
  pdl_wait();
  const int w = blockIdx.x * blockDim.y + threadIdx.y;
  const int c = column_block() * blockDim.x + threadIdx.x;
  const long long begin = (long long)w * p.window, end = begin + p.window;
  if (end >= p.tokens || c >= p.width) return;
  const unsigned run = p.key[end - 1], next = p.key[end];
  const unsigned first = p.key[begin], before = begin > 0 ? p.key[begin - 1] : ~0u;
  if (run >= (unsigned)p.vocab || next != run) return;  // it ends here
  if (first == run && before == run) return;            // it began in an earlier window
  Pack<T, 1> old;
  old.zero();
  if (p.accumulate) old.load(static_cast<const T*>(p.dtable) + (long long)run * p.ldt + c);
  float a[1] = {p.part[((size_t)w * 2 + 1) * p.width + c]};
  constexpr int U = 16;
  const int windows = (p.tokens + p.window - 1) / p.window;
  for (int k = w + 1;; k += U) {
    unsigned key[U];
    float f[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = min(k + u, windows - 1);
      key[u] = p.key[(long long)at * p.window];
      f[u] = p.part[(size_t)at * 2 * p.width + c];
    }
    bool on = true;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      on = on && k + u < windows && key[u] == run;
      a[0] = on ? a[0] + f[u] : a[0];
    }
    if (!on) break;
  }
  put_row<T, 1>(p, run, c, a, old);
}

// ----------------------------------------------------------------- host side

constexpr long long kMaxTokens = 1LL << 30;

int check(int dtype, long long tokens, int vocab, int width) {
  if (!type_ok(dtype)) return B2G_ERR_INVALID_TYPE;
  if (tokens < 0 || vocab < 0 || width < 0 || tokens > kMaxTokens || vocab > kMaxLength ||
      width > kMaxLength)
    return B2G_ERR_INVALID_DIM;
  return 0;
}

bool ld_ok(long long ld, int width) { return ld >= (width > 1 ? width : 1); }

int pow2_at_least(int n, int lo, int hi) {
  int t = lo;
  while (t < n && t < hi) t *= 2;
  return t;
}

// `rows` blocks times `columns` blocks.  z is as small as possible and y even over it, so
// that at most z blocks have no column (fewer than 2^16 threads: their column numbers stay
// below 2^31).
dim3 grid_of(long long rows, long long columns) {
  const long long z = ceil_div(columns, 65535);
  return dim3((unsigned)rows, (unsigned)ceil_div(columns, z), (unsigned)z);
}

template <typename T, int VEC>
cudaError_t fwd_launch(EmbFwd p, int width, int sms, cudaStream_t st) {
  p.chunks = width / VEC;
  // Few tokens: one chunk a thread, so that more SMs share the rows.
  const bool many = p.tokens * p.chunks >= 4LL * 2048 * sms;
  if constexpr (VEC == 1) {
    if (many) {
      const int words = width * (int)sizeof(T) / 4, tx = pow2_at_least(words / 16, 8, 256);
      const int ty = 256 / tx;
      return launch_train(emb_fwd_words_kernel<T, 4>, dim3((unsigned)ceil_div(p.tokens, ty)),
                          dim3(tx, ty), 0, st, p);
    }
  }
  const int u = many ? 4 : 1;
  const int tx = pow2_at_least((int)ceil_div(p.chunks, u), 8, 256), ty = 256 / tx;
  const dim3 grid = grid_of(ceil_div(p.tokens, ty), ceil_div(p.chunks, tx * u));
  if (many) return launch_train(emb_fwd_kernel<T, VEC, 4>, grid, dim3(tx, ty), 0, st, p);
  return launch_train(emb_fwd_kernel<T, VEC, 1>, grid, dim3(tx, ty), 0, st, p);
}

// Sorted tokens per window: enough windows (times column blocks) to fill the
// GPU about four times over, 16 to 128 tokens each.  (Shorter ones for narrower rows
// lose in the join what the window kernel gains: 14 us for 9 and 7 for 14 at 30000 x 128.)
int window_of(long long tokens, int width) {
  const long long col_blocks = ceil_div(width, 1024);
  int w = 16;
  while (w < kMaxWindow && ceil_div(tokens, w) * col_blocks > 4 * 152 * 2) w *= 2;
  return w;
}

struct BwdSizes {
  size_t key[2], pos[2], totals, part, total;
};

BwdSizes bwd_sizes(long long tokens, int width) {
  BwdSizes s;
  size_t at = 0;
  const size_t list = round_up((size_t)tokens * 4, 256);
  for (int i = 0; i < 2; ++i) s.key[i] = at, at += list;
  for (int i = 0; i < 2; ++i) s.pos[i] = at, at += list;
  s.totals = at, at += (size_t)kDigits * kSortCtas * 4;
  s.part = at;
  at += (size_t)ceil_div(tokens, window_of(tokens, width)) * 2 * width * sizeof(float);
  s.total = at;
  return s;
}

// One cluster sorts, with a block per 4096 tokens (a power of two, at most
// kSortCtas); the clearing blocks, in clusters of the same size, fill the GPU twice
// over.
cudaError_t launch_sort(const EmbSort& q, long long tokens, const TrainDevice& d, cudaStream_t st) {
  static std::atomic<int> configured[64];
  if (d.dev < 0 || d.dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[d.dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(
        emb_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortSmem);
    if (e != cudaSuccess) return e;
    configured[d.dev].store(1, std::memory_order_release);
  }
  int ctas = 1;
  while (ctas < kSortCtas && ctas * 4096LL < tokens) ctas *= 2;
  const long long bytes = q.rows * q.row_bytes;
  const long long want = ceil_div(bytes, 16LL * kSortThreads), most = 2LL * d.sms - ctas;
  const long long clear = (want < most ? want : most) / ctas * ctas;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ctas + (bytes && clear < ctas ? ctas : clear)));
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = kSortSmem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  EmbSort p = q;
  void* args[] = {&p, &ctas};
  return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(&emb_sort_kernel), args);
}

template <typename T, int VEC>
cudaError_t sum_launch(EmbSum p, cudaStream_t st) {
  p.chunks = p.width / VEC;
  const int tx = pow2_at_least(p.chunks, 8, 256), ty = 256 / tx;
  const long long windows = ceil_div(p.tokens, p.window);
  const dim3 grid = grid_of(ceil_div(windows, ty), ceil_div(p.chunks, tx));
  // Eight rows in flight a thread in short windows, where few threads run (4095 x 512
  // FP32: 9 us with four, 7 with eight); four in long ones, where eight cost the
  // occupancy that hides their latency (32768 x 4096 BF16: 66 us with four, 86 with
  // eight).
  const size_t smem = (size_t)ty * p.window * 8;
  const auto kern = p.window <= 16 ? (p.accumulate ? emb_window_kernel<T, VEC, 8, true>
                                                   : emb_window_kernel<T, VEC, 8, false>)
                                   : (p.accumulate ? emb_window_kernel<T, VEC, 4, true>
                                                   : emb_window_kernel<T, VEC, 4, false>);
  cudaError_t e = launch_train(kern, grid, dim3(tx, ty), smem, st, p);
  if (e == cudaSuccess && windows > 1) {
    const int jx = pow2_at_least(p.width, 8, 256), jy = 256 / jx;
    e = launch_train(emb_join_kernel<T>,
                     grid_of(ceil_div(windows, jy), ceil_div(p.width, jx)), dim3(jx, jy), 0, st, p);
  }
  return e;
}

}  // namespace
}  // namespace b2g

using namespace b2g;

extern "C" {

int b2g_embedding(int dtype, long long tokens, int vocab, int width, const void* ids, int id_bytes,
                  const void* table, long long ldt, float scale, void* out, long long ldo,
                  void* stream) {
  int rc = check(dtype, tokens, vocab, width);
  if (rc) return rc;
  if (id_bytes != 8 && id_bytes != 4) return B2G_ERR_INVALID_TYPE;
  if (!ld_ok(ldt, width) || !ld_ok(ldo, width)) return B2G_ERR_INVALID_LD;
  if (tokens == 0 || width == 0) return 0;
  if (!ids || !out || (vocab > 0 && !table)) return B2G_ERR_NULL;
  TrainDevice d;
  rc = train_device(&d);
  if (rc) return rc;
  EmbFwd p{tokens, vocab, 0, ids, id_bytes, table, ldt, scale, out, ldo, d.status};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool v = vec16(table) && vec16(out) && vec16_ld(ldt, dtype) && vec16_ld(ldo, dtype) &&
                 vec16_ld(width, dtype);
  if (dtype == B2G_F32)
    return launch_code(v ? fwd_launch<float, 4>(p, width, d.sms, st)
                         : fwd_launch<float, 1>(p, width, d.sms, st));
  return launch_code(v ? fwd_launch<Bf16, 8>(p, width, d.sms, st)
                       : fwd_launch<Bf16, 1>(p, width, d.sms, st));
}

int b2g_embedding_backward_workspace_size(int dtype, long long tokens, int vocab, int width,
                                          size_t* bytes) {
  const int rc = check(dtype, tokens, vocab, width);
  if (rc) return rc;
  if (!bytes) return B2G_ERR_NULL;
  *bytes = tokens && vocab && width ? bwd_sizes(tokens, width).total : 0;
  return 0;
}

int b2g_embedding_backward(int dtype, long long tokens, int vocab, int width, const void* ids,
                           int id_bytes, const void* dout, long long ldd, float scale,
                           long long padding, int accumulate, void* dtable, long long ldt,
                           void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check(dtype, tokens, vocab, width);
  if (rc) return rc;
  if (id_bytes != 8 && id_bytes != 4) return B2G_ERR_INVALID_TYPE;
  if (!ld_ok(ldd, width) || !ld_ok(ldt, width)) return B2G_ERR_INVALID_LD;
  if (vocab == 0 || width == 0 || (tokens == 0 && accumulate)) return 0;
  if (!dtable || (tokens > 0 && (!ids || !dout))) return B2G_ERR_NULL;
  TrainDevice d;
  rc = train_device(&d);
  if (rc) return rc;
  const long long es = (long long)type_size(dtype);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (tokens == 0)
    return cudaMemset2DAsync(dtable, ldt * es, 0, width * es, vocab, st) == cudaSuccess
               ? 0
               : B2G_ERR_CUDA;
  const BwdSizes s = bwd_sizes(tokens, width);
  if (!workspace || !vec16(workspace) || workspace_bytes < s.total) return B2G_ERR_WORKSPACE;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  EmbSort q;
  q.tokens = (int)tokens, q.vocab = vocab;
  int bits = 1;  // the keys run from 0 to vocab, which stands for "in no sum"
  while (bits < 32 && (unsigned)vocab >> bits) ++bits;
  q.passes = (bits + kDigitBits - 1) / kDigitBits;
  q.bits = (bits + q.passes - 1) / q.passes;
  q.ids = ids, q.id_bytes = id_bytes, q.padding = padding;
  for (int i = 0; i < 2; ++i) {
    q.key[i] = reinterpret_cast<unsigned*>(ws + s.key[i]);
    q.pos[i] = reinterpret_cast<int*>(ws + s.pos[i]);
  }
  q.totals = reinterpret_cast<unsigned*>(ws + s.totals);
  q.status = d.status;
  q.table = static_cast<unsigned char*>(dtable);
  q.rows = accumulate ? 0 : vocab;
  q.row_bytes = width * es, q.ld_bytes = vocab > 1 ? ldt * es : width * es;
  if (launch_sort(q, tokens, d, st) != cudaSuccess) return B2G_ERR_LAUNCH;
  const int sorted = q.passes & 1;
  EmbSum p{(int)tokens, vocab, width, 0, window_of(tokens, width), q.key[sorted], q.pos[sorted],
           dout, ldd, scale, accumulate != 0, dtable, ldt,
           reinterpret_cast<float*>(ws + s.part)};
  const bool v = vec16(dout) && vec16(dtable) && vec16_ld(ldd, dtype) && vec16_ld(ldt, dtype) &&
                 vec16_ld(width, dtype);
  if (dtype == B2G_F32)
    return launch_code(v ? sum_launch<float, 4>(p, st) : sum_launch<float, 1>(p, st));
  return launch_code(v ? sum_launch<Bf16, 8>(p, st) : sum_launch<Bf16, 1>(p, st));
}

}  // extern "C"
