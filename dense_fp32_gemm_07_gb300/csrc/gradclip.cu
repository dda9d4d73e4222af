// gradclip.cu -- the 2-norm of a list of tensors and clipping by it
// (b2g_grad_norm, b2g_clip_grad_norm in include/b2g_train.h).
//
// The tensors' addresses and lengths travel in the kernel's parameters, kTable
// of them per launch, so a call copies nothing to the device and can be
// captured.  Each tensor is cut into chunks of 2048 to 16384 elements; a block walks
// chunks b, b + grid, ... and leaves one FP32 sum of squares.  The clipping
// kernel adds those sums again in every block, in the same order (a few hundred
// floats from L2), which saves a launch, and walks the chunks backwards, so
// that it starts with what the first pass left in L2.
// Bound: bytes; one read for the norm, one read and one write for clipping: 537 M BF16
// elements in 49 tensors take 154 us (7.0 TB/s) and 361 us (5.9 TB/s).  Few elements: the
// latency of two launches (0.67 M FP32 elements in 17 tensors: 6.6 us).
#include "train_common.cuh"

namespace b2g {
namespace {

constexpr int kTable = 120;        // tensors per launch (kernel parameters stay under 4 KB)
constexpr int kThreads = 512;
// Elements of a chunk: 16384, or fewer (a power of two, 2048 at least) when that
// leaves SMs without one.
constexpr long long kMaxChunk = 16384, kMinChunk = 2048;

struct ClipTable {
  const void* in[kTable];
  void* out[kTable];
  long long n[kTable];
  unsigned first[kTable + 1];  // first chunk of each tensor; first[count]: all of them
  int count;
  int chunk;                   // elements of a chunk
  float* parts;                // sums of squares, one per block of every launch
  int part0, nparts;           // this launch's first, and the number of all
  float max_norm;
  float* norm;
};

// The tensor holding chunk c: the last one whose first chunk is at or below c.
__device__ __forceinline__ int tensor_of(const ClipTable& t, unsigned c) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= c)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Elements [0, head) of a chunk up to the first 16-byte boundary.
template <typename T>
__device__ __forceinline__ int head_of(const T* p, int n) {
  const int off = (int)((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
  const int head = off ? (int)(16 / sizeof(T)) - off : 0;
  return head < n ? head : n;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ ClipTable t) {
  constexpr int VEC = 16 / sizeof(T), U = 4;
  __shared__ float red[32];
  pdl_launch_dependents();
  pdl_wait();
  float sum = 0.f;
  for (unsigned c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const long long at = (long long)(c - t.first[i]) * t.chunk;
    const T* p = static_cast<const T*>(t.in[i]) + at;
    const int n = (int)(t.n[i] - at < t.chunk ? t.n[i] - at : t.chunk);
    const int head = head_of(p, n), vecs = (n - head) / VEC;
    const T* q = p + head;
    for (int v = threadIdx.x; v < vecs; v += kThreads * U) {
      Pack<T, VEC> k[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        k[u].zero();
        if (v + u * kThreads < vecs) k[u].load(q + (v + u * kThreads) * VEC);
      }
      // these squares first among themselves, so that few rounded additions
      // reach the long sum
      float s[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float f[VEC];
        k[u].get(f);
        s[u] = f[0] * f[0];
#pragma unroll
        for (int j = 1; j < VEC; ++j) s[u] = fmaf(f[j], f[j], s[u]);
      }
      sum += (s[0] + s[1]) + (s[2] + s[3]);
    }
    const int tail = head + vecs * VEC;
    int e = threadIdx.x < head ? threadIdx.x : tail + threadIdx.x - head;
    if (e < n) {  // at most 2 * (VEC - 1) loose elements, one a thread
      const float f = to_f32(p[e]);
      sum = fmaf(f, f, sum);
    }
  }
  sum = block_sum(sum, red, kThreads / 32);
  if (threadIdx.x == 0) t.parts[t.part0 + blockIdx.x] = sum;
}

// The norm from the blocks' sums; every block computes the same bits.
__device__ __forceinline__ float total_norm(const ClipTable& t, float* red) {
  float s = 0.f;
  for (int i = threadIdx.x; i < t.nparts; i += kThreads) s += t.parts[i];
  return sqrtf(block_sum(s, red, kThreads / 32));
}

__global__ void __launch_bounds__(kThreads) finish_kernel(const __grid_constant__ ClipTable t) {
  __shared__ float red[32];
  pdl_launch_dependents();
  pdl_wait();
  const float norm = total_norm(t, red);
  if (threadIdx.x == 0) *t.norm = norm;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) clip_kernel(const __grid_constant__ ClipTable t) {
  constexpr int VEC = 16 / sizeof(T), U = 4;
  __shared__ float red[32];
  pdl_launch_dependents();
  pdl_wait();
  const float norm = total_norm(t, red);
  if (blockIdx.x == 0 && t.part0 == 0 && threadIdx.x == 0) *t.norm = norm;
  const float ratio = t.max_norm / (norm + 1e-6f);
  const float coef = ratio > 1.f ? 1.f : ratio;  // a NaN norm stays NaN
  const unsigned all = t.first[t.count];
  for (unsigned k = blockIdx.x; k < all; k += gridDim.x) {
    const unsigned c = all - 1 - k;
    const int i = tensor_of(t, c);
    const long long at = (long long)(c - t.first[i]) * t.chunk;
    const T* p = static_cast<const T*>(t.in[i]) + at;
    T* o = static_cast<T*>(t.out[i]) + at;
    const int n = (int)(t.n[i] - at < t.chunk ? t.n[i] - at : t.chunk);
    if (((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15u) == 0) {
      const int head = head_of(p, n), vecs = (n - head) / VEC;
      for (int v = threadIdx.x; v < vecs; v += kThreads * U) {
        Pack<T, VEC> x[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (v + u * kThreads < vecs) x[u].load(p + head + (v + u * kThreads) * VEC);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (v + u * kThreads < vecs) {
            float f[VEC];
            x[u].get(f);
#pragma unroll
            for (int j = 0; j < VEC; ++j) f[j] *= coef;
            x[u].set(f);
            x[u].store(o + head + (v + u * kThreads) * VEC);
          }
        }
      }
      const int tail = head + vecs * VEC;
      const int e = threadIdx.x < head ? threadIdx.x : tail + threadIdx.x - head;
      if (e < n) o[e] = from_f32<T>(to_f32(p[e]) * coef);
    } else {
      for (int e = threadIdx.x; e < n; e += kThreads) o[e] = from_f32<T>(to_f32(p[e]) * coef);
    }
  }
}

// Four blocks of 512 threads an SM; one launch's blocks never outnumber its chunks.
int blocks_for(long long chunks, int sms) {
  const long long most = 4LL * sms;
  return (int)(chunks < most ? (chunks > 0 ? chunks : 1) : most);
}

int check(int dtype, int count, const void* const* tensors, const long long* numels) {
  if (!type_ok(dtype)) return B2G_ERR_INVALID_TYPE;
  if (count < 0) return B2G_ERR_INVALID_DIM;
  if (count > 0 && !numels) return B2G_ERR_NULL;
  for (int i = 0; i < count; ++i) {
    if (numels[i] < 0 || numels[i] > (1LL << 44)) return B2G_ERR_INVALID_DIM;
    if (tensors && numels[i] > 0 && !tensors[i]) return B2G_ERR_NULL;
  }
  return 0;
}

// The launches' tables one after another; fn(table, chunks of that launch).
template <typename Fn>
int for_each_table(int count, const void* const* in, void* const* out, const long long* n, int sms,
                   Fn fn) {
  long long total = 0;
  for (int i = 0; i < count; ++i) total += n[i];
  long long chunk = kMaxChunk;
  while (chunk > kMinChunk && total < chunk * 4 * sms) chunk /= 2;
  int part0 = 0;
  for (int i = 0; i < count || part0 == 0; i += kTable) {
    ClipTable t;
    t.count = 0;
    t.chunk = (int)chunk;
    long long chunks = 0;
    for (int j = i; j < count && t.count < kTable; ++j) {
      const int k = t.count;
      t.in[k] = in ? in[j] : nullptr, t.out[k] = out ? out[j] : nullptr, t.n[k] = n[j];
      t.first[k] = (unsigned)chunks;
      chunks += ceil_div(n[j], chunk);
      ++t.count;
      if (chunks > 0x7fffffffLL) return B2G_ERR_INVALID_DIM;
    }
    t.first[t.count] = (unsigned)chunks;
    t.part0 = part0;
    const int blocks = blocks_for(chunks, sms);
    const int rc = fn(t, blocks);
    if (rc) return rc;
    part0 += blocks;
  }
  return 0;
}

int all_parts(int count, const long long* n, int sms) {
  int parts = 0;
  const int rc = for_each_table(count, nullptr, nullptr, n, sms, [&](ClipTable&, int blocks) {
    parts += blocks;
    return 0;
  });
  return rc ? rc : parts;
}

int run_norm(int dtype, int count, const void* const* tensors, const long long* numels,
             float max_norm, void* const* outs, float* norm, void* workspace,
             size_t workspace_bytes, void* stream) {
  int rc = check(dtype, count, tensors, numels);
  if (rc) return rc;
  if (!norm || (count > 0 && !tensors)) return B2G_ERR_NULL;
  if (outs)
    for (int i = 0; i < count; ++i)
      if (numels[i] > 0 && !outs[i]) return B2G_ERR_NULL;
  TrainDevice d;
  rc = train_device(&d);
  if (rc) return rc;
  const int parts = all_parts(count, numels, d.sms);
  if (parts < 0) return parts;
  if (!workspace || !vec16(workspace) || workspace_bytes < (size_t)parts * sizeof(float))
    return B2G_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto fill = [&](ClipTable& t) {
    t.parts = static_cast<float*>(workspace);
    t.nparts = parts, t.max_norm = max_norm, t.norm = norm;
  };
  rc = for_each_table(count, tensors, nullptr, numels, d.sms, [&](ClipTable& t, int blocks) {
    fill(t);
    return launch_code(dtype == B2G_F32
                           ? launch_train(norm_kernel<float>, blocks, kThreads, 0, st, t)
                           : launch_train(norm_kernel<Bf16>, blocks, kThreads, 0, st, t));
  });
  if (rc) return rc;
  if (!outs) {
    ClipTable t;
    t.count = 0, t.chunk = 0, t.first[0] = 0, t.part0 = 0;
    fill(t);
    return launch_code(launch_train(finish_kernel, 1, kThreads, 0, st, t));
  }
  return for_each_table(count, tensors, outs, numels, d.sms, [&](ClipTable& t, int blocks) {
    fill(t);
    return launch_code(dtype == B2G_F32
                           ? launch_train(clip_kernel<float>, blocks, kThreads, 0, st, t)
                           : launch_train(clip_kernel<Bf16>, blocks, kThreads, 0, st, t));
  });
}

}  // namespace
}  // namespace b2g

using namespace b2g;

extern "C" {

int b2g_grad_norm(int dtype, int count, const void* const* tensors, const long long* numels,
                  float* norm, void* workspace, size_t workspace_bytes, void* stream) {
  return run_norm(dtype, count, tensors, numels, 0.f, nullptr, norm, workspace, workspace_bytes,
                  stream);
}

int b2g_clip_grad_norm(int dtype, int count, const void* const* tensors, const long long* numels,
                       float max_norm, void* const* outs, float* norm, void* workspace,
                       size_t workspace_bytes, void* stream) {
  if (!(max_norm >= 0.f)) return B2G_ERR_INVALID_DIM;
  if (count > 0 && !outs) return B2G_ERR_NULL;
  void* none = nullptr;
  return run_norm(dtype, count, tensors, numels, max_norm, outs ? outs : &none, norm, workspace,
                  workspace_bytes, stream);
}

int b2g_grad_norm_workspace_size(int dtype, int count, const long long* numels, size_t* bytes) {
  const int rc = check(dtype, count, nullptr, numels);
  if (rc) return rc;
  if (!bytes) return B2G_ERR_NULL;
  TrainDevice d;
  const int sms = train_device(&d) ? 152 : d.sms;  // without a device: GB300's count
  const int parts = all_parts(count, numels, sms);
  if (parts < 0) return parts;
  *bytes = (size_t)parts * sizeof(float);
  return 0;
}

}  // extern "C"
