// train_common.cuh -- what the training-step operators (include/b2g_train.h)
// share: element types as FP32 values in 16-byte vectors or one by one, block
// sums, the library's device state, and launch helpers.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/b2g_train.h"
#include "ptx.cuh"

namespace b2g {

// Status-word flag of an id or target outside its table (see b2g_status).
constexpr unsigned int kStatusIndex = 1u << 16;

// The current device as host.cu knows it: SM count, status word, wait limit.
struct TrainDevice {
  int dev, sms;
  unsigned int* status;
  unsigned long long wait_limit_ns;
  int debug_stop;
};
// Row lengths, classes and tokens of a product: a column index plus what a block strides
// over stays below 2^31.
constexpr int kMaxLength = 0x7fff0000;
int train_device(TrainDevice* out);  // 0 or a B2G_ERR_* code (host.cu)

using Bf16 = __nv_bfloat16;

// Two FP32 values in a 64-bit register pair, for the packed FP32 instructions
// (each lane rounded like the scalar one).
using F2 = unsigned long long;
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f2_split(F2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ float f2_sum(F2 v) {
  float a, b;
  f2_split(v, a, b);
  return a + b;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(Bf16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ Bf16 from_f32<Bf16>(float x) {
  return __float2bfloat16_rn(x);
}

// VEC consecutive elements as loaded: one element (VEC == 1) or 16 bytes.
template <typename T, int VEC>
struct Pack {
  static_assert(VEC * sizeof(T) == 16, "a pack is one element or 16 bytes");
  uint4 u;
  __device__ __forceinline__ void load(const T* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<uint4*>(p) = u; }
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&f)[VEC]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // bfloat16 is the upper half of a binary32
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  }
  __device__ __forceinline__ void get2(F2 (&f)[VEC / 2]) const {
    float g[VEC];
    get(g);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) f[i] = f2(g[2 * i], g[2 * i + 1]);
  }
  __device__ __forceinline__ void set2(const F2 (&f)[VEC / 2]) {
    float g[VEC];
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) f2_split(f[i], g[2 * i], g[2 * i + 1]);
    set(g);
  }
  __device__ __forceinline__ void set(const float (&f)[VEC]) {
    uint32_t w[4];
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(f[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    u = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <typename T>
struct Pack<T, 1> {
  T u;
  __device__ __forceinline__ void load(const T* p) { u = *p; }
  __device__ __forceinline__ void store(T* p) const { *p = u; }
  __device__ __forceinline__ void zero() { u = from_f32<T>(0.f); }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = to_f32(u); }
  __device__ __forceinline__ void set(const float (&f)[1]) { u = from_f32<T>(f[0]); }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum of v over the `warps` warps of a block (every thread gets it).  `red`
// holds 32 floats; a second call must use another buffer unless a barrier
// stands between the calls.
__device__ __forceinline__ float block_sum(float v, float* red, int warps) {
  v = warp_sum(v);
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return warp_sum(lane < warps ? red[lane] : 0.f);
}

// The same for two sums at once; `red` holds 64 floats.
__device__ __forceinline__ float2 block_sum2(float a, float b, float* red, int warps) {
  a = warp_sum(a), b = warp_sum(b);
  if (warps == 1) return make_float2(a, b);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a, red[32 + (threadIdx.x >> 5)] = b;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return make_float2(warp_sum(lane < warps ? red[lane] : 0.f),
                     warp_sum(lane < warps ? red[32 + lane] : 0.f));
}

// `bytes` (a multiple of 16) from global to shared memory, both 16-byte aligned;
// completion is counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// ------------------------------------------------------------------ host side

inline size_t type_size(int dtype) { return dtype == B2G_F32 ? 4 : 2; }
inline bool type_ok(int dtype) { return dtype == B2G_F32 || dtype == B2G_BF16; }
inline bool vec16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// A row stride (elements) that keeps rows on 16-byte boundaries.
inline bool vec16_ld(long long ld, int dtype) { return ld * (long long)type_size(dtype) % 16 == 0; }
inline size_t round_up(size_t v, size_t to) { return (v + to - 1) / to * to; }
inline long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

inline int launch_code(cudaError_t e) { return e == cudaSuccess ? 0 : B2G_ERR_LAUNCH; }

// Launch kern(args...) with programmatic dependent launch; the arguments must
// have the kernel's own parameter types.
template <typename... P, typename... A>
cudaError_t launch_train(void (*kern)(P...), dim3 grid, dim3 block, size_t smem,
                         cudaStream_t stream, A... args) {
  static_assert(sizeof...(P) == sizeof...(A), "one argument per kernel parameter");
  return [&](P... typed) {
    void* ptrs[] = {const_cast<void*>(static_cast<const void*>(&typed))...};
    return launch_pdl(reinterpret_cast<const void*>(kern), grid, block, ptrs, smem, stream);
  }(args...);
}

}  // namespace b2g
