// pair.cuh -- what the CTA-pair products of BF16 planes share (xent.cu, wgrad8.cu): tiles of
// 256 x 256 in two CTAs' tensor memory, operands of either order in 128-byte-swizzled
// stages, the way of a finished tile out of tensor memory.
#pragma once
#include "xent.cuh"

namespace b2g {

constexpr int kTile = 256;       // rows and (at most) columns of a pair's tile
constexpr int kBK = 64;          // k per stage: 128 bytes of BF16
constexpr int kEpiWarps = 8;     // two per tensor-memory quarter, 128 columns each
constexpr uint32_t kOutBytes = 4096;           // an epilogue warp's 32 rows of 128 bytes on their way out

__device__ __forceinline__ void mma_bf16_pair(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHi)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* m, int c0,
                                                 int c1, int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

// mbar_wait without a function call: registers are redistributed among the warps
// here, and a called function would have to fit the smallest share.  CLUSTER: for what
// the other CTA's threads wrote.
template <bool CLUSTER = false, typename P>
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, const P& p,
                                           unsigned int flag) {
  auto done = [&] { return CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
  if (done()) return true;
  const uint64_t t0 = global_ns();
  while (!done()) {
    if (global_ns() - t0 > p.wait_limit_ns) {
      atomicOr(p.status, flag);
      return false;
    }
  }
  return true;
}

// 128 rows (64 in MN-major order where `wide` is false) of an operand at (row m0, k block
// kt, plane) into a 16 KB stage tile.
template <bool MN>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap* m, int m0, int kt,
                                             int plane, uint32_t bar, bool wide = true) {
  if constexpr (MN) {
    tma_load_3d_pair(dst, m, m0, kt * kBK, plane, bar);
    if (wide) tma_load_3d_pair(dst + 8192, m, m0 + 64, kt * kBK, plane, bar);
  } else {
    tma_load_3d_pair(dst, m, kt * kBK, m0, plane, bar);
  }
}

// This warp's `span` columns (64 or 128) of the accumulators that `tfull` announces, added up
// over the unit's accumulation groups: acc holds FP32 sums rounded to nearest.
// Two loads are in flight at a time.  Returns false when a wait ran out.
template <typename P>
__device__ __forceinline__ bool collect(const P& p, float (&acc)[128], uint32_t tmem_lane,
                                        int span, int groups, int& a, uint32_t& aph, uint32_t tfull0,
                                        uint32_t tempty0, uint32_t tempty0_even, bool even,
                                        int lane) {
  for (int g = 0; g < groups; ++g) {
    if (!__all_sync(0xffffffffu, wait_phase(tfull0 + 8u * a, aph, p, kStatusTimeoutTmem)))
      return false;
    tc_fence_after_sync();
#pragma unroll
    for (int c = 0; c < 128; c += 64) {
      if (c >= span) continue;
      uint32_t v[32], w[32];
      tmem_ld32(tmem_lane + (uint32_t)(a * kTile + c), v);
      tmem_ld32(tmem_lane + (uint32_t)(a * kTile + c + 32), w);
      tmem_ld_wait();
      tie32(v);
      tie32(w);
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        acc[c + j] = g == 0 ? __uint_as_float(v[j]) : acc[c + j] + __uint_as_float(v[j]);
        acc[c + 32 + j] = g == 0 ? __uint_as_float(w[j]) : acc[c + 32 + j] + __uint_as_float(w[j]);
      }
    }
    tc_fence_before_sync();
    __syncwarp();
    if (lane == 0) {  // the tile may be overwritten
      if (even)
        mbar_arrive(tempty0 + 8u * a);
      else
        mbar_arrive_remote(tempty0_even + 8u * a);
    }
    if (++a == 2) a = 0, aph ^= 1u;
  }
  return true;
}

// A lane's row of 128 bytes to its warp's buffer, in the 128-byte swizzle.  Every write to
// the buffer goes through here and first waits for whoever still reads it: the last
// bulk-tensor store (lane 0 committed it; a unit of the other gradient may have left
// through one just before), then the warp's other lanes.
__device__ __forceinline__ void stage_rows(uint32_t buf, const uint4 (&w)[8], int lane) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t at = buf + lane * 128u + (uint32_t)((i ^ (lane & 7)) * 16);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[i].x), "r"(w[i].y),
                 "r"(w[i].z), "r"(w[i].w)
                 : "memory");
  }
}

// A warp's 32 rows of 128 bytes through its shared-memory buffer to (x, y, z) of
// an output tensor: eight 16-byte pieces a lane, in the 128-byte swizzle (no bank
// conflicts, and full lines leave the SM), then one bulk-tensor store, which
// leaves out rows and columns past the tensor.
__device__ __forceinline__ void store_rows(uint32_t buf, const CUtensorMap* m, int x, int y, int z,
                                           const uint4 (&w)[8], bool add, int lane) {
  stage_rows(buf, w, lane);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (add)
      asm volatile(
          "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group"
          " [%0, {%1, %2, %3}], [%4];" ::"l"(reinterpret_cast<uint64_t>(m)),
          "r"(x), "r"(y), "r"(z), "r"(buf)
          : "memory");
    else
      asm volatile(
          "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group"
          " [%0, {%1, %2, %3}], [%4];" ::"l"(reinterpret_cast<uint64_t>(m)),
          "r"(x), "r"(y), "r"(z), "r"(buf)
          : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}

// Before the block ends: the stores of this thread have been written.
__device__ __forceinline__ void stores_done() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// v (plus the old values) to a warp's rows of a result that a bulk-tensor store
// cannot write (alignment) or add to (BF16): 32 columns at a time through the buffer,
// so that each store is a stretch of one row.
template <typename T, int N, typename P>
__device__ __forceinline__ void put_rows(T* out, const float (&v)[N], const P& p, int row0,
                                         int left, uint32_t buf, int lane) {
#pragma unroll
  for (int c = 0; c < N; c += 32) {
    if (c < left) {
      uint4 w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        w[j] = make_uint4(__float_as_uint(v[c + 4 * j]), __float_as_uint(v[c + 4 * j + 1]),
                          __float_as_uint(v[c + 4 * j + 2]), __float_as_uint(v[c + 4 * j + 3]));
      stage_rows(buf, w, lane);
      __syncwarp();
      const int rows = min(32, p.rows - row0);
      auto at = [&](int i) {
        float x;
        asm volatile("ld.shared.f32 %0, [%1];"
                     : "=f"(x)
                     : "r"(buf + i * 128u + (uint32_t)(((lane >> 2) ^ (i & 7)) * 16 + (lane & 3) * 4)));
        return x;
      };
      if (c + lane < left) {
        // a loop of its own: stores that no loads can depend on (a 1000 x 5001 x 3333 BF16 weight
        // gradient 46 us with the loop below, 37 so)
        if (!p.accumulate) {
#pragma unroll 4
          for (int i = 0; i < rows; ++i) out[(long long)i * p.ldo + c + lane] = from_f32<T>(at(i));
        } else if constexpr (N > 64) {
#pragma unroll 4
          for (int i = 0; i < rows; ++i) {
            T* q = out + (long long)i * p.ldo + c + lane;
            *q = from_f32<T>(at(i) + to_f32(*q));
          }
        } else {
          // with the registers for it, the old values of 16 rows on their way together (64 tokens on
          // 4096 x 4096 BF16 165 us -> 53)
          T* q = out + c + lane;
#pragma unroll 1
          for (int i0 = 0; i0 < rows; i0 += 16, q += 16 * p.ldo) {
            T old[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (i0 + i < rows) old[i] = q[i * p.ldo];
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (i0 + i < rows) q[i * p.ldo] = from_f32<T>(at(i0 + i) + to_f32(old[i]));
          }
        }
      }
    }
  }
}

}  // namespace b2g
