// xent_few.cu -- the linear cross entropy of up to 64 tokens: scoring, and small
// training batches.
//
// With few tokens the products read the head w once and compute little, so this
// form is laid out around that read.  The classes are the rows of the MMA (M = 128
// per CTA) and the tokens its columns (N = 16, 32 or 64), where xent.cu's tiles
// would multiply mostly padding; the tile's height is chosen so that the SMs get
// equal shares of w; and an FP32 w is read by eight converter warps, three steps ahead
// in registers, and split into its BF16 planes on the way to shared memory, instead
// of by a pass over all of w (which costs 16 bytes an element: 478 us became 134 at 16
// x 32768 x 4096).  Modes:
//   kStats  z^T = w h^T: per token and CTA, the maximum and the sum of the
//           exponentials below it, and the target's logit
//   kDz     the same product, turned into dz (tokens x classes, BF16 planes)
//   kDh     dh^T = w^T dz^T: w's columns are the rows of the MMA ("MN-major" A), k
//           runs over the classes, cut into slices whose sums another kernel adds
// Bound: the bytes of w: 16 x 32768 x 4096, scoring, 46 us in BF16 (5.9 TB/s); FP32 134 us
// (4.0 TB/s).  What holds FP32's reads up has not been measured: of about 2200 cycles that a
// 64-k tile takes, issuing the split's instructions is some 520.
#include <atomic>

#include "xent.cuh"

namespace b2g {
namespace {

enum FewMode { kStats, kDz, kDh };

constexpr int kM = 128, kBK = 64;
constexpr int kMaxStages = 6;
constexpr uint32_t kPlane = kM * kBK * 2;      // a plane of A: 16 KB
// Tensor-memory columns of an accumulator: the tokens; with planes, three blocks of
// them.  The planes of B stand behind one another in shared memory, so one MMA
// multiplies a plane of A by several planes of B (N = 3, 2 and 1 times the tokens for
// A's planes 0, 1 and 2): three MMAs where the six products taken one by one would be
// six, each as long as its 128 rows of A.  The epilogue adds the blocks.
template <bool F32>
constexpr uint32_t kAccCols = F32 ? 256 : 64;
constexpr int kNumBars = 4 * kMaxStages + 5;
constexpr int kConvWarps = 8;

// BF16: a stage is 128 k, two 16 KB tiles of A with their tiles of B behind them, on
// one barrier (the issuing thread's time per stage is what small MMAs cost).  FP32: A
// comes from the converters as sets of three planes of 64 k, B has a ring of its own.
template <bool F32>
struct Cfg {
  static constexpr int kThreads = F32 ? 256 + 32 * kConvWarps : 256;
  static constexpr int kSub = F32 ? 1 : 2;      // 64-k tiles of a stage
  static constexpr uint32_t kA = (F32 ? 3 : 2) * kPlane;
};
constexpr int kSets = 3;                        // FP32: sets of planes

struct FewGemm {
  int rows;                    // classes of this piece (kStats, kDz) or width (kDh)
  int tokens, nt;              // nt: tokens rounded up to 16, 32 or 64
  int tile_rows, tiles, k_tiles, slices, group, planes;
  int a_stages, b_stages;      // a_stages: of both (BF16), or sets of planes
  const float* wf;             // FP32: row 0 of A
  long long ldw;
  int acols, arows;            // FP32: extents of w from there
  uint32_t a_tx;               // bytes the copies bring to a 64-k tile of A
  unsigned long long wait_limit_ns;
  int debug_stop;
  unsigned int* status;
  const void* target;
  int id_bytes, vocab, first;  // first: the class of row 0
  long long ignore;
  float2* stat;                // [CTAs][tokens]
  float* zt;
  const float* lse;
  const float* gloss;
  float* scale;
  Bf16* dz;
  long long dz_ld, dz_plane;
  float* part;                 // [slices][tokens][part_ld]
  long long part_ld;
};

__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHi)
      : "memory");
}

// A ring position.
struct Slot {
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++s == stages) s = 0, ph ^= 1u;
  }
};

// FP32 A on its way to three BF16 planes: this thread's four pieces of eight elements
// of a 64-k tile.  Eight lanes read 256 bytes of a row of w and write 128 bytes of a
// row of each plane (whole lines, no bank conflicts).  K-major: a piece is 8 k of a
// class; MN-major: 8 columns of a class (which is the k).
template <bool MN>
struct Pieces {
  float f[4][8];

  // (row of the tile's w, first column) of piece i of thread ct.
  static __device__ __forceinline__ void where(int i, int ct, int& row, int& col) {
    if (MN)
      row = (ct >> 4) + 16 * i, col = (ct & 15) * 8;  // 64 classes x 128 columns
    else
      row = (ct >> 3) + 32 * i, col = (ct & 7) * 8;   // 128 classes x 64 k
  }
  // Rows of w stand on 16-byte boundaries; past its end there are zeros.  Where all the
  // tile's columns exist the loads are predicated, not branched around: a branch would
  // wait for each load before the next one.
  __device__ __forceinline__ void load(const FewGemm& p, int m0, int k0, int ct) {
    const int c0 = MN ? m0 : k0, rows = MN ? 64 : p.tile_rows;
    const bool whole = c0 + (MN ? kM : kBK) <= p.acols;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int row, col;
      where(i, ct, row, col);
      const int r = (MN ? k0 : m0) + row, c = c0 + col;
      const bool in = r < p.arows && row < rows;
      const float* q = p.wf + (long long)r * p.ldw + c;
#pragma unroll
      for (int j = 0; j < 8; ++j) f[i][j] = 0.f;
      if (whole) {
#pragma unroll
        for (int j = 0; j < 8; j += 4)
          asm volatile(
              "{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %5, 0;\n\t"
              "@p ld.global.v4.f32 {%0, %1, %2, %3}, [%4];\n\t}"
              : "+f"(f[i][j]), "+f"(f[i][j + 1]), "+f"(f[i][j + 2]), "+f"(f[i][j + 3])
              : "l"(q + j), "r"((int)in));
      } else if (in) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j < p.acols) f[i][j] = q[j];
      }
    }
  }
  __device__ __forceinline__ void store(unsigned char* planes, int ct) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int row, col;
      where(i, ct, row, col);
      // K-major: row `row`, chunk col / 8; MN-major: block col / 64, row = k
      unsigned char* dst = planes + (MN ? (col >> 6) * 8192 : 0) + row * 128 +
                           (((col >> 3) & 7) ^ (row & 7)) * 16;
      uint32_t w[4];
#pragma unroll
      for (int pl = 0; pl < 3; ++pl) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = pl == 0   ? split_plane<true>(f[i][2 * j], f[i][2 * j + 1])
                 : pl == 1 ? split_plane<false>(f[i][2 * j], f[i][2 * j + 1])
                           : pack_bf16(f[i][2 * j], f[i][2 * j + 1]);
        *reinterpret_cast<uint4*>(dst + pl * kPlane) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
};

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

template <int MODE, bool F32>
__global__ void __launch_bounds__(Cfg<F32>::kThreads, 1)
    xent_few_kernel(const __grid_constant__ FewGemm p, const __grid_constant__ CUtensorMap mA,
                    const __grid_constant__ CUtensorMap mB) {
  constexpr bool MN = MODE == kDh;
  constexpr uint32_t kA = Cfg<F32>::kA;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(16) float zs[16][132];  // 16 tokens' logits of a tile (read as float4)
  __shared__ int cls[kFewTokens];              // each token's target within this piece, -1: none
  __shared__ float lse[kFewTokens], weight[kFewTokens];
  __shared__ uint32_t tmem_slot;
  const uint32_t raw = smem_addr(smem_raw);
  constexpr int kSub = Cfg<F32>::kSub;
  const uint32_t abase = (raw + 1023u) & ~1023u;
  const uint32_t bplane = (uint32_t)p.nt * 128u;
  const uint32_t bstage = (F32 ? 3 : kSub) * bplane;
  const uint32_t astage = F32 ? kA : kA + bstage;
  const uint32_t bbase = abase + (F32 ? kSets * kA : kA);
  const uint32_t bars = abase + (F32 ? kSets * kA + p.b_stages * bstage : p.a_stages * astage);
  auto afull = [&](int s) { return bars + 8u * s; };
  auto aempty = [&](int s) { return bars + 8u * (kMaxStages + s); };
  auto bfull = [&](int s) { return bars + 8u * (2 * kMaxStages + s); };
  auto bempty = [&](int s) { return bars + 8u * (3 * kMaxStages + s); };
  auto tfull = [&](int a) { return bars + 8u * (4 * kMaxStages + a); };
  auto tempty = [&](int a) { return bars + 8u * (4 * kMaxStages + 2 + a); };
  const uint32_t drain = bars + 8u * (4 * kMaxStages + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto wait = [&](uint32_t bar, uint32_t ph, unsigned int flag) {  // mbar_wait without a call
    if (mbar_try_wait(bar, ph)) return true;
    const uint64_t t0 = global_ns();
    while (!mbar_try_wait(bar, ph)) {
      if (global_ns() - t0 > p.wait_limit_ns) {
        atomicOr(p.status, flag);
        return false;
      }
    }
    return true;
  };
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(afull(s), F32 ? kConvWarps : 1);
      mbar_init(aempty(s), 1);
      mbar_init(bfull(s), 1);
      mbar_init(bempty(s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(tfull(s), 1);
      mbar_init(tempty(s), 4);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(&tmem_slot), 2 * kAccCols<F32>);
    tmem_relinquish();
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  pdl_wait();
  const uint32_t tmem = tmem_slot;
  if (MODE != kDh && threadIdx.x >= 64 && threadIdx.x < 64 + kFewTokens) {
    const int j = threadIdx.x - 64;
    int c = -1;
    float l = 0.f, g = 0.f;
    if (j < p.tokens) {
      const long long t = p.id_bytes == 8 ? static_cast<const long long*>(p.target)[j]
                                          : (long long)static_cast<const int*>(p.target)[j];
      const bool in = t >= 0 && t < p.vocab;
      if (in && t >= p.first && t < (long long)p.first + p.rows) c = (int)(t - p.first);
      if (MODE == kDz) {
        if (t != p.ignore && in)
          l = p.lse[j], g = p.gloss[j];
        else if (t != p.ignore && blockIdx.x == 0 && p.first == 0)
          atomicOr(p.status, kStatusIndex);
      }
    }
    cls[j] = c, lse[j] = l, weight[j] = g;
  }
  __syncthreads();
  const int units = p.tiles * p.slices;
  auto range = [&](int u, int& tile, int& slice, int& kt0, int& kt1) {
    tile = u / p.slices, slice = u - tile * p.slices;
    kt0 = (int)((long long)slice * p.k_tiles / p.slices);
    kt1 = (int)((long long)(slice + 1) * p.k_tiles / p.slices);
  };

  if (warp == 0) {
    // ------------------------------------------- copies: A and B, or FP32's B
    if (lane == 0) {
      const int stages = F32 ? p.b_stages : p.a_stages;
      const uint32_t full0 = F32 ? bfull(0) : afull(0), empty0 = F32 ? bempty(0) : aempty(0);
      const uint32_t tx = F32 ? bstage : kSub * p.a_tx + bstage;
      if (!F32) prefetch_tmap(&mA);
      prefetch_tmap(&mB);
      Slot at;
      int issued = 0;
      for (int u = blockIdx.x; u < units; u += gridDim.x) {
        int tile, slice, kt0, kt1;
        range(u, tile, slice, kt0, kt1);
        const int m0 = tile * p.tile_rows;
        for (int kt = kt0; kt < kt1; ++kt) {
          if (p.debug_stop >= 0 && issued >= p.debug_stop) goto copies_done;
          if (!wait(empty0 + 8u * at.s, at.ph ^ 1u, kStatusTimeoutEmpty)) goto copies_done;
          const uint32_t full = full0 + 8u * at.s;
          mbar_arrive_expect_tx(full, tx);
          if (F32) {
#pragma unroll
            for (int b = 0; b < 3; ++b)
              tma_load_3d(bbase + at.s * bstage + b * bplane, &mB, kt * kBK, 0, b, full);
          } else {
#pragma unroll
            for (int sub = 0; sub < kSub; ++sub) {
              const uint32_t dst = abase + at.s * astage + sub * kPlane;
              const int k = (kt * kSub + sub) * kBK;
              if (MN) {
                tma_load_3d(dst, &mA, m0, k, 0, full);
                tma_load_3d(dst + 8192, &mA, m0 + 64, k, 0, full);
              } else {
                tma_load_3d(dst, &mA, k, m0, 0, full);
              }
              tma_load_3d(bbase + at.s * astage + sub * bplane, &mB, k, 0, 0, full);
            }
          }
          ++issued;
          at.next(stages);
        }
      }
    copies_done:
      // leave only after every copy started here has landed
      for (int d = 0, pending = min(issued, stages); d < pending; ++d) {
        if (--at.s < 0) at.s = stages - 1, at.ph ^= 1u;
        if (!wait(full0 + 8u * at.s, at.ph, kStatusTimeoutDrain)) break;
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16(kM, p.nt, MN, false);  // N is N / 8 << 17
      // One thread issues everything, a few cycles an instruction: with the
      // descriptors built and the group found by division at every step, a stage of
      // 14 KB took 1260 cycles and w came in at 3.1 TB/s.
      const uint32_t a0 = desc_lo<MN>(abase), b0 = desc_lo<false>(bbase);
      const uint32_t a_step = astage >> 4;
      const uint32_t b_step = (F32 ? bstage : astage) >> 4, bp = bplane >> 4;
      Slot a, b, acc;
      for (int u = blockIdx.x; u < units; u += gridDim.x) {
        int tile, slice, kt0, kt1;
        range(u, tile, slice, kt0, kt1);
        int left = 0;  // stages of the accumulation group still to come
        for (int kt = kt0; kt < kt1; ++kt) {
          const bool begin = left == 0;
          if (begin) {
            left = min(p.group, kt1 - kt);
            if (!wait(tempty(acc.s), acc.ph ^ 1u, kStatusTimeoutTmem)) goto mma_done;
          }
          if (!wait(afull(a.s), a.ph, kStatusTimeoutFull)) goto mma_done;
          if (F32 && !wait(bfull(b.s), b.ph, kStatusTimeoutFull)) goto mma_done;
          tc_fence_after_sync();
          const uint32_t d = tmem + (uint32_t)acc.s * kAccCols<F32>;
          const uint32_t as = a0 + a.s * a_step, bs = b0 + (F32 ? b.s : a.s) * b_step;
          // FP32: plane 0 of A first (it covers all columns), then the smaller ones;
          // BF16: the stage's 64-k tiles.
#pragma unroll
          for (int i = 0; i < (F32 ? 3 : kSub); ++i) {
            const uint32_t ai = as + i * (kPlane >> 4), bi = bs + (F32 ? 0 : i * bp);
            const uint32_t id = F32 ? idesc + (uint32_t)((2 - i) * p.nt >> 3 << 17) : idesc;
#pragma unroll
            for (int kk = 0; kk < kBK / 16; ++kk)
              mma_bf16(d, ai + kk * kDescStep<MN>, bi + kk * kDescStep<false>, id,
                       begin && i == 0 && kk == 0 ? 0u : 1u);
          }
          mma_commit(aempty(a.s));
          if (F32) {
            mma_commit(bempty(b.s));
            b.next(p.b_stages);
          }
          a.next(p.a_stages);
          if (--left == 0) {
            mma_commit(tfull(acc.s));
            acc.next(2);
          }
        }
      }
    mma_done:
      mma_commit(drain);
      wait(drain, 0, kStatusTimeoutTmem);
    }
    __syncwarp();
  } else if (F32 && warp >= 8) {
    // ---------------------------------------------------------- converters
    const int ct = (int)threadIdx.x - 256;
    unsigned char* sets = smem_raw + (abase - raw);
    // This CTA's 64-k tiles in order; the pieces of the next three are on their way.
    struct Walk {
      int u, tile, kt, kt1;
    } w;
    auto enter = [&](int u) {  // the first tile at or after unit u
      w.u = u, w.kt = w.kt1 = 0;
      for (; w.u < units; w.u += gridDim.x) {
        int slice;
        range(w.u, w.tile, slice, w.kt, w.kt1);
        if (w.kt < w.kt1) break;
      }
    };
    auto fetch = [&](Pieces<MN>& x) {  // the walk's tile, if there is one
      if (w.u >= units) return false;
      x.load(p, w.tile * p.tile_rows, w.kt * kBK, ct);
      if (++w.kt == w.kt1) enter(w.u + gridDim.x);
      return true;
    };
    Slot a;
    auto put = [&](Pieces<MN>& x) {
      if (!__all_sync(0xffffffffu, wait(aempty(a.s), a.ph ^ 1u, kStatusTimeoutEmpty))) return false;
      x.store(sets + a.s * kA, ct);
      fence_proxy_async_smem();  // the MMA reads what was written here
      __syncwarp();
      if (lane == 0) mbar_arrive(afull(a.s));
      a.next(kSets);
      return true;
    };
    enter(blockIdx.x);
    Pieces<MN> x, y, z;
    bool have_x = fetch(x), have_y = fetch(y), have_z = fetch(z);
    while (have_x) {
      if (!put(x)) break;
      have_x = fetch(x);
      if (!have_y || !put(y)) break;
      have_y = fetch(y);
      if (!have_z || !put(z)) break;
      have_z = fetch(z);
    }
  } else if (warp >= 4 && warp < 8) {
    // ---------------------------------------------------------- epilogue
    const int q = warp & 3;
    const uint32_t tmem_lane = tmem + ((uint32_t)(32 * q) << 16);
    float scale = 1.f;
    if (MODE == kDz) {
      float m = 0.f;
      for (int j = lane; j < kFewTokens; j += 32) m = fmaxf(m, isfinite(weight[j]) ? fabsf(weight[j]) : 0.f);
      m = divisor_of(warp_max(m));
      if (blockIdx.x == 0 && threadIdx.x == 128) *p.scale = m;
      scale = 1.f / m;
    } else if (MODE == kDh) {
      scale = *p.scale;
    }
    const int et = threadIdx.x - 128;  // 0 .. 127 among the epilogue's threads
    float2 run[kFewTokens / 16];       // kStats: of token 16 c + et / 8, this thread's rows
#pragma unroll
    for (int c = 0; c < kFewTokens / 16; ++c) run[c] = make_float2(-INFINITY, 0.f);
    Slot at;
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      int tile, slice, kt0, kt1;
      range(u, tile, slice, kt0, kt1);
      float z[kFewTokens];
#pragma unroll
      for (int j = 0; j < kFewTokens; ++j) z[j] = 0.f;  // a slice may be empty
      for (int g = 0; g < (kt1 - kt0 + p.group - 1) / p.group && ok; ++g) {
        ok = __all_sync(0xffffffffu, wait(tfull(at.s), at.ph, kStatusTimeoutTmem));
        if (!ok) break;
        tc_fence_after_sync();
#pragma unroll
        for (int c = 0; c < kFewTokens; c += 16) {
          if (c < p.nt) {
#pragma unroll 1
            for (int b = F32 ? 2 : 0; b >= 0; --b) {  // the smallest products first
              uint32_t v[16];
              tmem_ld16(tmem_lane + (uint32_t)at.s * kAccCols<F32> + b * p.nt + c, v);
              tmem_ld_wait();
              tie16(v);
#pragma unroll
              for (int j = 0; j < 16; ++j) z[c + j] += __uint_as_float(v[j]);
            }
          }
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty(at.s));
        at.next(2);
      }
      if (MODE != kDh) {  // the barriers below need all four warps: go on together or not at all
        int all;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 q, %1, 0;\n\t"
            "bar.red.and.pred p, 1, 128, q;\n\tselp.s32 %0, 1, 0, p;\n\t}"
            : "=r"(all)
            : "r"((int)ok)
            : "memory");
        ok = all != 0;
      }
      if (!ok) break;
      const int local = 32 * q + lane, r = tile * p.tile_rows + local;
      const bool in = local < p.tile_rows && r < p.rows;
      if (MODE != kDh) {
        // 16 tokens at a time through shared memory, so that a thread has 16 classes
        // of one token: et / 8 of the 16, classes 16 (et % 8) .. + 15 of the tile.
        const int token16 = et >> 3, c0 = 16 * (et & 7);
        const int left = min(p.tile_rows, p.rows - tile * p.tile_rows) - c0;  // classes that exist
#pragma unroll
        for (int c = 0; c < kFewTokens / 16; ++c) {
          if (16 * c < p.tokens) {
#pragma unroll
            for (int j = 0; j < 16; ++j) zs[j][local] = z[16 * c + j];
            asm volatile("bar.sync 1, 128;" ::: "memory");
            const int token = 16 * c + token16;
            float x[16];
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const float4 v = *reinterpret_cast<const float4*>(&zs[token16][c0 + j]);
              x[j] = v.x, x[j + 1] = v.y, x[j + 2] = v.z, x[j + 3] = v.w;
            }
            const int mine = cls[token] - tile * p.tile_rows - c0;  // the target among these
            if (MODE == kStats) {
              float top = run[c].x;
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                if (j >= left) x[j] = -INFINITY;
                top = fmaxf(top, x[j]);
                if (j == mine && j < left && token < p.tokens) p.zt[token] = x[j];
              }
              const float ref = top == -INFINITY ? 0.f : top;
              float sum = run[c].y * exp_f32(run[c].x - ref), more = 0.f;
#pragma unroll
              for (int j = 0; j < 16; j += 2)
                sum += exp_f32(x[j] - ref), more += exp_f32(x[j + 1] - ref);
              run[c] = make_float2(top, sum + more);
            } else if (token < p.tokens && left > 0) {
              const float g = weight[token] * scale, l = lse[token];
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float e = exp_f32(x[j] - l) - (j == mine ? 1.f : 0.f);
                x[j] = g != 0.f ? g * e : 0.f;
              }
              Bf16* out = p.dz + (long long)token * p.dz_ld + tile * p.tile_rows + c0;
              for (int pl = 0; pl < p.planes; ++pl) {
                uint32_t b[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) b[j] = split_plane<false>(x[2 * j], x[2 * j + 1]);
                // tiles are multiples of 8 classes, and dz's rows padded past the last
                uint4* q = reinterpret_cast<uint4*>(out + pl * p.dz_plane);
                q[0] = make_uint4(b[0], b[1], b[2], b[3]);
                if (left > 8) q[1] = make_uint4(b[4], b[5], b[6], b[7]);
              }
            }
            asm volatile("bar.sync 1, 128;" ::: "memory");
          }
        }
      } else if (in) {
        float* out = p.part + (size_t)slice * p.tokens * p.part_ld + r;
#pragma unroll
        for (int j = 0; j < kFewTokens; ++j)
          if (j < p.tokens) out[j * p.part_ld] = scale * z[j];
      }
    }
    if (MODE == kStats) {  // the eight threads of a token, then one row of the CTA's own
#pragma unroll
      for (int c = 0; c < kFewTokens / 16; ++c) {
        float2 r = run[c];
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
          const float m = __shfl_xor_sync(0xffffffffu, r.x, o);
          const float s = __shfl_xor_sync(0xffffffffu, r.y, o);
          const float top = fmaxf(r.x, m), ref = top == -INFINITY ? 0.f : top;
          r = make_float2(top, r.y * exp_f32(r.x - ref) + s * exp_f32(m - ref));
        }
        const int token = 16 * c + (et >> 3);
        if ((et & 7) == 0 && token < p.tokens) p.stat[(size_t)blockIdx.x * p.tokens + token] = r;
      }
    }
  }

  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 2 * kAccCols<F32>);
  }
}

// ------------------------------------------------------------------- host side

constexpr int kPlanCtas = 152;  // GB300's SMs: the launch shapes are planned without a device

// Rows of a tile, 64 to 128: the fewest that keep the SMs' shares equal (32768
// classes: 112, two rounds of 152 tiles of 224 KB in BF16 at width 1024; 128 would
// leave a third of the SMs without a second tile).
int tile_rows_for(int rows) {
  int best = kM;
  long long cost = -1;
  for (int t = kM; t >= 64; t -= 8) {
    const long long c = ceil_div(ceil_div(rows, t), kPlanCtas) * (t + 8);
    if (cost < 0 || c < cost) best = t, cost = c;
  }
  return best;
}

int padded_tokens(int tokens) { return tokens <= 16 ? 16 : tokens <= 32 ? 32 : 64; }

template <int MODE, bool F32>
int launch(FewGemm p, const CUtensorMap& mA, const CUtensorMap& mB, const TrainDevice& d,
           cudaStream_t st) {
  static std::atomic<int> configured[64];
  p.planes = F32 ? 3 : 1;
  const uint32_t bstage = (uint32_t)((F32 ? 3 : Cfg<F32>::kSub) * p.nt * 128);
  p.a_stages = F32 ? kSets : p.nt == 64 ? 4 : p.nt == 32 ? 5 : 6;
  p.b_stages = F32 ? (p.nt == 64 ? 2 : 4) : 0;
  const size_t smem = 1024 + p.a_stages * ((size_t)Cfg<F32>::kA + (F32 ? 0 : bstage)) +
                      p.b_stages * (size_t)bstage + kNumBars * 8;
  p.wait_limit_ns = d.wait_limit_ns, p.debug_stop = d.debug_stop, p.status = d.status;
  if (d.dev < 0 || d.dev >= 64) return B2G_ERR_DEVICE;
  if (!configured[d.dev].load(std::memory_order_acquire)) {
    // the largest form: six BF16 stages of 36 KB
    if (cudaFuncSetAttribute(xent_few_kernel<MODE, F32>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             6 * 36 * 1024 + 1024 + 512) != cudaSuccess)
      return B2G_ERR_CUDA;
    configured[d.dev].store(1, std::memory_order_release);
  }
  const int units = p.tiles * p.slices;
  CUtensorMap a = mA, b = mB;
  void* args[] = {&p, &a, &b};
  return launch_code(launch_pdl(reinterpret_cast<const void*>(&xent_few_kernel<MODE, F32>),
                                dim3((unsigned)(units < kPlanCtas ? units : kPlanCtas)),
                                dim3(Cfg<F32>::kThreads), args, smem, st));
}

// The product of w's rows with h, for kStats and kDz.
template <int MODE>
int launch_rows(FewGemm p, const XentRows& r, const Planes& h, const FewHead& w,
                const TrainDevice& d, cudaStream_t st) {
  const int es = w.f32 ? 4 : 2;
  p.tokens = r.tokens, p.nt = padded_tokens(r.tokens);
  p.tile_rows = tile_rows_for(p.rows), p.tiles = (int)ceil_div(p.rows, p.tile_rows);
  p.k_tiles = (int)ceil_div(r.width, w.f32 ? kBK : 2 * kBK), p.slices = 1;
  // 64 and 1024 k.  (FP32: 256 k would take 131 us for 134 at 16 x 32768 x 4096, with three
  // times the error of the loss.)
  p.group = w.f32 ? 1 : 8;
  p.a_tx = (uint32_t)(p.tile_rows * kBK * es);
  p.target = r.target, p.id_bytes = r.id_bytes, p.vocab = r.vocab, p.ignore = r.ignore;
  CUtensorMap a = {}, b = {};
  const unsigned char* base = static_cast<const unsigned char*>(w.w) + (long long)p.first * w.ldw * es;
  p.wf = reinterpret_cast<const float*>(base), p.ldw = w.ldw;
  p.arows = p.rows, p.acols = r.width;
  int rc = w.f32 ? 0 : encode_rows(&a, false, base, r.width, p.rows, w.ldw, 1, 0, p.tile_rows);
  if (!rc) rc = encode_rows(&b, false, h.p, h.cols, h.rows, h.ld, h.planes, h.plane, p.nt);
  if (rc) return rc;
  return w.f32 ? launch<MODE, true>(p, a, b, d, st) : launch<MODE, false>(p, a, b, d, st);
}

}  // namespace

int few_stat_parts(int classes) {  // one per CTA
  const long long tiles = ceil_div(classes, tile_rows_for(classes));
  return (int)(tiles < kPlanCtas ? tiles : kPlanCtas);
}

// k slices of dh: what fills the SMs' rounds best, at least four k tiles each.
int few_slices(int width, int classes) {
  const long long tiles = ceil_div(width, kM), kt = ceil_div(classes, kBK);
  int best = 1;
  double cost = -1;
  for (int s = 1; s <= 32 && s * 4 <= (kt > 4 ? kt : 4); ++s) {
    const double c = (double)ceil_div(tiles * s, kPlanCtas) * ((double)ceil_div(kt, s) + 2);
    if (cost < 0 || c < cost) best = s, cost = c;
  }
  return best;
}

int launch_few_stats(const XentRows& r, const Planes& h, const FewHead& w, float2* stat, float* zt,
                     const TrainDevice& d, cudaStream_t st) {
  FewGemm p = {};
  p.rows = r.vocab, p.first = 0, p.stat = stat, p.zt = zt;
  return launch_rows<kStats>(p, r, h, w, d, st);
}

int launch_few_dz(const XentRows& r, const Planes& h, const FewHead& w, int first, int n,
                  const float* lse, const float* gloss, const Planes& dz, float* scale,
                  const TrainDevice& d, cudaStream_t st) {
  FewGemm p = {};
  p.rows = n, p.first = first, p.lse = lse, p.gloss = gloss, p.scale = scale;
  p.dz = const_cast<Bf16*>(dz.p), p.dz_ld = dz.ld, p.dz_plane = dz.plane;
  return launch_rows<kDz>(p, r, h, w, d, st);
}

int launch_few_dh(const XentRows& r, const Planes& dz, const FewHead& w, int first, int n,
                  const float* scale, int slices, float* part, long long ld, const TrainDevice& d,
                  cudaStream_t st) {
  FewGemm p = {};
  const int es = w.f32 ? 4 : 2;
  p.rows = r.width, p.tokens = r.tokens, p.nt = padded_tokens(r.tokens);
  p.tile_rows = kM, p.tiles = (int)ceil_div(r.width, kM);
  p.k_tiles = (int)ceil_div(n, w.f32 ? kBK : 2 * kBK);
  p.slices = slices;
  p.group = w.f32 ? 1 : kGroupK / (2 * kBK);
  p.a_tx = (uint32_t)(kM * kBK * es);
  p.scale = const_cast<float*>(scale), p.part = part, p.part_ld = ld;
  CUtensorMap a = {}, b = {};
  const unsigned char* base = static_cast<const unsigned char*>(w.w) + (long long)first * w.ldw * es;
  p.wf = reinterpret_cast<const float*>(base), p.ldw = w.ldw;
  p.arows = n, p.acols = r.width;
  int rc = w.f32 ? 0 : encode_rows(&a, false, base, r.width, n, w.ldw, 1, 0, kBK);
  if (!rc) rc = encode_rows(&b, false, dz.p, dz.cols, dz.rows, dz.ld, dz.planes, dz.plane, p.nt);
  if (rc) return rc;
  return w.f32 ? launch<kDh, true>(p, a, b, d, st) : launch<kDh, false>(p, a, b, d, st);
}

}  // namespace b2g
