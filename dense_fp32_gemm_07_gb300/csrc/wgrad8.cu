// wgrad8.cu -- a linear layer's weight gradient dw = dy^T x from an x kept in 8 bits
// (b2g_linear_dweight8 in include/b2g_train.h), on the 5th-generation tensor cores.
//
// dw (outs x width) is a sum over the tokens, so both operands are read with their rows
// as k ("MN-major") and nothing is transposed.  x's values have 4 significant bits and
// power-of-two scales: BF16 holds them exactly.  A first kernel writes them so; or, where there
// are few products for each of them, warps of the product's kernel on their way to the stages.
// BF16 dy is multiplied as it is; FP32 dy is split into three BF16 planes, dy = d0 + d1 + d2
// to 24 bits, and the three products d x are added up, the smallest first.
//
// The product runs on 256 x 256 tiles of a CTA pair (tcgen05.mma.cta_group::2, FP32
// accumulators in tensor memory, double buffered).  As many tiles as fill all pairs are
// whole; the rest are whole too, or halves of 128 columns, or their k range is cut into pieces,
// so that more of the pairs have work to the end.  A piece leaves FP32 sums, which a last
// kernel adds in order: straight from registers, 32 rows x 4 columns (512 bytes) at a time, the
// order in which a warp holds them.
//
// Bound: the tensor cores; short sums, writing the result.  BF16: 16384 tokens on 11008 x 4096
// 775 to 870 us (1.70 to 1.91 PFLOP/s, under the power cap), 4096 on 4096 x 4096 86 us, of
// which the products 70 and the preparation 8 to 10; 64 on 4096 x 4096 13.9 (34 MB written; 15.6
// with a preparation).  FP32: 4096 on 4096 x 4096 237 us, 1.74 PFLOP/s of the three products.
// Converting x on its way takes about 1150 cycles a k tile, the products alone 520: 80 KB through
// shared memory (dy and codes in, codes out, BF16 in, both operands out) are 640 cycles; the
// converting warps' loads, bit operations (360 cycles of a scheduler's, at half rate) and barriers
// follow one another, half hidden by two groups of warps with a k tile each; and the odd CTA's
// tiles wait for a fence of the cluster, which the five stages do not hide altogether.
#include <atomic>
#include <type_traits>

#include "eightbit.cuh"
#include "pair.cuh"

namespace b2g {
namespace {

// Warp 0 copies, warp 1 multiplies; with EIGHT warp 2 copies x's codes, kCvtWarps more warps
// write them to the stages as BF16, and warps 1 and 3 of the odd CTA tell the even one.
constexpr int kCvtWarps = 8;
// Groups of them with a k tile each: what the warps of one wait for, the other one hides.
constexpr int kCvtGroups = 2;
template <bool EIGHT>
constexpr int kThreads = 128 + 32 * (kEpiWarps + (EIGHT ? kCvtWarps : 0));
// Registers, as in the cross entropy's product: 128 * 72 + 256 * 216 = 64,512 of the 168 a
// thread that the block starts with; with EIGHT 128 * 72 + 256 * 120 + 256 * 80 = 60,416 of 96.
constexpr int kIssueRegs = 72;
template <bool EIGHT>
constexpr int kEpiRegs = EIGHT ? 120 : 216;
constexpr int kCvtRegs = 80;
constexpr uint32_t kOperand = 128 * kBK * 2;    // a CTA's 128 rows of one plane: 16 KB
// A stage holds all planes of a k tile of dy, and x's.  With EIGHT two of the twelve operands'
// places hold codes.
template <int PLANES, bool EIGHT>
constexpr int kStages = (EIGHT ? 10 : 12) / (PLANES + 1);
template <int PLANES>
constexpr uint32_t kStageBytes = (PLANES + 1) * kOperand;
constexpr int kMaxStages = 6;
constexpr int kCodeTiles = 4;                   // 64 tokens x 128 codes
constexpr uint32_t kCodeBytes = kBK * 128;
// Barriers on which a group of converting warps of the odd CTA announces its k tiles in turns.
// Their tiles reach as far as the stages, so that none is announced a second time before the
// even CTA has been told of the first.
constexpr int kTellSlots = 3;
static_assert(kCvtGroups == 2 && kCvtGroups * kTellSlots >= kStages<1, true>);
constexpr int kNumBars = 2 * kMaxStages + 5 + 2 * kCodeTiles + kCvtGroups * kTellSlots;
constexpr int kSmemBytes = 12 * kOperand + kEpiWarps * kOutBytes + 1024 + kNumBars * 8 + 16;
constexpr uint32_t kTmemCols = 2 * kTile;
constexpr int kPairs = 76;  // what the work is shared out among (GB300: 152 SMs)

struct Dw8Gemm {
  int rows, cols;            // outs, width
  int tiles_m, tiles_n, k_tiles;
  int tile_n;                // columns of a tile: 256, or 128
  int full, rest;            // whole tiles a pair; tiles that remain
  int halves;                // which then go as two of 128 columns
  unsigned piece;            // k tiles of a pair's piece of the rest
  unsigned span;             // k tiles that a tile of the rest counts for: its own, or whole pieces
  int split;                 // pieces leave sums
  int group;                 // k tiles that add up in tensor memory before FP32 takes over
  unsigned long long wait_limit_ns;
  int debug_stop;            // >= 0: the copy issuer stops early (timeout test)
  unsigned int* status;
  int add;                   // a bulk-tensor store adds to what is there
  int out_tma;               // whole tiles leave by bulk-tensor stores; else element by element
  void* out;
  long long ldo;
  int out_bf16, accumulate;
  float* part;               // the sums, [slot][16 warps][columns / 4][32 rows][4]
  const unsigned char* scales;  // with EIGHT: x's, of `tokens` rows
  long long lds;
  int tokens;
};
struct alignas(64) Dw8Maps {
  CUtensorMap dy, x, out;    // x: BF16, or with EIGHT the codes
};

struct Unit {
  int tile, kt0, kt1, slot;  // slot: of the sums, -1 for a result
  int col, cols;             // its columns of the tile
};

// The k-th unit of this pair; false: there is none.
__device__ __forceinline__ bool unit_at(const Dw8Gemm& p, int pair, int pairs, int k, Unit& u) {
  if (k < p.full) {
    u = Unit{k * pairs + pair, 0, p.k_tiles, -1, 0, p.tile_n};
    return true;
  }
  k -= p.full;
  if (p.halves) {
    u = Unit{p.full * pairs + (pair >> 1), 0, p.k_tiles, -1, (pair & 1) * 128, 128};
    return k == 0 && pair < 2 * p.rest;
  }
  const unsigned all = (unsigned)p.rest * p.span;  // below 2^32
  const unsigned from = pair * p.piece, to = min(from + p.piece, all);
  const unsigned tile = from / p.span, edge = (tile + 1) * p.span;  // a piece spans two tiles at most
  if (k > 1 || from >= to || (k == 1 && to <= edge)) return false;
  const unsigned a = k ? edge : from, base = (tile + k) * p.span;
  const unsigned b = min(k ? to : min(to, edge), base + p.k_tiles);
  u = Unit{p.full * pairs + (int)tile + k, (int)(a - base), (int)(b - base), p.split ? 2 * pair + k : -1,
           0, p.tile_n};
  return true;
}

// Tiles in groups of 16 rows of tiles, so that a wave shares operand rows in L2.
__device__ __forceinline__ void tile_at(const Dw8Gemm& p, int tile, int& tm, int& tn) {
  constexpr int kGroup = 16;
  const int per = kGroup * p.tiles_n, g = tile / per, first = g * kGroup;
  const int size = min(p.tiles_m - first, kGroup), r = tile - g * per;
  tm = first + r % size;
  tn = r / size;
}

__device__ __forceinline__ int groups_of(const Dw8Gemm& p, int kts) {
  return (kts + p.group - 1) / p.group;
}

// Where a slot's sums of a warp's 32 rows (block `rows` of 8) and columns (`half` of 2) begin;
// four columns of its 32 rows follow one another.
__device__ __forceinline__ size_t sums_at(unsigned slot, int rows, int half, int tile_n) {
  return ((size_t)slot * 16 + rows * 2 + half) * (32 * (tile_n / 2));
}
__device__ __forceinline__ void put_sums(float* part, const float (&v)[128], int left, int lane) {
  float4* to = reinterpret_cast<float4*>(part) + lane;
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (4 * j < left) to[32 * j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}

// This warp's columns of rows row0 .. row0 + 31 of a finished tile to the result.
__device__ __forceinline__ void put_tile(const Dw8Gemm& p, const CUtensorMap* m, float (&v)[128], int row0,
                                         int n0, int left, uint32_t buf, int lane) {
  if (p.out_tma && !p.out_bf16) {
#pragma unroll
    for (int c = 0; c < 128; c += 32) {
      if (c < left) {
        uint4 w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          w[j] = make_uint4(__float_as_uint(v[c + 4 * j]), __float_as_uint(v[c + 4 * j + 1]),
                            __float_as_uint(v[c + 4 * j + 2]), __float_as_uint(v[c + 4 * j + 3]));
        store_rows(buf, m, n0 + c, row0, 0, w, p.add, lane);
      }
    }
  } else if (p.out_tma) {
#pragma unroll
    for (int c = 0; c < 128; c += 64) {
      if (c < left) {
        uint4 w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = c + 8 * j;
          w[j] = make_uint4(pack_bf16(v[i], v[i + 1]), pack_bf16(v[i + 2], v[i + 3]),
                            pack_bf16(v[i + 4], v[i + 5]), pack_bf16(v[i + 6], v[i + 7]));
        }
        store_rows(buf, m, n0 + c, row0, 0, w, false, lane);
      }
    }
  } else if (p.out_bf16) {
    put_rows(static_cast<Bf16*>(p.out) + (long long)row0 * p.ldo + n0, v, p, row0, left, buf, lane);
  } else {
    put_rows(static_cast<float*>(p.out) + (long long)row0 * p.ldo + n0, v, p, row0, left, buf, lane);
  }
}

// A unit of one accumulation group to BF16, or its sums, 64 columns at a time; of each four the
// second and third are back in their places.
// False when the wait for it ran out.
__device__ __forceinline__ bool put_bf16(const Dw8Gemm& p, const Unit& u, const CUtensorMap* m,
                                         uint32_t tmem_lane, int span, int rows, int half, int row0, int n0,
                                         int left, int& a, uint32_t& aph, uint32_t tfull0, uint32_t tempty0,
                                         uint32_t tempty0_even, bool even, uint32_t buf, int lane) {
  if (!__all_sync(0xffffffffu, wait_phase(tfull0 + 8u * a, aph, p, kStatusTimeoutTmem))) return false;
  tc_fence_after_sync();
#pragma unroll 1
  for (int c = 0; c < span; c += 64) {
    uint32_t v[32], x[32];
    tmem_ld32(tmem_lane + (uint32_t)(a * kTile + c), v);
    tmem_ld32(tmem_lane + (uint32_t)(a * kTile + c + 32), x);
    tmem_ld_wait();
    tie32(v);
    tie32(x);
    if (c + 64 == span) {  // the tile may be overwritten
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if (even)
          mbar_arrive(tempty0 + 8u * a);
        else
          mbar_arrive_remote(tempty0_even + 8u * a);
      }
    }
    if (c >= left) continue;
    if (u.slot >= 0) {
      uint4* to = reinterpret_cast<uint4*>(p.part + sums_at(u.slot, rows, half, p.tile_n)) + 8 * c + lane;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (c + 4 * j < left) to[32 * j] = make_uint4(v[4 * j], v[4 * j + 2], v[4 * j + 1], v[4 * j + 3]);
        if (c + 4 * j + 32 < left)
          to[32 * j + 256] = make_uint4(x[4 * j], x[4 * j + 2], x[4 * j + 1], x[4 * j + 3]);
      }
    } else if (!p.out_tma) {
      float f[64];
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        f[j] = __uint_as_float(v[j]), f[j + 1] = __uint_as_float(v[j + 2]);
        f[j + 2] = __uint_as_float(v[j + 1]), f[j + 3] = __uint_as_float(v[j + 3]);
        f[32 + j] = __uint_as_float(x[j]), f[33 + j] = __uint_as_float(x[j + 2]);
        f[34 + j] = __uint_as_float(x[j + 1]), f[35 + j] = __uint_as_float(x[j + 3]);
      }
      put_rows(static_cast<Bf16*>(p.out) + (long long)row0 * p.ldo + n0 + c, f, p, row0, left - c, buf, lane);
    } else {
      uint4 w[8];
      auto two = [](uint32_t lo, uint32_t hi) { return pack_bf16(__uint_as_float(lo), __uint_as_float(hi)); };
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 8 * j;
        w[j] = make_uint4(two(v[i], v[i + 2]), two(v[i + 1], v[i + 3]), two(v[i + 4], v[i + 6]),
                          two(v[i + 5], v[i + 7]));
        w[4 + j] = make_uint4(two(x[i], x[i + 2]), two(x[i + 1], x[i + 3]), two(x[i + 4], x[i + 6]),
                              two(x[i + 5], x[i + 7]));
      }
      store_rows(buf, m, n0 + c, row0, 0, w, false, lane);
    }
  }
  if (++a == 2) a = 0, aph ^= 1u;
  return true;
}

// Sixteen codes times their scale as BF16, exactly (up to BF16's range); of each four columns the
// second and third change places.  A code's bits in BF16's places are its value times 2^-120,
// subnormal ones too, so that one multiplication does, but for RARE ones.
__device__ __forceinline__ bool rare_codes(const uint4& w, uint32_t byte) {  // NaN; scales above 2^7
  constexpr uint32_t low = 0x7F7F7F7Fu, one = 0x01010101u;
  const uint32_t nan =
      ((w.x & low) + one) | ((w.y & low) + one) | ((w.z & low) + one) | ((w.w & low) + one);
  return (nan & 0x80808080u) || byte > 134u;
}
template <bool RARE>
__device__ __forceinline__ void codes_to_bf16(const uint4& codes, uint32_t byte, uint32_t (&o)[8]) {
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (RARE) {
      const float s = scale_value(byte);
      float f[4];
      decode2(w[i] & 0xFFFFu, f[0], f[1]);
      decode2(w[i] >> 16, f[2], f[3]);
      o[2 * i] = pack_bf16(f[0] * s, f[2] * s), o[2 * i + 1] = pack_bf16(f[1] * s, f[3] * s);
    } else {
      auto two = [](const uint32_t& bits) { return *reinterpret_cast<const __nv_bfloat162*>(&bits); };
      const __nv_bfloat162 s = two((byte + 120u) * 0x00800080u);  // 2^(byte - 7)
      const __nv_bfloat162 a = __hmul2(two((w[i] << 4 & 0x07F007F0u) | (w[i] << 8 & 0x80008000u)), s);
      const __nv_bfloat162 b = __hmul2(two((w[i] >> 4 & 0x07F007F0u) | (w[i] & 0x80008000u)), s);
      o[2 * i] = *reinterpret_cast<const uint32_t*>(&a), o[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
}

// CTA r of a pair stages columns 128r .. of the tile's part of dy and its half of x's and
// holds rows 128r .. of the accumulator.  Both CTAs' copies of a stage complete on the even
// CTA's `full` barrier; its warp 1 issues the pair's MMAs and commits "stage read" and
// "accumulator final" to both CTAs.  Every wait is bounded: on a timeout the kernel flags
// the status word, waits (bounded) for what it started, frees its tensor memory and returns.
//
// With EIGHT x's operand comes from its codes: warp 2 copies 64 tokens x 128 codes at a time, and the
// converting warps write them as BF16 in the order of a bulk-tensor copy with the 128-byte
// swizzle; `full` then counts their arrivals too.
template <int PLANES, bool EIGHT>
__global__ void __launch_bounds__(kThreads<EIGHT>, 1)
    dw8_kernel(const __grid_constant__ Dw8Gemm p, const __grid_constant__ Dw8Maps maps) {
  constexpr int S = kStages<PLANES, EIGHT>;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // 128-byte swizzle atoms: 1024-byte aligned
  const uint32_t outs = base + 12 * kOperand;    // the epilogue warps' buffers
  const uint32_t bars = outs + kEpiWarps * kOutBytes;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (kMaxStages + s); };
  auto tfull = [&](int a) { return bars + 8u * (2 * kMaxStages + a); };
  auto tempty = [&](int a) { return bars + 8u * (2 * kMaxStages + 2 + a); };
  const uint32_t drain = bars + 8u * (2 * kMaxStages + 4);
  const uint32_t codes = base + 10 * kOperand;
  auto cfull = [&](int c) { return bars + 8u * (2 * kMaxStages + 5 + c); };
  auto cempty = [&](int c) { return bars + 8u * (2 * kMaxStages + 5 + kCodeTiles + c); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + (bars - raw) + kNumBars * 8);
  const uint32_t rank = cluster_ctarank() & 1u;
  const bool even = rank == 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  auto tell = [&](int g, int i) {
    return bars + 8u * (2 * kMaxStages + 5 + 2 * kCodeTiles + g * kTellSlots + i);
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), EIGHT ? 2 + kCvtWarps / kCvtGroups : 1);
      mbar_init(empty(s), 1);
    }
    if (EIGHT)
      for (int i = 0; i < kCvtGroups * kTellSlots; ++i) mbar_init(tell(0, i), kCvtWarps / kCvtGroups);
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull(a), 1);
      mbar_init(tempty(a), 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    if (EIGHT)
      for (int c = 0; c < kCodeTiles; ++c) {
        mbar_init(cfull(c), 1);
        mbar_init(cempty(c), kCvtWarps / kCvtGroups);
      }
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_addr(tmem_slot), kTmemCols);
    tmem_relinquish_pair();
  }
  __syncwarp();
  tc_fence_before_sync();
  cluster_sync();
  tc_fence_after_sync();
  pdl_wait();
  const uint32_t tmem =
      even ? *tmem_slot : ld_shared_cluster_u32(mapa_shared(smem_addr(tmem_slot), 0));
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == 0) {
      // ---------------------------------------------------------- copy issuer
      if (lane == 0) {
        prefetch_tmap(&maps.dy), prefetch_tmap(&maps.x);
        int s = 0, issued = 0;
        uint32_t ph = 0;
        const uint32_t full_even = even ? full(0) : mapa_shared(full(0), 0);
        bool on = true;
        Unit u;
        for (int k = 0; on && unit_at(p, pair, pairs, k, u); ++k) {
          int tm, tn;
          tile_at(p, u.tile, tm, tn);
          const int m0 = tm * kTile + (int)rank * 128;
          const int n0 = tn * p.tile_n + u.col + (int)rank * (u.cols / 2);
          const bool wide = u.cols > 128;
          const uint32_t tx = 2 * (PLANES * kOperand + (EIGHT ? 0 : (uint32_t)(u.cols / 2) * kBK * 2));
          for (int kt = u.kt0; kt < u.kt1; ++kt) {
            if ((p.debug_stop >= 0 && issued >= p.debug_stop) ||
                !wait_phase(empty(s), ph ^ 1u, p, kStatusTimeoutEmpty)) {
              on = false;
              break;
            }
            const uint32_t st = base + s * kStageBytes<PLANES>;
            if (even) mbar_arrive_expect_tx(full(s), tx);
            const uint32_t fb = full_even + 8u * s;
#pragma unroll
            for (int i = 0; i < PLANES; ++i)
              load_operand<true>(st + i * kOperand, &maps.dy, m0, kt, i, fb);
            if (!EIGHT) load_operand<true>(st + PLANES * kOperand, &maps.x, n0, kt, 0, fb, wide);
            ++issued;
            if (++s == S) s = 0, ph ^= 1u;
          }
        }
        // leave only after the copies started here have landed (the odd CTA sees the MMAs
        // release the stages they read)
        for (int d = 0, pending = min(issued, S); d < pending; ++d) {
          if (--s < 0) s = S - 1, ph ^= 1u;
          if (!wait_phase(even ? full(s) : empty(s), ph, p, kStatusTimeoutDrain)) break;
        }
      }
      __syncwarp();
    } else if (warp == 1 && even) {
      // ---------------------------------------------------------- MMA issuer
      if (lane == 0) {
        int s = 0, a = 0;
        uint32_t ph = 0, aph = 0;
        const uint32_t empty_odd = mapa_shared(empty(0), 1), tfull_odd = mapa_shared(tfull(0), 1);
        const uint32_t a0 = desc_lo<true>(base), b0 = desc_lo<true>(base + PLANES * kOperand);
        constexpr uint32_t step = kDescStep<true>;
        bool on = true;
        Unit u;
        for (int k = 0; on && unit_at(p, pair, pairs, k, u); ++k) {
          const int groups = groups_of(p, u.kt1 - u.kt0);
          const uint32_t idesc = idesc_bf16(kTile, u.cols, true, true);
          for (int g = 0; on && g < groups; ++g) {
            if (!(on = wait_phase<true>(tempty(a), aph ^ 1u, p, kStatusTimeoutTmem))) break;
            tc_fence_after_sync();
            const uint32_t d = tmem + (uint32_t)(a * kTile);
            const int kts = min(p.group, u.kt1 - u.kt0 - g * p.group);
            for (int it = 0; it < kts; ++it) {
              if (!(on = wait_phase<EIGHT>(full(s), ph, p, kStatusTimeoutFull))) break;
              tc_fence_after_sync();
              const uint32_t off = (uint32_t)s * (kStageBytes<PLANES> >> 4);
#pragma unroll
              for (int i = PLANES - 1; i >= 0; --i)
#pragma unroll
                for (int kk = 0; kk < kBK / 16; ++kk)
                  mma_bf16_pair(d, a0 + off + i * (kOperand >> 4) + kk * step, b0 + off + kk * step,
                                idesc, (it > 0 || i < PLANES - 1 || kk > 0) ? 1u : 0u);
              mma_commit_pair(empty(s));
              mma_commit_pair(empty_odd + 8u * s);
              if (++s == S) s = 0, ph ^= 1u;
            }
            if (!on) break;
            mma_commit_pair(tfull(a));
            mma_commit_pair(tfull_odd + 8u * a);
            if (++a == 2) a = 0, aph ^= 1u;
          }
        }
        mma_commit_pair(drain);
        wait_phase(drain, 0, p, kStatusTimeoutTmem);
      }
      __syncwarp();
    } else if (EIGHT && warp == 2) {
      // ---------------------------------------------------------- copies of codes
      if (lane == 0) {
        prefetch_tmap(&maps.x);
        int c = 0, issued = 0;
        uint32_t ph = 0;
        bool on = true;
        Unit u;
        for (int k = 0; on && unit_at(p, pair, pairs, k, u); ++k) {
          int tm, tn;
          tile_at(p, u.tile, tm, tn);
          const int n0 = tn * p.tile_n + u.col + (int)rank * (u.cols / 2);
          for (int kt = u.kt0; kt < u.kt1; ++kt) {
            if (!(on = wait_phase(cempty(c), ph ^ 1u, p, kStatusTimeoutEmpty))) break;
            mbar_arrive_expect_tx(cfull(c), u.cols > 128 ? kCodeBytes : kCodeBytes / 2);
            tma_load_3d(codes + c * kCodeBytes, &maps.x, n0, kt * kBK, 0, cfull(c));
            if (u.cols > 128)
              tma_load_3d(codes + c * kCodeBytes + kCodeBytes / 2, &maps.x, n0 + 64, kt * kBK, 0, cfull(c));
            ++issued;
            if (++c == kCodeTiles) c = 0, ph ^= 1u;
          }
        }
        for (int d = 0, pending = min(issued, kCodeTiles); d < pending; ++d) {
          if (--c < 0) c = kCodeTiles - 1, ph ^= 1u;
          if (!wait_phase(cfull(c), ph, p, kStatusTimeoutDrain)) break;
        }
      }
      __syncwarp();
    } else if (EIGHT && !even) {
      // ---------------------------------------------------------- the odd CTA's converted tiles
      // Warps 1 and 3 tell the even CTA of a group's tiles each: its MMAs read them in this CTA's
      // shared memory.  The converting warps' writes (and their fence.proxy.async) reach the MMAs'
      // issuer by two links: the release and acquire of `tell` within this CTA, then the fence here
      // and the issuer's acquire, both for the cluster.  The fence takes about 1400 cycles, more
      // than a k tile does; so each group has a thread of its own for it, and one fence does for
      // all of the tiles that are there.
      if (lane == 0) {
        const int group = warp >> 1;
        const uint32_t full_even = mapa_shared(full(0), 0);
        int s = group, i = 0;
        uint32_t ph = 0;
        unsigned seen = 0;
        bool on = true;
        Unit u;
        for (int k = 0; on && unit_at(p, pair, pairs, k, u); ++k) {
          int kt = u.kt0 + (int)((group - seen) & (kCvtGroups - 1));
          seen += u.kt1 - u.kt0;
          while (kt < u.kt1) {
            if (!(on = wait_phase(tell(group, i), ph, p, kStatusTimeoutFull))) break;
            int n = 0;
            do {
              ++n, kt += kCvtGroups;
              if (++i == kTellSlots) i = 0, ph ^= 1u;
            } while (n < kTellSlots && kt < u.kt1 && mbar_test_wait(tell(group, i), ph));
            fence_cluster();
            for (; n; --n) {
              mbar_arrive_remote_relaxed(full_even + 8u * s);
              if ((s += kCvtGroups) >= S) s -= S;
            }
          }
        }
      }
      __syncwarp();
    }
  } else if (EIGHT && warp >= 4 + kEpiWarps) {
    // ---------------------------------------------------------- codes to BF16
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCvtRegs));
    constexpr int G = kCvtGroups, N = 2 * G;  // every G-th k tile is a group's; chunks a thread
    constexpr int kRows = kBK / G;            // tokens that a group's threads hold at a time
    const int group = (warp - 4 - kEpiWarps) / (kCvtWarps / G);
    const int t = (threadIdx.x - (128 + 32 * kEpiWarps)) & (256 / G - 1);
    // 16 columns of tokens `token` and (with two groups) token + 32, in either half of the columns:
    // chunk h is of half h & 1.  Eight lanes' units of 16 bytes lie in eight different places of
    // 128 bytes, here and there.
    const int chunk = t & 3, token = t >> 2;
    const uint32_t from0 = codes + token * 64 + chunk * 16;
    const uint32_t to0 = base + PLANES * kOperand + token * 128 + ((2 * chunk ^ (token & 7)) << 4);
    int s = group, c = group, told = 0;
    uint32_t ph = 0, cph = 0;
    unsigned seen = 0;
    bool on = true;
    Unit u;
    for (int k = 0; on && unit_at(p, pair, pairs, k, u); ++k) {
      int tm, tn;
      tile_at(p, u.tile, tm, tn);
      const int col = tn * p.tile_n + u.col + (int)rank * (u.cols / 2) + 16 * chunk;
      const bool wide = u.cols > 128;
      int kt = u.kt0 + (int)((group - seen) & (G - 1));
      seen += u.kt1 - u.kt0;
      // the scales of this group's next k tile are on their way
      uint32_t b[N];
      int row = kt * kBK + token;
      const unsigned char* from = p.scales + row * p.lds + col / kScaleBlock;
      auto scales = [&] {
#pragma unroll
        for (int h = 0; h < N; ++h) {
          b[h] = 127u;
          if (row + kRows * (h >> 1) < p.tokens && col + 64 * (h & 1) < p.cols)
            b[h] = from[(h >> 1) * kRows * p.lds + (h & 1) * (64 / kScaleBlock)];
        }
      };
      scales();
      for (; kt < u.kt1; kt += G) {
        // both are asked for before either answer is waited for
        const bool here = mbar_try_wait(cfull(c), cph), clear = mbar_try_wait(empty(s), ph ^ 1u);
        if (!here) on = wait_phase(cfull(c), cph, p, kStatusTimeoutFull);
        if (!clear) on = wait_phase(empty(s), ph ^ 1u, p, kStatusTimeoutEmpty) && on;
        on = __all_sync(0xffffffffu, on);
        if (!on) break;
        uint4 q[N];
        bool rare = false;
#pragma unroll
        for (int h = 0; h < N; ++h) {
          q[h] = make_uint4(0, 0, 0, 0);
          if (wide || !(h & 1))
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(q[h].x), "=r"(q[h].y), "=r"(q[h].z), "=r"(q[h].w)
                         : "r"(from0 + c * kCodeBytes + (h & 1) * (kCodeBytes / 2) + (h >> 1) * kRows * 64));
        }
#pragma unroll
        for (int h = 0; h < N; ++h) rare = rare | rare_codes(q[h], b[h]);
        auto convert = [&](auto kind) {
#pragma unroll
          for (int h = 0; h < N; ++h) {
            uint32_t o[8];
            codes_to_bf16<kind.value>(q[h], b[h], o);
            const uint32_t to = to0 + s * kStageBytes<PLANES> + (h & 1) * (kOperand / 2) + (h >> 1) * kRows * 128;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(o[0]), "r"(o[1]),
                         "r"(o[2]), "r"(o[3]));
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to ^ 16u), "r"(o[4]), "r"(o[5]),
                         "r"(o[6]), "r"(o[7]));
          }
        };
        if (rare)
          convert(std::true_type());
        else
          convert(std::false_type());
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(cempty(c));
          mbar_arrive(even ? full(s) : tell(group, told));
        }
        if (++told == kTellSlots) told = 0;
        row += G * kBK, from += (long long)G * kBK * p.lds;
        scales();
        if ((s += G) >= S) s -= S, ph ^= 1u;
        if ((c += G) >= kCodeTiles) c -= kCodeTiles, cph ^= 1u;
      }
    }
  } else {
    // ---------------------------------------------------------- epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs<EIGHT>));
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t tmem_row = tmem + ((uint32_t)(32 * q) << 16);
    const uint32_t buf = outs + (uint32_t)(warp - 4) * kOutBytes;
    const uint32_t tempty_even = even ? 0u : mapa_shared(tempty(0), 0);
    int a = 0;
    uint32_t aph = 0;
    Unit u;
    for (int k = 0; unit_at(p, pair, pairs, k, u); ++k) {
      const int span = u.cols / 2;  // this warp's columns
      int tm, tn;
      tile_at(p, u.tile, tm, tn);
      const int rows = (int)rank * 4 + q, row0 = tm * kTile + 32 * rows;
      const int n0 = tn * p.tile_n + u.col + half * span;
      const int left = row0 < p.rows ? min(span, p.cols - n0) : 0;
      const uint32_t lane0 = tmem_row + (uint32_t)(half * span);
      if constexpr (EIGHT) {
        if (!put_bf16(p, u, &maps.out, lane0, span, rows, half, row0, n0, left, a, aph, tfull(0), tempty(0),
                      tempty_even, even, buf, lane))
          break;
      } else {
        float acc[128];
        if (!collect(p, acc, lane0, span, groups_of(p, u.kt1 - u.kt0), a, aph, tfull(0), tempty(0),
                     tempty_even, even, lane))
          break;
        if (left > 0 && u.slot >= 0)
          put_sums(p.part + sums_at(u.slot, rows, half, p.tile_n), acc, left, lane);
        else if (left > 0)
          put_tile(p, &maps.out, acc, row0, n0, left, buf, lane);
      }
    }
    if (lane == 0) stores_done();
  }

  __syncwarp();
  tc_fence_before_sync();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(*tmem_slot, kTmemCols);
  }
}

// The remaining tiles' results: their pieces' sums, added in the order of k.  Block (t, y, z)
// takes 32 of the columns and all 32 rows that one warp y of tile t left, four columns a warp;
// where a tile has more than kFewPieces pieces (MANY), 16 columns, and two warps each half of
// the pieces, one and the next in turns.  The results leave through shared memory, row by row.
constexpr int kFewPieces = 8;
template <bool MANY>
constexpr int kJoinCols = MANY ? 16 : 32;
template <typename T, bool MANY>
__global__ void __launch_bounds__(256) dw8_join_kernel(const __grid_constant__ Dw8Gemm p, int pairs) {
  constexpr int kCols = kJoinCols<MANY>, kPitch = kCols + 4;
  __shared__ __align__(16) float sm[(MANY ? 2 : 1) * 32 * kPitch];
  pdl_launch_dependents();
  const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int span = p.tile_n / 2, rows = blockIdx.y >> 1, half = blockIdx.y & 1;
  const int j0 = blockIdx.z * kCols;  // the block's first column
  int tm, tn;
  tile_at(p, p.full * pairs + t, tm, tn);
  const int r0 = tm * kTile + 32 * rows, c0 = tn * p.tile_n + half * span + j0;
  const int left = min(min(span - j0, kCols), p.cols - c0);
  if (r0 >= p.rows || left <= 0) return;
  const unsigned from = (unsigned)t * p.span, first = from / p.piece;
  const unsigned n = (from + p.k_tiles - 1) / p.piece - first + 1;
  // a piece that began before the tile: its second fragment
  const unsigned shift = first * p.piece < from ? 1 : 0;
  const size_t step = sums_at(2, 0, 0, p.tile_n);
  const float* at = p.part + sums_at(2 * first, rows, half, p.tile_n) + j0 * 32 + lane * 4;
  pdl_wait();
  const int j = MANY ? warp & 3 : warp, mine = MANY ? warp >> 2 : 0;  // columns 4 j ..
  if (4 * j < left) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    auto sum = [&](unsigned i) {
      return *reinterpret_cast<const float4*>(at + j * 128 + i * step +
                                              (i == 0 && shift ? sums_at(1, 0, 0, p.tile_n) : 0));
    };
    auto add = [&](const float4& v) { s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w; };
    if constexpr (MANY) {
#pragma unroll 8
      for (unsigned i = mine; i < n; i += 2) add(sum(i));
    } else {
      float4 v[kFewPieces];
#pragma unroll
      for (int i = 0; i < kFewPieces; ++i)
        if (i < n) v[i] = sum(i);
#pragma unroll
      for (int i = 0; i < kFewPieces; ++i)
        if (i < n) add(v[i]);
    }
    *reinterpret_cast<float4*>(sm + (mine * 32 + lane) * kPitch + 4 * j) = s;
  }
  __syncthreads();
  // the rows: 4 columns a lane where they can be written together
  const int rows_left = min(32, p.rows - r0);
  T* out = static_cast<T*>(p.out) + (long long)r0 * p.ldo + c0;
  const bool vec = (reinterpret_cast<uintptr_t>(p.out) | (uintptr_t)(p.ldo * sizeof(T))) % (4 * sizeof(T)) == 0;
  constexpr int kLanes = kCols / 4;  // lanes a row
  for (int i = threadIdx.x / kLanes; i < rows_left; i += 256 / kLanes) {
    const int c = (threadIdx.x % kLanes) * 4;
    float f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = sm[i * kPitch + c + e];
      if (MANY) f[e] += sm[(32 + i) * kPitch + c + e];
    }
    T* o = out + (long long)i * p.ldo + c;
    if (vec && c + 4 <= left) {
      if (p.accumulate) {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] += to_f32(o[e]);
      }
      if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float4*>(o) = make_float4(f[0], f[1], f[2], f[3]);
      else
        *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < left) o[e] = from_f32<T>(p.accumulate ? f[e] + to_f32(o[e]) : f[e]);
    }
  }
}

// ---------------------------------------------------------------- operands

// Bound: bytes (4096 x 4096 8 us, 6.4 TB/s).
// x from its 8-bit form to BF16 rows, and (DY) dy to `planes` BF16 planes where it cannot be
// read as it is.  The first blocks work on x.
struct Prepare {
  Walk wx, wd;
  int tokens;
  Rows8 k;
  int width;
  Bf16* x;
  long long ldx;
  const void* dy;
  long long lddy;
  int outs, planes;
  Bf16* d;
  long long ldd;
};

template <typename T, bool DY>
__global__ void __launch_bounds__(256) dw8_prepare_kernel(const __grid_constant__ Prepare p) {
  constexpr int V = kVec<T>;
  pdl_launch_dependents();
  const bool second = DY && blockIdx.x >= p.wx.blocks;
  const Walk& walk = second ? p.wd : p.wx;
  const Places at(walk, second ? blockIdx.x - p.wx.blocks : blockIdx.x);
  pdl_wait();
  auto in = [&](int u) { return at.row_of(u) < walk.rows && at.chunk_of(u) < walk.chunks; };
  if (!second) {
    Codes<8> k[kPasses];
    uint32_t byte[kPasses];
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
      const long long row = at.row_of(u);
      const int c = at.chunk_of(u);
      if (in(u)) {
        load_codes<8, true>(k[u], p.k, row, c, p.width);
        byte[u] = p.k.s[row * p.k.lds + c / (kScaleBlock / 8)];
      }
    }
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
      if (in(u)) {
        const float s = scale_value(byte[u]);
        float f[8];
        k[u].get(f);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= s;
        Pack<Bf16, 8> o;
        o.set(f);
        o.store(p.x + at.row_of(u) * p.ldx + at.chunk_of(u) * 8);
      }
    }
  } else if constexpr (DY) {
    Fetched raw[kPasses];
    auto row_of = [&](int u) { return static_cast<const T*>(p.dy) + at.row_of(u) * p.lddy; };
#pragma unroll
    for (int u = 0; u < kPasses; ++u) fetch<T>(raw[u], row_of(u), at.chunk_of(u) * V, p.outs, in(u));
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
      Pack<T, V> k;
      finish<T>(k, raw[u], row_of(u), at.chunk_of(u) * V, p.outs, in(u));
      if (!in(u)) continue;
      Bf16* to = p.d + at.row_of(u) * p.ldd + at.chunk_of(u) * V;
      if constexpr (V == 8) {
        *reinterpret_cast<uint4*>(to) = k.u;
      } else {
        float f[4];
        k.get(f);
#pragma unroll
        for (int pl = 0; pl < 3; ++pl) {
          const uint32_t a = pl == 0 ? split_plane<true>(f[0], f[1]) : split_plane<false>(f[0], f[1]);
          const uint32_t b = pl == 0 ? split_plane<true>(f[2], f[3]) : split_plane<false>(f[2], f[3]);
          *reinterpret_cast<uint2*>(to + (long long)pl * p.tokens * p.ldd) = make_uint2(a, b);
        }
      }
    }
  }
}

// ----------------------------------------------------------------- host side

int check(int dtype, int tokens, int outs, int width) {
  if (!type_ok(dtype)) return B2G_ERR_INVALID_TYPE;
  if (tokens < 0 || outs < 0 || width < 0 || tokens > kMaxLength || outs > kMaxLength ||
      width > kMaxLength)
    return B2G_ERR_INVALID_DIM;
  return 0;
}

// How the tiles are shared out, and where the operands' copies and the sums stand in the
// workspace.
struct Layout {
  int planes;
  bool copy_dy;
  long long ldx, ldd;
  int tile_n, tiles_m, tiles_n, k_tiles, pairs, full, rest;
  long long piece, span;
  bool split, halves;
  bool eight;      // x from its codes, without a copy
  long long cost;  // of a pair's work, in cycles
  size_t x, d, part, total;
};

// Cycles of a k tile: BF16 its copies (64 bytes a cycle and SM), with EIGHT the conversion and its
// announcement to the other CTA, FP32 its three products.
long long k_tile_cost(int planes, int tile_n, bool eight) {
  return planes == 3 ? 1900 : eight ? 1150 : kTile + tile_n;
}
// Cycles of a whole BF16 tile's way out, behind which the next one's products go on.  Without them
// 192 tokens on 4096 x 4096 were prepared (17.2 us; 15.8 from the codes).
constexpr long long kOutCost = 12;  // a column
// The launch that prepares x, and the bytes that it moves in a cycle.
constexpr long long kPrepareCost = 4000, kPrepareBytes = 3200;
// Halves of a tile: their products take as long as the whole one's (2048 tokens on 1024 x 1024
// BF16: 17.0 us so), but there is half as much to write at the end (300 on 512 x 256: 7.4 us for
// 8.1; 1000 on 1025 x 777: 15.6 for 17.5).
constexpr long long kHalfSaves = 1500;
// Leaving sums instead of a result, and a second time; the launch that adds them, and for each
// piece.  2048 tokens on 1024 x 1024 BF16, us without the operands' preparation: whole tiles
// 14.3; each cut in 2, 3, 4: 14.7, 13.8, 13.1; one piece a pair across tiles 15.3.
constexpr long long kSumCost = 2200, kSecondCost = 4500, kJoinCost = 3000, kJoinPiece = 90;

// false: more tiles than can be counted.
bool layout(int dtype, int tokens, int outs, int width, const void* dy, long long lddy, bool eight, Layout& l) {
  l.eight = eight;
  l.planes = dtype == B2G_F32 ? 3 : 1;
  l.copy_dy = dtype == B2G_F32 || !vec16(dy) || lddy % 8;
  // the copies' rows on 128-byte lines: off them a k tile of BF16 takes twice as long
  l.ldx = (long long)round_up(width, 64), l.ldd = (long long)round_up(outs, 64);
  l.tile_n = width > 128 ? 256 : 128;
  l.k_tiles = (int)ceil_div(tokens, kBK);
  l.tiles_m = (int)ceil_div(outs, kTile), l.tiles_n = (int)ceil_div(width, l.tile_n);
  const long long tiles = (long long)l.tiles_m * l.tiles_n;
  if (tiles > 0x3fffffffLL) return false;
  l.full = (int)(tiles / kPairs), l.rest = (int)(tiles % kPairs);
  // The rest: a tile a pair; half a tile a pair; each tile cut into the same pieces; or all of
  // their k cut into one piece a pair, some of which then lie across two tiles and leave two sums.
  l.piece = l.span = l.k_tiles, l.split = l.halves = false;
  long long pieces = l.rest;
  const long long kt = k_tile_cost(l.planes, l.tile_n, eight);
  const long long out = kOutCost * l.tile_n;
  l.cost = l.full * (l.k_tiles * kt > out ? l.k_tiles * kt : out);
  if (l.rest) {
    long long best = l.k_tiles * kt;
    const long long half = best - kHalfSaves;
    if (l.tile_n == 256 && 2 * l.rest <= kPairs) best = half, l.halves = true, pieces = 2 * l.rest;
    const long long slices = kPairs / l.rest;
    for (long long s = 2; s <= slices && s <= l.k_tiles; ++s) {
      const long long len = ceil_div(l.k_tiles, s), used = ceil_div(l.k_tiles, len);
      const long long cost = len * kt + kSumCost + kJoinCost + l.rest * used * kJoinPiece;
      if (cost < best)
        best = cost, l.piece = len, l.span = len * used, l.split = true, l.halves = false, pieces = l.rest * used;
    }
    const long long len = ceil_div((long long)l.rest * l.k_tiles, kPairs);
    const long long n = ceil_div((long long)l.rest * l.k_tiles, len);
    const long long cost = len * kt + kSumCost + kSecondCost + kJoinCost + (n + l.rest) * kJoinPiece;
    if (len < l.k_tiles && cost < best)
      best = cost, l.piece = len, l.span = l.k_tiles, l.split = true, l.halves = false, pieces = n;
    l.cost += best;
  }
  l.pairs = l.full ? kPairs : (int)pieces;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += round_up(bytes, 256);
    return o;
  };
  l.x = eight ? 0 : take((size_t)tokens * l.ldx * 2);
  l.d = l.copy_dy ? take((size_t)l.planes * tokens * l.ldd * 2) : 0;
  l.part = l.split ? take((size_t)2 * pieces * kTile * l.tile_n * 4) : 0;
  l.total = at;
  return true;
}

// {width, tokens} codes, boxes of 64 x kBK.
int encode_codes(CUtensorMap* m, const void* codes, int width, int tokens, long long ldq) {
  auto enc = tensor_map_encoder();
  if (!enc) return B2G_ERR_TENSOR_MAP;
  cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)tokens, 1}, strides[2] = {(cuuint64_t)ldq, 16};
  cuuint32_t box[3] = {64, kBK, 1}, estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(codes), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS ? 0 : B2G_ERR_TENSOR_MAP;
}

// Either way's layout; x is read from its codes where that costs less than preparing it, which
// takes a launch (there is one all the same where dy has to be copied).  Us, prepared and from the
// codes: 300 tokens on 512 x 256 7.3 and 7.0; 5844 on 128 x 6944 43 and 33; 16384 on 512 x 8192
// 141 and 143; 8192 on 2048 x 2048 48.5 and 72; 4096 on 4096 x 4096 86 and 127.  Codes off the
// 16-byte boundaries are prepared in any case.
bool layouts(int dtype, int tokens, int outs, int width, const void* dy, long long lddy, Layout& prepared,
             Layout& l) {
  if (!layout(dtype, tokens, outs, width, dy, lddy, false, prepared)) return false;
  l = prepared;
  if (prepared.planes > 1 || prepared.k_tiles > kGroupK / kBK) return true;
  layout(dtype, tokens, outs, width, dy, lddy, true, l);
  if (l.cost >= prepared.cost + (l.copy_dy ? 0 : kPrepareCost) + (long long)tokens * width / kPrepareBytes * 3)
    l = prepared;
  return true;
}
bool codes_fit(const void* codes, long long ldq) { return vec16(codes) && ldq % 16 == 0; }

// Both layouts for a workspace query; without a product they need nothing.
int query(int dtype, int tokens, int outs, int width, const void* dy, long long lddy, const size_t* bytes,
          Layout& prepared, Layout& l) {
  const int rc = check(dtype, tokens, outs, width);
  if (rc) return rc;
  if (!bytes) return B2G_ERR_NULL;
  l = prepared = {};
  if (!tokens || !outs || !width) return 0;
  return layouts(dtype, tokens, outs, width, dy, lddy, prepared, l) ? 0 : B2G_ERR_INVALID_DIM;
}

template <int PLANES, bool EIGHT>
int launch(const Dw8Gemm& g, const Dw8Maps& maps, int pairs, const TrainDevice& d, cudaStream_t st) {
  static std::atomic<int> done[64];
  if (d.dev < 0 || d.dev >= 64) return B2G_ERR_DEVICE;
  if (!done[d.dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(dw8_kernel<PLANES, EIGHT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmemBytes) != cudaSuccess)
      return B2G_ERR_CUDA;
    // the warps' shares of registers have to be there at the start, or raising them never ends
    constexpr int regs = 128 * kIssueRegs + 32 * kEpiWarps * kEpiRegs<EIGHT> + (EIGHT ? 32 * kCvtWarps * kCvtRegs : 0);
    cudaFuncAttributes has;
    if (cudaFuncGetAttributes(&has, dw8_kernel<PLANES, EIGHT>) != cudaSuccess ||
        has.numRegs * kThreads<EIGHT> < regs)
      return B2G_ERR_CUDA;
    done[d.dev].store(1, std::memory_order_release);
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.blockDim = dim3(kThreads<EIGHT>);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  void* args[] = {const_cast<Dw8Gemm*>(&g), const_cast<Dw8Maps*>(&maps)};
  return launch_code(cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(&dw8_kernel<PLANES, EIGHT>), args));
}

}  // namespace
}  // namespace b2g

using namespace b2g;

extern "C" {

int b2g_linear_dweight8_workspace_size(int dtype, int tokens, int outs, int width, const void* dy,
                                       long long lddy, size_t* bytes) {
  Layout l, prepared;
  const int rc = query(dtype, tokens, outs, width, dy, lddy, bytes, prepared, l);
  if (!rc) *bytes = l.total > prepared.total ? l.total : prepared.total;
  return rc;
}

int b2g_linear_dweight8_workspace_size_ex(int dtype, int tokens, int outs, int width, const void* dy,
                                          long long lddy, const void* codes, long long ldq,
                                          size_t* bytes) {
  Layout l, prepared;
  const int rc = query(dtype, tokens, outs, width, dy, lddy, bytes, prepared, l);
  if (!rc) *bytes = codes_fit(codes, ldq) ? l.total : prepared.total;
  return rc;
}

int b2g_linear_dweight8(int dtype, int tokens, int outs, int width, const void* dy, long long lddy,
                        const void* codes, long long ldq, const void* scales, long long lds,
                        int accumulate, void* dw, long long lddw, void* workspace,
                        size_t workspace_bytes, void* stream) {
  int rc = check(dtype, tokens, outs, width);
  if (rc) return rc;
  auto least = [](int n) { return n > 1 ? n : 1; };
  if (lddy < least(outs) || ldq < least(width) || lds < scale_count(least(width)) ||
      lddw < least(width))
    return B2G_ERR_INVALID_LD;
  if (outs == 0 || width == 0 || (tokens == 0 && accumulate)) return 0;
  if (!dw || (tokens > 0 && (!dy || !codes || !scales))) return B2G_ERR_NULL;
  TrainDevice d;
  rc = train_device(&d);
  if (rc) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool f32 = dtype == B2G_F32;
  const size_t es = type_size(dtype);
  if (tokens == 0)
    return cudaMemset2DAsync(dw, lddw * es, 0, width * es, outs, st) == cudaSuccess ? 0 : B2G_ERR_CUDA;
  Layout l, prepared;
  if (!layouts(dtype, tokens, outs, width, dy, lddy, prepared, l)) return B2G_ERR_INVALID_DIM;
  if (!codes_fit(codes, ldq)) l = prepared;
  if (l.total && (!workspace || !vec16(workspace) || workspace_bytes < l.total)) return B2G_ERR_WORKSPACE;
  unsigned char* ws = static_cast<unsigned char*>(workspace);

  Dw8Gemm g = {};
  g.rows = outs, g.cols = width;
  g.tiles_m = l.tiles_m, g.tiles_n = l.tiles_n, g.k_tiles = l.k_tiles, g.tile_n = l.tile_n;
  g.full = l.full, g.rest = l.rest, g.halves = l.halves, g.piece = (unsigned)l.piece, g.span = (unsigned)l.span, g.split = l.split;
  g.part = reinterpret_cast<float*>(ws + l.part);
  // what adds up in tensor memory, which truncates, before FP32 registers take over: FP32 256
  // tokens (48 steps; error of dw 5e-7 at 1000 x 1025 x 777, the plain form's 5.7e-7); BF16
  // what its own rounding hides
  g.group = f32 ? 4 : kGroupK / kBK;
  g.wait_limit_ns = d.wait_limit_ns, g.debug_stop = d.debug_stop, g.status = d.status;
  g.out = dw, g.ldo = lddw, g.out_bf16 = !f32, g.accumulate = accumulate != 0;
  // a bulk-tensor store writes whole 16-byte units, those past the last column too; and it
  // adds in the output's type: right for FP32 only
  g.out_tma = vec16(dw) && vec16_ld(lddw, dtype) && vec16_ld(width, dtype) && !(accumulate && !f32);
  g.add = accumulate != 0;
  g.scales = static_cast<const unsigned char*>(scales), g.lds = lds, g.tokens = tokens;

  Bf16* const x = reinterpret_cast<Bf16*>(ws + l.x);
  Bf16* const planes = reinterpret_cast<Bf16*>(ws + l.d);
  if (!l.eight || l.copy_dy) {
    Prepare q = {};
    q.tokens = tokens;
    q.k = Rows8{static_cast<unsigned char*>(const_cast<void*>(codes)), ldq,
                static_cast<unsigned char*>(const_cast<void*>(scales)), lds, 0};
    q.width = width, q.x = x, q.ldx = l.ldx;
    q.k.vec = codes_vec(q.k, 8);
    q.dy = dy, q.lddy = lddy, q.outs = outs, q.planes = l.copy_dy ? l.planes : 0;
    q.d = planes, q.ldd = l.ldd;
    if (!l.eight) q.wx = walk_of(tokens, (int)ceil_div(width, 8), 1);
    if (l.copy_dy) q.wd = walk_of(tokens, (int)ceil_div(outs, f32 ? 4 : 8), 1);
    if (q.wx.blocks + q.wd.blocks > 0x7fffffffLL) return B2G_ERR_INVALID_DIM;
    const dim3 grid((unsigned)(q.wx.blocks + q.wd.blocks));
    rc = launch_code(f32 ? launch_train(dw8_prepare_kernel<float, true>, grid, dim3(256), 0, st, q)
                     : l.copy_dy ? launch_train(dw8_prepare_kernel<Bf16, true>, grid, dim3(256), 0, st, q)
                                 : launch_train(dw8_prepare_kernel<Bf16, false>, grid, dim3(256), 0, st, q));
    if (rc) return rc;
  }
  Dw8Maps maps = {};
  rc = l.copy_dy ? encode_rows(&maps.dy, false, planes, outs, tokens, l.ldd, l.planes,
                               (long long)tokens * l.ldd, 64)
                 : encode_rows(&maps.dy, false, dy, outs, tokens, lddy, 1, 0, 64);
  if (!rc)
    rc = l.eight ? encode_codes(&maps.x, codes, width, tokens, ldq)
                 : encode_rows(&maps.x, false, x, width, tokens, l.ldx, 1, 0, 64);
  if (!rc && g.out_tma) rc = encode_rows(&maps.out, f32, dw, width, outs, lddw, 1, 0, 32);
  if (rc) return rc;
  rc = f32       ? launch<3, false>(g, maps, l.pairs, d, st)
       : l.eight ? launch<1, true>(g, maps, l.pairs, d, st)
                 : launch<1, false>(g, maps, l.pairs, d, st);
  if (rc || !l.split) return rc;
  // of a tile; one more where pieces lie across tiles
  const bool many = ceil_div(l.k_tiles, l.piece) + (l.span % l.piece ? 1 : 0) > kFewPieces;
  const dim3 blocks((unsigned)l.rest, 16, (unsigned)(l.tile_n / 2 / (many ? kJoinCols<true> : kJoinCols<false>)));
  auto join = [&](auto kernel) {
    return launch_code(launch_train(kernel, blocks, dim3(256), 0, st, g, l.pairs));
  };
  if (f32) return many ? join(dw8_join_kernel<float, true>) : join(dw8_join_kernel<float, false>);
  return many ? join(dw8_join_kernel<Bf16, true>) : join(dw8_join_kernel<Bf16, false>);
}

}  // extern "C"
