// xent.cu -- softmax cross entropy of a linear layer and its gradients
// (b2g_linear_xent, b2g_linear_xent_backward in include/b2g_train.h), on the
// 5th-generation tensor cores.
//
// With z = h w^T (tokens x vocab):
//   forward   lse_i = log sum_j exp z_ij,  loss_i = lse_i - z_{i,t_i}
//   backward  dz_ij = g_i (exp(z_ij - lse_i) - [j == t_i]),  dh = dz w,  dw = dz^T h
// z is never stored.  The forward product's epilogue keeps, for each row and
// each 128 columns, the maximum and the sum of the exponentials below it, which a
// second kernel joins; the backward pass forms z again for a piece of the
// vocabulary, turns it into dz on its way out of tensor memory, and multiplies
// that piece by w and by h.  So a training step costs 8 tokens vocab width
// operations where one that stores z costs 6, and no tokens x vocab array in
// FP32.
//
// One kernel makes all four products, C = A B^T over k, on 256 x 256 tiles of a
// CTA pair (tcgen05.mma.cta_group::2, BF16 operands, FP32 accumulators in tensor
// memory, double buffered).  What differs is which index of an operand is
// contiguous in memory and what happens to a finished tile:
//   kStats  h w^T, k = width: row statistics and the target's logit
//   kDz     h w^T, k = width: dz, rounded to BF16
//   kProd   both gradients in one launch, whose tiles fill the CTA pairs together:
//           job 0: dz w,   k = vocab piece: w's columns contiguous ("MN-major" B)
//           job 1: dz^T h, k = tokens: both operands MN-major
// so no transposed copy of anything is made.  FP32 operands are split into three
// BF16 planes, x = x0 + x1 + x2 to 24 bits, of which the six products whose weight is at
// least 2^-16 of the largest are added up (the next ones are below FP32's rounding); dz
// is stored as three planes the same way.  The three planes of a k tile are in shared
// memory together and each is copied there once, half the copies that fetching both
// planes of each product would take.
//
// Bound: the tensor cores (from a few hundred tokens up), or reading w (few
// tokens).  2048 x 32768 x 2048 BF16: the loss 172 us, its gradients 514 us, 1.60 PFLOP/s
// over all four products.
#include <atomic>

#include "pair.cuh"

namespace b2g {
namespace {

enum Mode { kStats, kDz, kProd };

constexpr int kStages = 6;
constexpr int kThreads = 128 + 32 * kEpiWarps;  // warp 0 copies, warp 1 multiplies, 2 and 3 idle
// Registers: the block starts with 168 a thread (64,512 of the SM's 65,536); the
// first warpgroup gives up its share so that the epilogue's threads can hold 128
// sums each: 128 * 72 + 256 * 216 = 64,512.
constexpr int kIssueRegs = 72, kEpiRegs = 216;
constexpr uint32_t kATile = 128 * kBK * 2;     // a CTA's 128 rows of A: 16 KB
constexpr uint32_t kBTile = 128 * kBK * 2;     // its 128 rows of B
constexpr uint32_t kStageBytes = kATile + kBTile;
constexpr uint32_t kStageStep = kStageBytes >> 4;  // in descriptors
static_assert(kStages % 3 == 0, "a k tile's three planes lie in stages of one phase");
constexpr int kNumBars = 2 * kStages + 5;
constexpr int kSmemBytes =
    kStages * kStageBytes + kEpiWarps * kOutBytes + 1024 + kNumBars * 8 + 16;
constexpr uint32_t kTmemCols = 2 * kTile;

struct XentGemm {
  int rows, cols;              // extents of the product
  int tiles_m, tiles_n, group_m, k_tiles;
  int tile_n;                  // columns of a tile, at most 256
  uint32_t stage_tx;           // bytes a CTA's copies bring to a stage
  int planes;                  // BF16 planes of the operands and of dz: 1 (BF16) or 3 (FP32)
  int slices;                  // k slices per tile (kProd)
  int group;                   // k tiles that add up in tensor memory before FP32 takes over
  unsigned long long wait_limit_ns;
  int debug_stop;              // >= 0: the copy issuer stops early (timeout test)
  unsigned int* status;
  // kStats, kDz
  const void* target;
  int id_bytes, vocab;
  long long ignore;
  int col0;                    // the class of column 0
  float2* stat;                // [parts][rows]: maximum, sum of exp(z - maximum)
  float* zt;                   // the target's logit
  const float* lse;
  const float* gloss;
  float* scale;                // what dz is divided by: written by kDz, read by kProd
  // kProd
  int to_part;                 // the output map is [slices][rows][..] FP32 sums
  int add;                     // to_part: add to what is there
  int out_tma;                 // it is the result; else `out` is written element by element
  void* out;
  long long ldo;
  int out_bf16, accumulate;
};

// Columns of a tile that one epilogue warp takes, and the warps that have any: a tile of
// up to 128 columns is shared between two like a wider one (100 x 5000 x 512 BF16, loss and
// gradients: 38 us for 44).
__host__ __device__ __forceinline__ int span_of(int tile_n) { return tile_n > 128 ? 128 : 64; }
__host__ __device__ __forceinline__ int parts_of(int tile_n) { return tile_n > 64 ? 2 : 1; }

// What a launch computes: one product (job 0), or with kProd two.  Pair p's units: first
// the long ones of job 0 (p, p + pairs, ...), of which the first `rest` pairs have one more
// than the others; these take `extra` units of job 1 meanwhile, then all go on alike.  One
// launch instead of two: 1000 x 11007 x 777 FP32, loss and gradients, 331 us for 352; 300 x
// 4000 x 256 BF16 33 for 40; 2048 x 32768 x 2048 BF16, gradients, 504 to 525 for 517 to 536.
struct XentJobs {
  XentGemm p[2];
  int units[2];
  int full, rest, extra;
};
struct alignas(64) XentMaps {
  CUtensorMap a[2], b[2], out[2];
};

// Whether A is MN-major, as a type.
template <bool B>
struct Mn {
  static constexpr bool value = B;
};

// The k-th unit of this pair; false: there is none.
template <int MODE>
__device__ __forceinline__ bool unit_at(const XentJobs& j, int pair, int pairs, int k, int& job,
                                        int& unit) {
  job = 0, unit = k * pairs + pair;
  if constexpr (MODE == kProd) {
    const bool more = pair < j.rest;
    const int mine = j.full + (more ? 1 : 0);
    if (k < mine) return true;
    k -= mine, job = 1;
    const int others = pairs - j.rest;
    if (!more && k < j.extra)
      unit = k * others + pair - j.rest;
    else
      unit = j.extra * others + (k - (more ? 0 : j.extra)) * pairs + pair;
    return unit < j.units[1];
  } else {
    return unit < j.units[0];
  }
}

// Unit u: k slice u % slices of tile u / slices; tiles in groups of group_m rows
// of tiles, so that a wave shares operand rows in L2.
__device__ __forceinline__ void unit_of(const XentGemm& p, int u, int& tm, int& tn, int& slice) {
  const int tile = u / p.slices;
  slice = u - tile * p.slices;
  const int per_group = p.group_m * p.tiles_n;
  const int g = tile / per_group, first = g * p.group_m;
  const int size = min(p.tiles_m - first, p.group_m);
  const int r = tile - g * per_group;
  tm = first + r % size;
  tn = r / size;
}

__device__ __forceinline__ void slice_range(const XentGemm& p, int slice, int& kt0, int& kt1) {
  kt0 = (int)((long long)slice * p.k_tiles / p.slices);
  kt1 = (int)((long long)(slice + 1) * p.k_tiles / p.slices);
}

// Three planes: the products (a, b) of A's and B's planes in the order in which they are
// added: a + b = 2, then 1, then 0, the smallest first.  The planes are copied in the
// order 1, 2, 0, so that the first product needs the first stage only; the first two
// stages are free again before the last product.
constexpr int kPairs = 6;
__device__ __forceinline__ constexpr int plane_a(int i) { return (0x102010 >> (20 - 4 * i)) & 15; }
__device__ __forceinline__ constexpr int plane_b(int i) { return (0x120100 >> (20 - 4 * i)) & 15; }
__device__ __forceinline__ constexpr int stage_of(int plane) { return (plane + 2) % 3; }

// A unit's k tiles add up in tensor memory in groups of `group`, and the groups' sums
// in registers, rounded to nearest.  The tensor core truncates when it adds to its FP32
// accumulator, which over a long k would add up to a bias of steps * 2^-24; a short
// group bounds that.
__device__ __forceinline__ int groups_of(const XentGemm& p, int kts) {
  return (kts + p.group - 1) / p.group;
}

// ------------------------------------------------------------------ epilogues

__device__ __forceinline__ long long target_at(const XentGemm& p, int i) {
  return p.id_bytes == 8 ? static_cast<const long long*>(p.target)[i]
                         : (long long)static_cast<const int*>(p.target)[i];
}

// kStats: maximum and sum over this warp's `left` columns (at most 128) of row r.
__device__ __forceinline__ void epi_stats(const XentGemm& p, float (&z)[128], int r, int n0,
                                          int left, int part) {
  if (r >= p.rows) return;
  if (left < 128) {
#pragma unroll
    for (int j = 0; j < 128; ++j)
      if (j >= left) z[j] = -INFINITY;
  }
  const long long t = target_at(p, r);
  if (t >= n0 && t < (long long)n0 + left) {
    const int at = (int)(t - n0);
    float zt = 0.f;
#pragma unroll
    for (int j = 0; j < 128; ++j) zt = j == at ? z[j] : zt;
    p.zt[r] = zt;
  }
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int j = 0; j < 128; ++j) m[j & 3] = fmaxf(m[j & 3], z[j]);
  const float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
  const float ref = top == -INFINITY ? 0.f : top;  // a row of -infinity
  float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 128; ++j) s[j & 3] += exp_f32(z[j] - ref);
  p.stat[(size_t)part * p.rows + r] = make_float2(top, (s[0] + s[1]) + (s[2] + s[3]));
}

// kDz: dz of this warp's columns of row r = row0 + lane, divided by the largest
// weight, as one or three BF16 planes.  The division keeps a mean's equal weights
// out of the rounding to BF16 (a factor 1/n would shift all of them alike, by up
// to 2^-8).
template <int PLANES>
__device__ __forceinline__ void epi_dz(const XentGemm& p, float (&z)[128], int row0, int lane,
                                       int n0, int left, float inv_scale, uint32_t buf,
                                       const CUtensorMap* m) {
  if (row0 >= p.rows) return;
  const int r = row0 + lane;
  float lse = 0.f, g = 0.f;
  int at = -1;  // the target's column
  if (r < p.rows) {
    const long long t = target_at(p, r);
    const bool in = t >= 0 && t < p.vocab;
    if (t != p.ignore && in)
      lse = p.lse[r], g = p.gloss[r] * inv_scale;
    else if (t != p.ignore && n0 == 0 && p.col0 == 0)
      atomicOr(p.status, kStatusIndex);
    const long long first = (long long)p.col0 + n0;
    if (t >= first && t < first + 128) at = (int)(t - first);
  }
  const bool live = g != 0.f;  // also for a NaN weight
#pragma unroll
  for (int c = 0; c < 128; c += 64) {
    if (c < left) {
#pragma unroll
      for (int j = c; j < c + 64; ++j) {
        const float e = exp_f32(z[j] - lse) - (j == at ? 1.f : 0.f);
        z[j] = live ? g * e : 0.f;
      }
#pragma unroll 1
      for (int pl = 0; pl < PLANES; ++pl) {
        uint4 w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t b[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            b[i] = split_plane<false>(z[c + 8 * j + 2 * i], z[c + 8 * j + 2 * i + 1]);
          }
          w[j] = make_uint4(b[0], b[1], b[2], b[3]);
        }
        store_rows(buf, m, n0 + c, row0, pl, w, false, lane);
      }
    }
  }
}

// The largest finite |weight| of the rows that have a gradient (the others' weights may be
// anything), by the block's epilogue threads (`tid` of 32 * kEpiWarps) through `red`.
__device__ __forceinline__ float largest_weight(const XentGemm& p, float* red, int tid) {
  float m = 0.f;
  for (int i = tid; i < p.rows; i += 32 * kEpiWarps) {
    const float g = fabsf(p.gloss[i]);
    const long long t = target_at(p, i);
    if (t != p.ignore && t >= 0 && t < p.vocab && isfinite(g)) m = fmaxf(m, g);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((tid & 31) == 0) red[tid >> 5] = m;
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory");
#pragma unroll
  for (int i = 0; i < kEpiWarps; ++i) m = fmaxf(m, red[i]);
  return m;
}

// kProd: this warp's columns of rows row0 .. row0 + 31 to the partial sums
// or the result.
__device__ __forceinline__ void epi_prod(const XentGemm& p, float (&v)[128], int row0, int lane,
                                         int n0, int left, int slice, float scale, uint32_t buf,
                                         const CUtensorMap* m) {
  if (row0 >= p.rows) return;
#pragma unroll
  for (int j = 0; j < 128; ++j) v[j] *= scale;
  if (p.to_part || (p.out_tma && !p.out_bf16)) {
#pragma unroll
    for (int c = 0; c < 128; c += 32) {
      if (c < left) {
        uint4 w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          w[j] = make_uint4(__float_as_uint(v[c + 4 * j]), __float_as_uint(v[c + 4 * j + 1]),
                            __float_as_uint(v[c + 4 * j + 2]), __float_as_uint(v[c + 4 * j + 3]));
        store_rows(buf, m, n0 + c, row0, p.to_part ? slice : 0, w, p.add, lane);
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

// ------------------------------------------------------------------ the kernel
//
// CTA r of a pair stages rows 128r .. 128r+127 of the tile's A and half of its B and
// holds rows 128r .. of the accumulator.  Both CTAs' copies of a stage complete
// on the even CTA's `full` barrier; its warp 1 issues the pair's MMAs and commits
// "stage read" and "accumulator final" to both CTAs.  Every wait is bounded: on a
// timeout the kernel flags the status word, waits (bounded) for what it started,
// frees its tensor memory and returns.
template <int MODE, int PLANES>
__global__ void __launch_bounds__(kThreads, 1)
    xent_gemm_kernel(const __grid_constant__ XentJobs jobs, const __grid_constant__ XentMaps maps) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ float wred[kEpiWarps];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // 128-byte swizzle atoms: 1024-byte aligned
  const uint32_t outs = base + kStages * kStageBytes;  // the epilogue warps' buffers
  const uint32_t bars = outs + kEpiWarps * kOutBytes;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (kStages + s); };
  auto tfull = [&](int a) { return bars + 8u * (2 * kStages + a); };
  auto tempty = [&](int a) { return bars + 8u * (2 * kStages + 2 + a); };
  const uint32_t drain = bars + 8u * (2 * kStages + 4);
  uint32_t* tmem_slot =
      reinterpret_cast<uint32_t*>(smem_raw + (bars - raw) + kNumBars * 8);
  const uint32_t rank = cluster_ctarank() & 1u;
  const bool even = rank == 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull(a), 1);
      mbar_init(tempty(a), 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
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
  const XentGemm& p0 = jobs.p[0];  // what both jobs have in common

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == 0) {
      // ---------------------------------------------------------- copy issuer
      if (lane == 0) {
        for (int j = 0; j < (MODE == kProd ? 2 : 1); ++j)
          if (jobs.units[j]) prefetch_tmap(&maps.a[j]), prefetch_tmap(&maps.b[j]);
        int s = 0, issued = 0;
        uint32_t ph = 0;
        const uint32_t full_even = even ? full(0) : mapa_shared(full(0), 0);
        // false: stop
        auto copy_unit = [&](auto mn, const XentGemm& p, const CUtensorMap* mA,
                             const CUtensorMap* mB, int u) {
          constexpr bool A_MN = decltype(mn)::value;
          int tm, tn, slice, kt0, kt1;
          unit_of(p, u, tm, tn, slice);
          slice_range(p, slice, kt0, kt1);
          const int ma = tm * kTile + (int)rank * 128, nb = tn * p.tile_n + (int)rank * (p.tile_n / 2);
          const bool wide = p.tile_n > 128;
          const uint32_t tx = 2 * p.stage_tx;
          for (int kt = kt0; kt < kt1; ++kt) {
#pragma unroll
            for (int i = 0; i < PLANES; ++i) {
              const int plane = PLANES == 1 ? 0 : (i + 1) % 3;
              if (p0.debug_stop >= 0 && issued >= p0.debug_stop) return false;
              if (!wait_phase(empty(s), ph ^ 1u, p0, kStatusTimeoutEmpty)) return false;
              const uint32_t st = base + s * kStageBytes;
              if (even) mbar_arrive_expect_tx(full(s), tx);
              const uint32_t fb = full_even + 8u * s;
              load_operand<A_MN>(st, mA, ma, kt, plane, fb);
              load_operand<MODE == kProd>(st + kATile, mB, nb, kt, plane, fb, wide);
              ++issued;
              if (++s == kStages) s = 0, ph ^= 1u;
            }
          }
          return true;
        };
        for (int k = 0, job, u; unit_at<MODE>(jobs, pair, pairs, k, job, u); ++k) {
          const bool on = MODE == kProd && job == 1
                              ? copy_unit(Mn<MODE == kProd>(), jobs.p[1], &maps.a[1],
                                          &maps.b[1], u)
                              : copy_unit(Mn<false>(), jobs.p[0], &maps.a[0], &maps.b[0], u);
          if (!on) break;
        }
        // leave only after the copies started here have landed (the odd CTA sees
        // the MMAs release the stages they read)
        for (int d = 0, pending = min(issued, kStages); d < pending; ++d) {
          if (--s < 0) s = kStages - 1, ph ^= 1u;
          if (!wait_phase(even ? full(s) : empty(s), ph, p0, kStatusTimeoutDrain))
            break;
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer (even CTA)
      if (even && lane == 0) {
        int s = 0, a = 0;
        uint32_t ph = 0, aph = 0;
        // One thread issues everything, a few cycles an instruction: what can be is
        // computed once.
        const uint32_t empty_odd = mapa_shared(empty(0), 1), tfull_odd = mapa_shared(tfull(0), 1);
        const uint32_t b0 = desc_lo<MODE == kProd>(base + kATile);
        constexpr uint32_t bstep = kDescStep<MODE == kProd>;
        // false: a wait has run out
        auto mma_unit = [&](auto mn, const XentGemm& p, int u) {
          constexpr bool A_MN = decltype(mn)::value;
          const uint32_t idesc = idesc_bf16(kTile, p.tile_n, A_MN, MODE == kProd);
          const uint32_t a0 = desc_lo<A_MN>(base);
          constexpr uint32_t astep = kDescStep<A_MN>;
          const int group = p.group;
          int tm, tn, slice, kt0, kt1;
          unit_of(p, u, tm, tn, slice);
          slice_range(p, slice, kt0, kt1);
          const int groups = groups_of(p, kt1 - kt0);
          for (int g = 0; g < groups; ++g) {
            if (!wait_phase<true>(tempty(a), aph ^ 1u, p0, kStatusTimeoutTmem))
              return false;
            tc_fence_after_sync();
            const uint32_t d = tmem + (uint32_t)(a * kTile);
            const int kts = min(group, kt1 - kt0 - g * group);
            for (int it = 0; it < kts; ++it) {
              if (!wait_phase(full(s), ph, p0, kStatusTimeoutFull))
                return false;
              tc_fence_after_sync();
              const uint32_t off = (uint32_t)s * kStageStep;
              if constexpr (PLANES == 1) {
#pragma unroll
                for (int kk = 0; kk < kBK / 16; ++kk)
                  mma_bf16_pair(d, a0 + off + kk * astep, b0 + off + kk * bstep, idesc,
                                (it > 0 || kk > 0) ? 1u : 0u);
                mma_commit_pair(empty(s));
                mma_commit_pair(empty_odd + 8u * s);
                if (++s == kStages) s = 0, ph ^= 1u;
              } else {
#pragma unroll
                for (int i = 0; i < kPairs; ++i) {
                  const uint32_t ai = a0 + off + stage_of(plane_a(i)) * kStageStep;
                  const uint32_t bi = b0 + off + stage_of(plane_b(i)) * kStageStep;
                  if (i == 1) {  // the other two planes
                    if (!wait_phase(full(s + 1), ph, p0, kStatusTimeoutFull) ||
                        !wait_phase(full(s + 2), ph, p0, kStatusTimeoutFull))
                      return false;
                    tc_fence_after_sync();
                  }
#pragma unroll
                  for (int kk = 0; kk < kBK / 16; ++kk)
                    mma_bf16_pair(d, ai + kk * astep, bi + kk * bstep, idesc,
                                  (it > 0 || i > 0 || kk > 0) ? 1u : 0u);
                  // planes 2, 1 and 0 have been read after products 2, 4 and 5
                  if (i == 2 || i >= 4) {
                    const int done = s + stage_of(i == 2 ? 2 : 5 - i);
                    mma_commit_pair(empty(done));
                    mma_commit_pair(empty_odd + 8u * done);
                  }
                }
                s += 3;
                if (s == kStages) s = 0, ph ^= 1u;
              }
            }
            mma_commit_pair(tfull(a));
            mma_commit_pair(tfull_odd + 8u * a);
            if (++a == 2) a = 0, aph ^= 1u;
          }
          return true;
        };
        for (int k = 0, job, u; unit_at<MODE>(jobs, pair, pairs, k, job, u); ++k)
          if (!(MODE == kProd && job == 1 ? mma_unit(Mn<MODE == kProd>(), jobs.p[1], u)
                                        : mma_unit(Mn<false>(), jobs.p[0], u)))
            break;
        mma_commit_pair(drain);
        wait_phase(drain, 0, p0, kStatusTimeoutTmem);
      }
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------- epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t tmem_row = tmem + ((uint32_t)(32 * q) << 16);
    const uint32_t buf = outs + (uint32_t)(warp - 4) * kOutBytes;
    const uint32_t tempty_even = even ? 0u : mapa_shared(tempty(0), 0);
    float scale = 1.f;
    if constexpr (MODE == kDz) {
      scale = divisor_of(largest_weight(p0, wred, threadIdx.x - 128));
      if (blockIdx.x == 0 && threadIdx.x == 128) *p0.scale = scale;
      scale = 1.f / scale;
    } else if constexpr (MODE != kStats) {
      scale = *p0.scale;
    }
    int a = 0;
    uint32_t aph = 0;
    for (int k = 0, job, u; unit_at<MODE>(jobs, pair, pairs, k, job, u); ++k) {
      const XentGemm& p = jobs.p[MODE == kProd ? job : 0];
      const CUtensorMap* out = &maps.out[MODE == kProd ? job : 0];
      const int span = span_of(p.tile_n);
      int tm, tn, slice, kt0, kt1;
      unit_of(p, u, tm, tn, slice);
      slice_range(p, slice, kt0, kt1);
      float acc[128];
      if (!collect(p0, acc, tmem_row + (uint32_t)(half * span), span, groups_of(p, kt1 - kt0), a, aph,
                   tfull(0), tempty(0), tempty_even, even, lane))
        break;
      const int row0 = tm * kTile + (int)rank * 128 + 32 * q;
      const int n0 = tn * p.tile_n + half * span;
      // this warp's columns of the tile that exist
      const int left = min(min(p.tile_n - half * span, span), p.cols - n0);
      if (left > 0) {
        if constexpr (MODE == kStats)
          epi_stats(p, acc, row0 + lane, n0, left, tn * parts_of(p.tile_n) + half);
        else if constexpr (MODE == kDz)
          epi_dz<PLANES>(p, acc, row0, lane, n0, left, scale, buf, out);
        else
          epi_prod(p, acc, row0, lane, n0, left, slice, scale, buf, out);
      }
    }
    if constexpr (MODE != kStats) {
      if (lane == 0) stores_done();
    }
  }

  __syncwarp();
  tc_fence_before_sync();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(*tmem_slot, kTmemCols);
  }
}

// ---------------------------------------------------------------- small kernels

// Rows of one or two matrices as `planes` BF16 planes with rows of ld elements (zeros
// past cols): plane 0 is x rounded, plane 1 what that leaves rounded, plane 2 the rest
// (FP32 in three planes: 24 bits).  Bound: bytes (11007 + 1000 rows of 777 FP32: 13 us, 6.7
// TB/s).
struct PlaneCopy {
  const void* x[2];
  long long ldx[2];
  int rows[2];  // 0: no such matrix
  Bf16* y[2];
  int cols, planes;
  long long ld;
};
template <typename T>
__global__ void __launch_bounds__(256) planes_kernel(const __grid_constant__ PlaneCopy p) {
  pdl_launch_dependents();
  pdl_wait();
  const long long groups = p.ld / 8, total = groups * ((long long)p.rows[0] + p.rows[1]);
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (long long)gridDim.x * 256) {
    const long long at = i / groups;
    const int c = (int)(i - at * groups) * 8;
    const bool second = at >= p.rows[0];
    const long long r = second ? at - p.rows[0] : at;
    const T* x = static_cast<const T*>(second ? p.x[1] : p.x[0]) + r * (second ? p.ldx[1] : p.ldx[0]);
    Bf16* y = (second ? p.y[1] : p.y[0]) + r * p.ld + c;
    const long long plane = (second ? p.rows[1] : p.rows[0]) * p.ld;
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = c + j < p.cols ? to_f32(x[c + j]) : 0.f;
    for (int pl = 0; pl < p.planes; ++pl) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = p.planes == 1 ? pack_bf16(f[2 * j], f[2 * j + 1])
               : pl == 0     ? split_plane<true>(f[2 * j], f[2 * j + 1])
                             : split_plane<false>(f[2 * j], f[2 * j + 1]);
      *reinterpret_cast<uint4*>(y + pl * plane) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// lse and loss of 32 rows: thread (x, y) joins the statistics y, y + 32, ... of
// row x, then warp y == 0 joins the 32 results in order.
__global__ void __launch_bounds__(1024) xent_join_kernel(const float2* stat, const float* zt,
                                                         int parts, int rows, const void* target,
                                                         int id_bytes, long long ignore, int vocab,
                                                         float* lse, float* loss,
                                                         unsigned int* status) {
  __shared__ float2 acc[32][33];
  pdl_launch_dependents();
  pdl_wait();
  const int r = blockIdx.x * 32 + threadIdx.x;
  float top = -INFINITY, sum = 0.f;
  auto join = [&](float2 x) {
    const float now = fmaxf(top, x.x), ref = now == -INFINITY ? 0.f : now;
    sum = sum * exp_f32(top - ref) + x.y * exp_f32(x.x - ref);
    top = now;
  };
  if (r < rows) {
#pragma unroll 4
    for (int i = threadIdx.y; i < parts; i += 32) join(stat[(size_t)i * rows + r]);
  }
  acc[threadIdx.y][threadIdx.x] = make_float2(top, sum);
  __syncthreads();
  if (threadIdx.y != 0 || r >= rows) return;
#pragma unroll 4
  for (int i = 1; i < 32; ++i) join(acc[i][threadIdx.x]);
  const float l = top + logf(sum);
  lse[r] = l;
  const long long t = id_bytes == 8 ? static_cast<const long long*>(target)[r]
                                    : (long long)static_cast<const int*>(target)[r];
  const bool in = t >= 0 && t < vocab;
  if (t != ignore && !in) atomicOr(status, kStatusIndex);
  if (loss) loss[r] = t == ignore ? 0.f : in ? l - zt[r] : __int_as_float(0x7fc00000);
}

// out = the slices' sums added in order (plus out when accumulate).
template <typename T>
__global__ void __launch_bounds__(256) xent_reduce_kernel(const float* part, int slices,
                                                          long long part_ld, long long part_slice,
                                                          int rows, int cols, T* out,
                                                          long long ldo, int accumulate) {
  pdl_launch_dependents();
  pdl_wait();
  const long long total = (long long)rows * cols;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (long long)gridDim.x * 256) {
    const long long r = i / cols;
    const int c = (int)(i - r * cols);
    const float* q = part + r * part_ld + c;
    float s = 0.f;
#pragma unroll 4
    for (int k = 0; k < slices; ++k) s += q[k * part_slice];
    T* o = out + r * ldo + c;
    *o = from_f32<T>(accumulate ? s + to_f32(*o) : s);
  }
}

// ------------------------------------------------------------------- host side

// As an operand whose k runs along the columns, `box` rows a copy; as one whose k
// runs along the rows; and as the output of 32-row stores.
int map_k(CUtensorMap* m, const Planes& x, int box) {
  return encode_rows(m, false, x.p, x.cols, x.rows, x.ld, x.planes, x.plane, box);
}
int map_mn(CUtensorMap* m, const Planes& x) {
  return encode_rows(m, false, x.p, x.cols, x.rows, x.ld, x.planes, x.plane, 64);
}
int map_out(CUtensorMap* m, const Planes& x) {
  return encode_rows(m, false, x.p, x.cols, x.rows, x.ld, x.planes, x.plane, 32);
}

// The launch shapes are planned for this many pairs (GB300: 152 SMs), so that the
// workspace query needs no device.
constexpr int kPlanPairs = 76;
constexpr int kMaxSlices = 76;

// Rows of h a CTA copies to a stage: all 128, or fewer where the tokens fit one
// CTA's half (what its other rows then multiply is never stored).
int token_box(int tokens) { return tokens >= 128 ? 128 : (int)round_up(tokens, 8); }

// What a k tile of a pair's tile costs, in cycles.  BF16: its copies, 64 bytes a cycle
// and SM (`rows`: those of both operands that a CTA copies, twice).  FP32: six products of
// which each takes as long in a tile of 128 columns as in one of 256 (1000 x 11007 x 777,
// loss and gradients: 433 us where 128 saves a third of the columns, 386 with 256,
// one k tile a group).
long long k_tile_cost(int planes, long long rows) { return planes == 1 ? rows : 3200; }
// What a column of a tile costs once a launch, after its last k tile: narrow tiles win
// where all have a pair of their own (FP32, 300 x 4000 x 256, all gradients: 54 us for 68).
constexpr long long kColumnCost = 30;

// Columns of a tile of h w^T, a multiple of `step`: what makes the pairs' rounds
// cheapest.  BF16, 2048 x 32768 classes: 256; 100 tokens: 224 (two full rounds; 256 leaves
// a quarter of the pairs idle in the second one).  Steps of 32, the ones in which every form
// of a pair's MMA takes its N; steps of 16 would make one call in three 1 to 5 % cheaper by
// this count.
int choose_tile_n(int planes, int tokens, int classes, int k_tiles, int step) {
  const long long tiles_m = ceil_div(tokens, kTile), a = 2 * token_box(tokens);
  int best = kTile;
  long long cost = -1;
  for (int tn = kTile; tn >= 64; tn -= step) {
    const long long c = ceil_div(tiles_m * ceil_div(classes, tn), kPlanPairs) * k_tiles *
                            k_tile_cost(planes, a + tn) + (planes == 1 ? 0 : kColumnCost * tn);
    if (cost < 0 || c < cost) best = tn, cost = c;
  }
  return best;
}

// The statistics' parts: an epilogue warp's columns each.
int stat_parts(int classes, int tile_n) {
  const int tiles = (int)ceil_div(classes, tile_n), last = classes - (tiles - 1) * tile_n;
  return (tiles - 1) * parts_of(tile_n) + (last > span_of(tile_n) ? 2 : 1);
}

template <int MODE, int PLANES>
int resident_pairs(int dev, int sms) {
  static std::atomic<int> cached[64];
  if (dev < 0 || dev >= 64) return 0;
  int pairs = cached[dev].load(std::memory_order_acquire);
  if (pairs) return pairs;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.gridDim = dim3((unsigned)(sms & ~1));
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(xent_gemm_kernel<MODE, PLANES>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kSmemBytes) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&pairs, xent_gemm_kernel<MODE, PLANES>, &cfg) != cudaSuccess ||
      pairs < 1)
    return 0;
  cached[dev].store(pairs, std::memory_order_release);
  return pairs;
}

// Fills in the tiling and launches the jobs that have a tile width.
template <int MODE, int PLANES>
int launch_planes(XentJobs& jobs, const XentMaps& maps, const TrainDevice& d, cudaStream_t st) {
  const int pairs = resident_pairs<MODE, PLANES>(d.dev, d.sms);
  if (!pairs) return B2G_ERR_CUDA;
  long long units = 0, cost[2] = {0, 0};
  for (int j = 0; j < 2; ++j) {
    XentGemm& p = jobs.p[j];
    p.wait_limit_ns = d.wait_limit_ns, p.debug_stop = d.debug_stop, p.status = d.status;
    jobs.units[j] = 0;
    if (!p.tile_n) continue;
    p.tiles_m = (int)ceil_div(p.rows, kTile), p.tiles_n = (int)ceil_div(p.cols, p.tile_n);
    p.group_m = 16;
    const long long n = (long long)p.tiles_m * p.tiles_n * p.slices;
    units += n;
    if (units > 0x3fffffffLL) return B2G_ERR_INVALID_DIM;
    jobs.units[j] = (int)n;
    cost[j] = ceil_div(p.k_tiles, p.slices) * k_tile_cost(PLANES, kTile + p.tile_n);
  }
  const int used = (int)(units < pairs ? units : pairs);
  jobs.full = jobs.units[0] / used, jobs.rest = jobs.units[0] % used, jobs.extra = 0;
  if (jobs.rest && jobs.units[1]) {  // as many as job 0's last units take, one more or not
    const long long others = used - jobs.rest, most = ceil_div(jobs.units[1], others);
    long long best = -1;
    for (long long e = cost[0] / cost[1], i = 0; i < 2; ++i, ++e) {
      const long long x = e < most ? e : most;
      const long long after = jobs.units[1] > x * others ? jobs.units[1] - x * others : 0;
      const long long all = after / used, left = after % used;
      const long long t0 = cost[0] + (all + (left > 0)) * cost[1];
      const long long t1 = (x + all + (left > jobs.rest)) * cost[1];
      if (best < 0 || (t0 > t1 ? t0 : t1) < best) best = t0 > t1 ? t0 : t1, jobs.extra = (int)x;
    }
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * used));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  void* args[] = {&jobs, const_cast<XentMaps*>(&maps)};
  return launch_code(
      cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(&xent_gemm_kernel<MODE, PLANES>), args));
}

// k tiles of an accumulation group.  FP32, the time of loss and gradients at 1000 x 11007 x
// 777 and the relative error of dh at 1205 x 1703 x 2136 (FP32 library products: 1.2e-6):
// 1: 384 us, 1.9e-7; 2: 357 us, 5.3e-7; 4: 349 us, 1.3e-6; 8: 348 us, 2.8e-6.  Logits of BF16
// operands: 16, whose error of the loss is that of FP32 products.  Products that are
// rounded to BF16: kGroupK.
int group_of(int dtype, bool logits) {
  return dtype == B2G_F32 ? 2 : logits ? 16 : kGroupK / kBK;
}

template <int MODE>
int launch_gemm(XentJobs& jobs, const XentMaps& maps, const TrainDevice& d, cudaStream_t st) {
  return jobs.p[0].planes == 1 ? launch_planes<MODE, 1>(jobs, maps, d, st)
                               : launch_planes<MODE, 3>(jobs, maps, d, st);
}

struct Call {
  int dtype, tokens, vocab, width;
  const void* h;
  long long ldh;
  const void* w;
  long long ldw;
};

int check(const Call& c) {
  if (!type_ok(c.dtype)) return B2G_ERR_INVALID_TYPE;
  if (c.tokens < 0 || c.vocab < 1 || c.width < 1 || c.tokens > kMaxLength ||
      c.vocab > kMaxLength || c.width > kMaxLength)
    return B2G_ERR_INVALID_DIM;
  if (c.ldh < c.width || c.ldw < c.width) return B2G_ERR_INVALID_LD;
  return 0;
}

// Columns of a tile of a gradient (128 or 256) and its k slices: the cheapest rounds, with
// `beside` cycles of the other gradient's units to fill them up, counting what several
// slices' partial sums cost (written and read at about 3400 bytes
// a cycle, and a launch that adds them).  Slices have at least 8 k tiles each; a narrower
// tile or another slice has to save a twentieth.
struct Plan {
  int tile_n, slices;
};
Plan plan_product(int planes, long long rows, int cols, int k_tiles, long long beside) {
  Plan best{kTile, 1};
  long long cost = -1;
  for (int tn = kTile; tn >= 128; tn -= 128) {
    const long long tiles = ceil_div(rows, kTile) * ceil_div(cols, tn);
    for (int s = 1; s == 1 || (s <= kMaxSlices && s <= k_tiles / 8); ++s) {
      const long long unit = ceil_div(k_tiles, s) * k_tile_cost(planes, kTile + tn);
      const long long alone = ceil_div(tiles * s, kPlanPairs) * unit;
      const long long shared = (tiles * s * unit + beside) / kPlanPairs;
      const long long c = (alone > shared ? alone : shared) + kColumnCost * tn +
                          (s > 1 ? 4000 + s * rows * cols * 8 / 3400 : 0);
      if (cost < 0 || c < cost - cost / 20) best = Plan{tn, s}, cost = c;
    }
  }
  return best;
}

// dz for one piece of the vocabulary stays below this (the piece is a multiple
// of 256 classes, at least one).
constexpr size_t kDzBytes = size_t(512) << 20;
struct Layout {
  bool few;                          // the few-token form
  int planes;
  bool copy_h, copy_w;
  long long ldc;                     // row length of the copies
  size_t h, w, stat, zt, scale, dz, hpart, wpart, total;
  int piece, pieces;                 // classes per piece
  long long dz_ld, part_ld;
  int slices_h, slices_w, tile_h, tile_w;  // of dz w and of dz^T h
  int tile_n;                        // of h w^T
  int parts;                         // its statistics' parts
  bool h_sums;                       // dh goes through FP32 sums
};

Layout layout(const Call& c, bool backward) {
  Layout l;
  l.planes = c.dtype == B2G_F32 ? 3 : 1;
  l.copy_h = c.dtype == B2G_F32 || !vec16(c.h) || c.ldh % 8;
  l.few = c.tokens <= kFewTokens && vec16(c.w) && vec16_ld(c.ldw, c.dtype);
  l.copy_w = !l.few && (c.dtype == B2G_F32 || !vec16(c.w) || c.ldw % 8);
  l.ldc = (long long)round_up(c.width, 8);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += round_up(bytes, 256);
    return o;
  };
  l.h = l.copy_h ? take((size_t)l.planes * c.tokens * l.ldc * 2) : 0;
  l.w = l.copy_w ? take((size_t)l.planes * c.vocab * l.ldc * 2) : 0;
  l.stat = l.zt = l.scale = l.dz = l.hpart = l.wpart = 0;
  l.piece = c.vocab, l.pieces = 1, l.slices_h = l.slices_w = 1, l.h_sums = false;
  l.tile_h = l.tile_w = kTile;
  const int k_tiles = (int)ceil_div(c.width, kBK);
  if (!backward) {
    l.tile_n = choose_tile_n(l.planes, c.tokens, c.vocab, k_tiles, 32);
    l.parts = l.few ? few_stat_parts(c.vocab) : stat_parts(c.vocab, l.tile_n);
    l.stat = take((size_t)l.parts * c.tokens * sizeof(float2));
    l.zt = take((size_t)c.tokens * sizeof(float));
  } else {
    const long long fit = (long long)(kDzBytes / ((size_t)l.planes * c.tokens * 2)) / kTile * kTile;
    const long long most = fit < kTile ? kTile : fit;
    l.pieces = (int)ceil_div(c.vocab, most);
    l.piece = (int)round_up((size_t)ceil_div(c.vocab, l.pieces), kTile);
    l.pieces = (int)ceil_div(c.vocab, l.piece);
    l.tile_n = choose_tile_n(l.planes, c.tokens, l.piece, k_tiles, 64);  // whole 64-column stores
    l.dz_ld = l.piece;
    l.part_ld = (long long)round_up(c.width, 4);
    const int classes = l.piece < c.vocab ? l.piece : c.vocab;
    const int kh = (int)ceil_div(classes, kBK), kw = (int)ceil_div(c.tokens, kBK);
    const Plan pw = plan_product(l.planes, classes, c.width, kw, 0);
    const Plan ph = plan_product(l.planes, c.tokens, c.width, kh,
                                 ceil_div(classes, kTile) * ceil_div(c.width, pw.tile_n) * kw *
                                     k_tile_cost(l.planes, kTile + pw.tile_n));
    l.tile_h = ph.tile_n, l.slices_h = ph.slices, l.tile_w = pw.tile_n, l.slices_w = pw.slices;
    l.scale = take(sizeof(float));
    l.dz = take((size_t)l.planes * c.tokens * l.dz_ld * 2);
    if (l.few) l.slices_h = l.pieces * few_slices(c.width, c.vocab < l.piece ? c.vocab : l.piece);
    l.h_sums = l.few || l.slices_h > 1 || l.pieces > 1;
    if (l.h_sums)
      l.hpart = take((size_t)l.slices_h * c.tokens * l.part_ld * 4);
    if (l.slices_w > 1) l.wpart = take((size_t)l.slices_w * l.piece * l.part_ld * 4);
  }
  l.total = at;
  return l;
}

// h and w (unless pw is NULL) themselves, or their planes written to the workspace.
int operands(const Call& c, const Layout& l, unsigned char* ws, const TrainDevice& d,
             cudaStream_t st, Planes* ph, Planes* pw) {
  PlaneCopy q = {};
  q.cols = c.width, q.planes = l.planes, q.ld = l.ldc;
  int n = 0;
  auto one = [&](const void* x, long long ldx, int rows, bool copy, size_t at, Planes* out) {
    *out = Planes{static_cast<const Bf16*>(x), rows, c.width, ldx, 0, 1};
    if (!copy) return;
    Bf16* to = reinterpret_cast<Bf16*>(ws + at);
    *out = Planes{to, rows, c.width, l.ldc, (long long)rows * l.ldc, l.planes};
    q.x[n] = x, q.ldx[n] = ldx, q.rows[n] = rows, q.y[n] = to, ++n;
  };
  one(c.h, c.ldh, c.tokens, l.copy_h, l.h, ph);
  if (pw) one(c.w, c.ldw, c.vocab, l.copy_w, l.w, pw);
  if (!n) return 0;
  const long long blocks = ceil_div(l.ldc / 8 * ((long long)q.rows[0] + q.rows[1]), 256);
  const dim3 grid((unsigned)(blocks < 16LL * d.sms ? blocks : 16LL * d.sms));
  return launch_code(c.dtype == B2G_F32
                         ? launch_train(planes_kernel<float>, grid, dim3(256), 0, st, q)
                         : launch_train(planes_kernel<Bf16>, grid, dim3(256), 0, st, q));
}

template <typename T>
int reduce(const float* part, int slices, long long ld, long long slice, int rows, int cols,
           void* out, long long ldo, int accumulate, const TrainDevice& d, cudaStream_t st) {
  const long long blocks = ceil_div((long long)rows * cols, 256), most = 16LL * d.sms;
  return launch_code(launch_train(xent_reduce_kernel<T>, dim3((unsigned)(blocks < most ? blocks : most)),
                                  dim3(256), 0, st, part, slices, ld, slice, rows, cols,
                                  static_cast<T*>(out), ldo, accumulate));
}

}  // namespace
}  // namespace b2g

using namespace b2g;

extern "C" {

int b2g_linear_xent_workspace_size(int dtype, int tokens, int vocab, int width, const void* h,
                                   long long ldh, const void* w, long long ldw, int backward,
                                   size_t* bytes) {
  const Call c{dtype, tokens, vocab, width, h, ldh, w, ldw};
  const int rc = check(c);
  if (rc) return rc;
  if (!bytes) return B2G_ERR_NULL;
  *bytes = tokens ? layout(c, backward != 0).total : 0;
  return 0;
}

int b2g_linear_xent(int dtype, int tokens, int vocab, int width, const void* h, long long ldh,
                    const void* w, long long ldw, const void* target, int id_bytes,
                    long long ignore_index, float* loss, float* lse, void* workspace,
                    size_t workspace_bytes, void* stream) {
  const Call c{dtype, tokens, vocab, width, h, ldh, w, ldw};
  int rc = check(c);
  if (rc) return rc;
  if (id_bytes != 8 && id_bytes != 4) return B2G_ERR_INVALID_TYPE;
  if (tokens == 0) return 0;
  if (!h || !w || !target || !lse) return B2G_ERR_NULL;
  TrainDevice d;
  rc = train_device(&d);
  if (rc) return rc;
  const Layout l = layout(c, false);
  if (!workspace || !vec16(workspace) || workspace_bytes < l.total) return B2G_ERR_WORKSPACE;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Planes ph, pw;
  rc = operands(c, l, ws, d, st, &ph, l.few ? nullptr : &pw);
  if (rc) return rc;
  float2* stat = reinterpret_cast<float2*>(ws + l.stat);
  float* zt = reinterpret_cast<float*>(ws + l.zt);
  auto join = [&] {
    return launch_code(launch_train(xent_join_kernel, dim3((unsigned)ceil_div(tokens, 32)),
                                    dim3(32, 32), 0, st, (const float2*)stat, (const float*)zt,
                                    l.parts, tokens, target, id_bytes, ignore_index, vocab, lse,
                                    loss, d.status));
  };
  if (l.few) {
    const XentRows rows{tokens, vocab, width, target, id_bytes, ignore_index};
    rc = launch_few_stats(rows, ph, FewHead{w, ldw, dtype == B2G_F32}, stat, zt, d, st);
    return rc ? rc : join();
  }
  XentMaps maps = {};
  rc = map_k(&maps.a[0], ph, token_box(tokens));
  if (!rc) rc = map_k(&maps.b[0], pw, l.tile_n / 2);
  if (rc) return rc;
  XentJobs jobs = {};
  XentGemm& p = jobs.p[0];
  p.tile_n = l.tile_n, p.stage_tx = (token_box(tokens) + l.tile_n / 2) * 128;
  p.rows = tokens, p.cols = vocab;
  p.k_tiles = (int)ceil_div(width, kBK), p.planes = l.planes, p.slices = 1;
  p.group = group_of(dtype, true);
  p.target = target, p.id_bytes = id_bytes, p.vocab = vocab, p.ignore = ignore_index;
  p.stat = stat, p.zt = zt;
  rc = launch_gemm<kStats>(jobs, maps, d, st);
  return rc ? rc : join();
}

int b2g_linear_xent_backward(int dtype, int tokens, int vocab, int width, const void* h,
                             long long ldh, const void* w, long long ldw, const void* target,
                             int id_bytes, long long ignore_index, const float* lse,
                             const float* grad_loss, void* dh, long long lddh, int accumulate,
                             void* dw, long long lddw, void* workspace, size_t workspace_bytes,
                             void* stream) {
  const Call c{dtype, tokens, vocab, width, h, ldh, w, ldw};
  int rc = check(c);
  if (rc) return rc;
  if (id_bytes != 8 && id_bytes != 4) return B2G_ERR_INVALID_TYPE;
  if ((dh && lddh < width) || (dw && lddw < width)) return B2G_ERR_INVALID_LD;
  if (tokens == 0 && (!dw || accumulate)) return 0;
  if (!dh && !dw) return 0;
  if (tokens > 0 && (!h || !w || !target || !lse || !grad_loss)) return B2G_ERR_NULL;
  TrainDevice d;
  rc = train_device(&d);
  if (rc) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const long long es = (long long)type_size(dtype);
  if (tokens == 0)
    return cudaMemset2DAsync(dw, lddw * es, 0, width * es, vocab, st) == cudaSuccess ? 0
                                                                                    : B2G_ERR_CUDA;
  const Layout l = layout(c, true);
  if (!workspace || !vec16(workspace) || workspace_bytes < l.total) return B2G_ERR_WORKSPACE;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  Planes ph, pw;
  rc = operands(c, l, ws, d, st, &ph, l.few ? nullptr : &pw);
  if (rc) return rc;
  const XentRows few_rows{tokens, vocab, width, target, id_bytes, ignore_index};
  const FewHead head{w, ldw, dtype == B2G_F32};
  XentGemm base = {};
  base.planes = l.planes, base.slices = 1;
  base.out_bf16 = dtype == B2G_BF16;
  base.scale = reinterpret_cast<float*>(ws + l.scale);
  base.group = group_of(dtype, false);
  float* hpart = reinterpret_cast<float*>(ws + l.hpart);
  float* wpart = reinterpret_cast<float*>(ws + l.wpart);
  const bool f32 = dtype == B2G_F32;
  const long long hslice = (long long)tokens * l.part_ld, wslice = (long long)l.piece * l.part_ld;
  const auto reduce_to = f32 ? reduce<float> : reduce<Bf16>;
  for (int i = 0; i < l.pieces; ++i) {
    const int first = i * l.piece;
    const int n = vocab - first < l.piece ? vocab - first : l.piece;
    Planes piece = {};
    if (!l.few) piece = pw, piece.p += (long long)first * pw.ld, piece.rows = n;
    const Planes dz{reinterpret_cast<Bf16*>(ws + l.dz), tokens, n, l.dz_ld,
                    (long long)tokens * l.dz_ld, l.planes};
    // dz of these classes
    if (l.few) {
      rc = launch_few_dz(few_rows, ph, head, first, n, lse, grad_loss, dz, base.scale, d, st);
      const int each = l.slices_h / l.pieces;
      if (!rc && dh)
        rc = launch_few_dh(few_rows, dz, head, first, n, base.scale, each,
                           hpart + (size_t)i * each * hslice, l.part_ld, d, st);
    } else {
      XentJobs jobs = {};
      XentMaps maps = {};
      XentGemm& p = jobs.p[0];
      p = base;
      p.rows = tokens, p.cols = n, p.k_tiles = (int)ceil_div(width, kBK);
      p.tile_n = l.tile_n, p.stage_tx = (token_box(tokens) + l.tile_n / 2) * 128;
      p.group = group_of(dtype, true);
      p.target = target, p.id_bytes = id_bytes, p.vocab = vocab, p.ignore = ignore_index;
      p.col0 = first, p.lse = lse, p.gloss = grad_loss;
      rc = map_k(&maps.a[0], ph, token_box(tokens));
      if (!rc) rc = map_k(&maps.b[0], piece, l.tile_n / 2);
      if (!rc) rc = map_out(&maps.out[0], dz);
      if (!rc) rc = launch_gemm<kDz>(jobs, maps, d, st);
    }
    if (rc) return rc;
    XentJobs jobs = {};
    XentMaps maps = {};
    jobs.p[0] = jobs.p[1] = base;
    if (dh && !l.few) {  // dh += dz w over these classes
      XentGemm& p = jobs.p[0];
      p.rows = tokens, p.cols = width, p.k_tiles = (int)ceil_div(n, kBK);
      p.tile_n = l.tile_h, p.stage_tx = kATile + l.tile_h / 2 * 128;
      p.slices = l.slices_h < p.k_tiles ? l.slices_h : p.k_tiles;
      p.to_part = l.h_sums, p.add = i > 0;
      p.out = dh, p.ldo = lddh;
      // a bulk-tensor store writes whole 16-byte units, those past the last column too
      p.out_tma = vec16(dh) && vec16_ld(lddh, dtype) && vec16_ld(width, dtype);
      rc = map_k(&maps.a[0], dz, 128);
      if (!rc) rc = map_mn(&maps.b[0], piece);
      if (!rc && (p.to_part || p.out_tma))
        rc = p.to_part ? encode_rows(&maps.out[0], true, hpart, width, tokens, l.part_ld,
                                     l.slices_h, hslice, 32)
                       : encode_rows(&maps.out[0], f32, dh, width, tokens, lddh, 1, 0, 32);
      if (rc) return rc;
    }
    unsigned char* dw_rows =
        dw ? static_cast<unsigned char*>(dw) + (long long)first * lddw * es : nullptr;
    if (dw) {  // these classes' rows of dw = dz^T h
      XentGemm& p = jobs.p[1];
      p.rows = n, p.cols = width, p.k_tiles = (int)ceil_div(tokens, kBK);
      p.tile_n = l.tile_w, p.stage_tx = kATile + l.tile_w / 2 * 128;
      p.slices = l.slices_w;
      p.to_part = l.slices_w > 1;
      p.out = dw_rows, p.ldo = lddw, p.accumulate = accumulate != 0;
      // as for dh; and it adds in the output's type: right for FP32 only
      p.out_tma = vec16(dw_rows) && vec16_ld(lddw, dtype) && vec16_ld(width, dtype) &&
                  !(accumulate && !f32);
      p.add = !p.to_part && accumulate;
      rc = map_mn(&maps.a[1], dz);
      if (!rc) rc = map_mn(&maps.b[1], ph);
      if (!rc && (p.to_part || p.out_tma))
        rc = p.to_part ? encode_rows(&maps.out[1], true, wpart, width, n, l.part_ld, l.slices_w,
                                     wslice, 32)
                       : encode_rows(&maps.out[1], f32, dw_rows, width, n, lddw, 1, 0, 32);
      if (rc) return rc;
    }
    if (jobs.p[0].tile_n || jobs.p[1].tile_n) rc = launch_gemm<kProd>(jobs, maps, d, st);
    if (!rc && jobs.p[1].to_part)
      rc = reduce_to(wpart, l.slices_w, l.part_ld, wslice, n, width, dw_rows, lddw,
                     jobs.p[1].accumulate, d, st);
    if (rc) return rc;
  }
  if (dh && l.h_sums)
    return reduce_to(hpart, l.slices_h, l.part_ld, hslice, tokens, width, dh, lddh, 0, d, st);
  return 0;
}

}  // extern "C"
