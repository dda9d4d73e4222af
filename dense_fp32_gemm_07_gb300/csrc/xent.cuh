// xent.cuh -- what the two forms of the linear cross entropy share (xent.cu: CTA
// pairs on 256 x 256 tiles; xent_few.cu: up to 64 tokens): tensor-core descriptors,
// the split of FP32 into BF16 planes, exponentials, tensor maps.
#pragma once
#include <cudaTypedefs.h>

#include "tcgen05.cuh"
#include "train_common.cuh"

namespace b2g {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();  // host.cu

// kind::f16 with BF16 operands and an FP32 accumulator; A or B MN-major when asked.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4)                                  // D: FP32
         | (1u << 7) | (1u << 10)                   // A, B: BF16
         | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16)
         | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Shared-memory descriptors of a 128-byte-swizzled operand, as two 32-bit words: the
// low one holds the address in 16-byte units (so a step inside the operand is an
// addition) and the leading offset, the high one is constant.
// K-major: rows of 128 bytes hold 64 k of one row of the operand; groups of 8 rows are
// 1024 bytes apart.  MN-major: rows of 128 bytes hold 64 rows of the operand at one k;
// groups of 8 k are 1024 bytes apart, blocks of 64 rows (one bulk-tensor box of 64 x
// 64) 8192 bytes.
constexpr uint32_t kDescHi = (1024u >> 4)     // stride offset
                             | (1u << 14)     // descriptor version (sm_100 family)
                             | (2u << 29);    // layout: 128-byte swizzle
template <bool MN>
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) {
  return ((saddr & 0x3FFFFu) >> 4) | ((MN ? 8192u >> 4 : 1u) << 16);
}
// What 16 k further adds: 32 bytes of each row, or 16 rows.
template <bool MN>
constexpr uint32_t kDescStep = MN ? 2048u >> 4 : 32u >> 4;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Two FP32 values to their next BF16 plane: the rounded pair is returned and x, y
// become what it leaves (exact).  The FIRST plane saturates, so that FP32's largest
// values do not round to infinity.
template <bool FIRST>
__device__ __forceinline__ uint32_t split_plane(float& x, float& y) {
  uint32_t b;
  if (FIRST)
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(b) : "f"(y), "f"(x));
  else
    b = pack_bf16(x, y);
  x -= __uint_as_float(b << 16);
  y -= __uint_as_float(b & 0xFFFF0000u);
  return b;
}

// e^x as the hardware's base-2 exponential (relative error 2^-22) of x log2(e),
// whose rounding adds |x| 2^-24: x is at most about 0 here, so that error grows
// only where e^x is small.  Results below 2^-126 become 0.
__device__ __forceinline__ float exp_f32(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}

// k of BF16 operands whose products add up in tensor memory, for a result that is rounded to
// BF16: 2048 steps, each of which truncates the sum to 24 bits.  Terms of one sign lose at
// most 2^-12 of it by that, a sixteenth of what rounding the result may cost; without a
// limit dh over 2^28 classes of 8 columns came out 5 % short.
constexpr int kGroupK = 1 << 15;

// What dz is divided by before it is rounded to BF16, for the largest of the weights: at
// least FP32's smallest normal number, so that its reciprocal is finite.
__device__ __forceinline__ float divisor_of(float largest) { return fmaxf(largest, 0x1p-126f); }

// The loads into v are complete; tying v to the wait keeps its uses behind it.
__device__ __forceinline__ void tie16(uint32_t (&v)[16]) {
  asm volatile(""
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                 "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                 "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])::"memory");
}
__device__ __forceinline__ void tie32(uint32_t (&v)[32]) {
  asm volatile(""
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                 "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                 "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]),
                 "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                 "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                 "+r"(v[30]), "+r"(v[31])::"memory");
}

// {inner, outer, planes} BF16 or FP32 elements, boxes of 128 bytes x box_outer
// rows with the 128-byte swizzle; ld and plane in elements.
inline int encode_rows(CUtensorMap* m, bool f32, const void* base, long long inner, long long outer,
           long long ld, int planes, long long plane, int box_outer) {
  auto enc = tensor_map_encoder();
  if (!enc) return B2G_ERR_TENSOR_MAP;
  const cuuint64_t es = f32 ? 4 : 2;
  cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)outer, (cuuint64_t)planes};
  cuuint64_t strides[2] = {(cuuint64_t)ld * es, planes > 1 ? (cuuint64_t)plane * es : 16};
  cuuint32_t box[3] = {(cuuint32_t)(128 / es), (cuuint32_t)box_outer, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r =
      enc(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
          const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? 0 : B2G_ERR_TENSOR_MAP;
}

// A matrix as BF16 planes: rows x cols, rows ld apart, planes `plane` apart.
struct Planes {
  const Bf16* p;
  int rows, cols;
  long long ld, plane;
  int planes;
};
// What a call multiplies: its sizes, its operands as BF16 planes (w unless it is
// read as FP32), and where its rows' targets and results are.
struct XentRows {
  int tokens, vocab, width;
  const void* target;
  int id_bytes;
  long long ignore;
};

// ---- up to kFewTokens tokens (xent_few.cu) ----

constexpr int kFewTokens = 64;

// w in its own type: rows of classes on 16-byte boundaries.
struct FewHead {
  const void* w;
  long long ldw;
  bool f32;
};

// Statistics' parts, and k slices of dh (for `classes` classes), of the few-token form.
int few_stat_parts(int classes);
int few_slices(int width, int classes);

// Row statistics ([parts][tokens]) and the target's logit of each token.
int launch_few_stats(const XentRows& r, const Planes& h, const FewHead& w, float2* stat, float* zt,
                     const TrainDevice& d, cudaStream_t st);
// dz of classes first .. first + n - 1 divided by the largest weight, which goes to *scale.
int launch_few_dz(const XentRows& r, const Planes& h, const FewHead& w, int first, int n,
                  const float* lse, const float* gloss, const Planes& dz, float* scale,
                  const TrainDevice& d, cudaStream_t st);
// Sums of scale * dz w over `slices` parts of those classes: [slices][tokens][ld].
int launch_few_dh(const XentRows& r, const Planes& dz, const FewHead& w, int first, int n,
                  const float* scale, int slices, float* part, long long ld, const TrainDevice& d,
                  cudaStream_t st);

}  // namespace b2g
