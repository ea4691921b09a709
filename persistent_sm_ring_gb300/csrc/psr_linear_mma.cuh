// The matrix products of the linear layer on tcgen05 (sm_103a), C[i][j] = sum_k A(i, k) B(j, k).
//
// Either operand may be stored K-major (A[i][k]) or MN-major (A[k][i]); the shared-memory descriptors and the
// instruction descriptor take both, so no operand is transposed in memory: forward x w^T is K-major twice,
// dx = dz w has w MN-major, dw = dz^T x has both MN-major.  Two kernels:
//
//  * pair_gemm: a pair of CTAs (cta_group::2) computes tiles of 256 rows and 512 or 256 columns, each CTA 128 rows and 128
//    columns of each 256-column half.  512 columns fill tensor memory and move 48 B/clk per SM at the tensor rate, but the
//    next tile's products wait for the epilogue; 256 columns move 64 B/clk, and the accumulator is double-buffered.  The warps
//    that issue loads and products run converged, with one lane's predicate on those instructions, so that their operands
//    come from uniform registers: issued by a lane on its own, a K step of 64 took 330 ns instead of 273 (the products alone 265).
//  * stream_gemm: for few rows of A.  The output is computed transposed, W's rows on the 128 tensor memory lanes
//    and the tokens in the columns, so that W streams through once.  The (tile, K step) units are dealt out
//    evenly over one CTA per SM; a tile whose K range is split leaves fp32 partials that a second kernel joins.
//
// Both come in modes: what becomes of the sums in the linear layer, or in the loss of the output projection.
#pragma once
#include <algorithm>
#include <cfloat>
#include <mutex>
#include <type_traits>

#include "psr_control.cuh"
#include "psr_device.cuh"
#include "psr_gemm_tile.cuh"
#include "psr_host.h"

namespace psr {
namespace linear {

constexpr int kBK = 64;  // K per stage: one 128-byte swizzle atom of 16-bit elements
enum : uint32_t { SITE_FULL = 41, SITE_EMPTY = 42, SITE_ACC = 43, SITE_ACC_EMPTY = 44, SITE_LAUNCH = 45 };

// What becomes of an fp32 sum: z = sum + bias, y = act(z) + residual.
struct Epilogue {
  const void* bias;
  const void* res;
  void* y;
  void* z;
  long long ldr, ldy, ldz;
  int act;
  int half;  // fp16 (0: bf16)
  int vec;   // every row and column offset that the tiles use is 16-byte aligned
};

// Modes.  kLayer: the linear layer's epilogue.  The others serve the loss of the output projection, whose logits are the products of x
// and W: kStats reduces them to sums of exponentials, kSlope turns them into the loss's slope, kSum sends products of the slope
// with W into dx (over several pieces of W's rows), kWeight products of the slope with x into dw.
enum Mode { kLayer, kStats, kSlope, kSum, kWeight };

// What the loss's modes use besides.  In pair_gemm the rows that count are packed, and their number is known on the device alone.
struct Head {
  const int* rows;        // rows that count (kWeight: those summed over); null: the host's number
  const int* index;       // kSum: the row of dx of each
  // kStats, kSlope: the column of each row's target, of which the first here is col0 (stream_gemm: negative for a row that does not
  // count, whose slopes and whose dx are zeros whatever stands in W)
  const int* target;
  const int64_t* ids;     // (stream_gemm's kStats: the caller's)
  long long step;
  int col0;
  float2* stats;          // kStats: (r, s) of each row's columns in groups of kGroup (pair_gemm) or 32: sum exp(l) = s 2^r
  float* sums;            // the logits' sums in the same order, or null
  long long group_at, row_at;  // strides of those
  float* at;              // the targets' logits
  const float4* coef;     // kSlope, by row: lse log2(e), a, b, c: slope = a p - b - [target] c
  float* acc;             // kSum: fp32 sums of earlier pieces
  long long ldacc;
  int first, last;        // kSum: piece
  const float* unit;      // kSum, kWeight: what the sums are multiplied by at the end
};
constexpr float kLog2e = 1.4426950408889634f;

// sum exp(l) as s 2^r.  Any r would do; these stay finite where a logit is infinite.
struct ExpSum {
  float r, s;
};
__device__ __forceinline__ float exp_ref(float r, float most) { return fminf(fmaxf(r, most * kLog2e), FLT_MAX); }

// act(z) and act'(z) in fp32, branch-free: expf, erff and tanhf of the CUDA library cost the epilogue 30 to 40 issue
// slots an element (a 256-column half of a 1024-deep tile then waits on its epilogue).  The exponential and the reciprocal
// are the special function unit's (2^-22 each).
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float sigmoid(float x) { return rcp_approx(1.f + ex2_approx(-1.4426950408889634f * x)); }
// Phi(z); *e = exp(-z^2 / 2).  Phi(-|z|) = e t P(t), t = 1 / (1 + 0.295 |z|), P a polynomial of degree 5 whose coefficients a
// linear program fitted over |z| <= 14.5 for the least of the absolute error in units of 1e-7 and the relative one in units of
// 3e-5: as evaluated here it is off by at most 2.5e-7, and by 4e-5 of itself, so that the left tail keeps its digits too.
__device__ __forceinline__ float normal_cdf(float z, float* e) {
  const float t = rcp_approx(fmaf(0.295f, fabsf(z), 1.f));
  *e = ex2_approx(-0.72134752044448170f * z * z);
  float q = fmaf(-0.0838146742f, t, 0.251207165f);
  q = fmaf(q, t, -0.0539902122f);
  q = fmaf(q, t, 0.160338289f);
  q = fmaf(q, t, 0.107865875f);
  q = fmaf(q, t, 0.118393462f);
  const float h = q * t * *e;
  return z < 0.f ? h : 1.f - h;
}

// (1 + tanh u)/2 = sigmoid(2u), u = sqrt(2/pi) (z + 0.044715 z^3)
constexpr float kTwoU = 1.5957691216057307f, kCube = 0.044715f, kLog2eTwoU = 1.4426950408889634f * kTwoU;
__device__ __forceinline__ float tanh_cdf(float z, float z2) {
  return rcp_approx(1.f + ex2_approx(z * fmaf(-kLog2eTwoU * kCube, z2, -kLog2eTwoU)));
}

__device__ __forceinline__ float act_fwd(int act, float z) {
  switch (act) {
    case PSR_ACT_RELU: return z > 0.f ? z : (z == z ? 0.f : z);
    case PSR_ACT_GELU: {
      float e;
      return z * normal_cdf(z, &e);
    }
    case PSR_ACT_GELU_TANH: return z * tanh_cdf(z, z * z);
    case PSR_ACT_SILU: return z * sigmoid(z);
    default: return z;
  }
}
__device__ __forceinline__ float act_slope(int act, float z) {
  switch (act) {
    case PSR_ACT_RELU: return z > 0.f ? 1.f : 0.f;
    case PSR_ACT_GELU: {
      float e;
      const float f = normal_cdf(z, &e);
      return fmaf(z * 0.39894228040143268f, e, f);
    }
    case PSR_ACT_GELU_TANH: {
      const float z2 = z * z, s = tanh_cdf(z, z2), q = fmaf(-s, s, s);  // q: 0 far from 0, where z^2 may be infinite
      return q == 0.f ? s : fmaf(q, z * fmaf(3.f * kCube * kTwoU, z2, kTwoU), s);
    }
    case PSR_ACT_SILU: {
      const float s = sigmoid(z);
      return s * (1.f + z * (1.f - s));
    }
    default: return 1.f;
  }
}

// 16-bit elements of a type known at run time
__device__ __forceinline__ float load16(const void* p, long long i, int half) {
  return half ? __half2float(static_cast<const __half*>(p)[i]) : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void store16(void* p, long long i, int half, float v) {
  if (half) static_cast<__half*>(p)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}
__device__ __forceinline__ uint32_t pack16(float lo, float hi, int half) {
  if (!half) return pack_bf16x2(lo, hi);
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void unpack16(uint32_t v, int half, float& lo, float& hi) {
  if (half) {
    const float2 f = __half22float2(*reinterpret_cast<__half2*>(&v));
    lo = f.x;
    hi = f.y;
  } else {
    lo = __uint_as_float(v << 16);
    hi = __uint_as_float(v & 0xFFFF0000u);
  }
}

// One copy of the code for kernels that run their epilogue once: there, fetching instructions is what takes the time.
static __device__ __noinline__ float act_call(int act, float z) { return act_fwd(act, z); }
static __device__ __noinline__ float4 act_call4(int act, float4 z) {  // (side by side: 64 x 1024 x 64 with silu 14.0 to 9 us)
  auto apply = [&](auto a) {
    constexpr int A = decltype(a)::value;
    return make_float4(act_fwd(A, z.x), act_fwd(A, z.y), act_fwd(A, z.z), act_fwd(A, z.w));
  };
  switch (act) {
    case PSR_ACT_RELU: return apply(std::integral_constant<int, PSR_ACT_RELU>());
    case PSR_ACT_GELU: return apply(std::integral_constant<int, PSR_ACT_GELU>());
    case PSR_ACT_GELU_TANH: return apply(std::integral_constant<int, PSR_ACT_GELU_TANH>());
    case PSR_ACT_SILU: return apply(std::integral_constant<int, PSR_ACT_SILU>());
    default: return z;
  }
}

__device__ __forceinline__ void finish(const Epilogue& e, long long i, int j, float v) {
  if (e.bias) v += load16(e.bias, j, e.half);
  if (e.z) store16(e.z, i * e.ldz + j, e.half, v);
  if (e.act) v = act_call(e.act, v);
  if (e.res) v += load16(e.res, i * e.ldr + j, e.half);
  store16(e.y, i * e.ldy + j, e.half, v);
}

// Instruction descriptor: idesc_bf16_f32 with either operand MN-major and fp16 operands if `half`.
__host__ __device__ constexpr uint32_t idesc16(uint32_t M, uint32_t N, bool a_mn, bool b_mn, bool half) {
  return (idesc_bf16_f32(M, N, b_mn) | ((a_mn ? 1u : 0u) << 15)) & ~(half ? ((1u << 7) | (1u << 10)) : 0u);
}

// Descriptor low word of the 16-element K step kk of an operand tile of one stage: K-major rows of 128 bytes, or
// (MN) boxes of 64 K rows x 64 columns, 8 KiB apart.
template <bool MN>
__device__ __forceinline__ uint32_t operand_lo(uint32_t tile, int kk) {
  return MN ? sdesc_lo(tile + kk * 2048, 8192) : sdesc_lo(tile + kk * 32, 16);
}

// The products of one K step of 64 columns: four of 16, from the descriptors' low words of the first, issued by the lanes that have
// `lead` set (one).  PAIR: for a pair of CTAs.
template <bool PAIR, bool AMN, bool BMN>
__device__ __forceinline__ void mma_step(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate, uint32_t lead) {
#define PSR_MMA_STEP(GROUP)                                                                                          \
  asm volatile(                                                                                                      \
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"                                                                 \
      "setp.ne.b32 q, %6, 0;\n\t"                                                                                    \
      "setp.ne.b32 p, %5, 0;\n\t"                                                                                    \
      "mov.b64 a, {%1, %3};\n\t"                                                                                     \
      "mov.b64 b, {%2, %3};\n\t"                                                                                     \
      "@q tcgen05.mma.cta_group::" GROUP ".kind::f16 [%0], a, b, %4, p;\n\t"                                         \
      "setp.eq.b32 p, 0, 0;\n\t"                                                                                     \
      "add.s64 a, a, %7;\n\t"                                                                                        \
      "add.s64 b, b, %8;\n\t"                                                                                        \
      "@q tcgen05.mma.cta_group::" GROUP ".kind::f16 [%0], a, b, %4, p;\n\t"                                         \
      "add.s64 a, a, %7;\n\t"                                                                                        \
      "add.s64 b, b, %8;\n\t"                                                                                        \
      "@q tcgen05.mma.cta_group::" GROUP ".kind::f16 [%0], a, b, %4, p;\n\t"                                         \
      "add.s64 a, a, %7;\n\t"                                                                                        \
      "add.s64 b, b, %8;\n\t"                                                                                        \
      "@q tcgen05.mma.cta_group::" GROUP ".kind::f16 [%0], a, b, %4, p;\n\t}\n" ::"r"(d),                            \
      "r"(a), "r"(b), "r"(sdesc_hi_sw128(1024)), "r"(idesc), "r"(accumulate), "r"(lead), "n"(AMN ? 128 : 2),         \
      "n"(BMN ? 128 : 2)                                                                                             \
      : "memory")
  if constexpr (PAIR) PSR_MMA_STEP("2");
  else PSR_MMA_STEP("1");
#undef PSR_MMA_STEP
}
// Arrive on the barrier (of both CTAs of the pair) when the lane's products so far have completed.
__device__ __forceinline__ void commit_pair(uint64_t* bar, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %2, 0;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}\n" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void commit_one(uint64_t* bar, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(smem_u32(bar)),
      "r"(lead)
      : "memory");
}
__device__ __forceinline__ void load_one(uint32_t dst, const CUtensorMap* m, int x, int y, uint64_t* bar, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(smem_u32(bar)), "r"(lead)
      : "memory");
}

// An arrival at the pair's other CTA, and a meeting of the two, that do not order global memory between them: a release at
// cluster scope would wait until the thread's stores have been performed, a microsecond.  (What they order are reads of tensor
// memory, which have completed, and the CTAs' ends: before it leaves, a CTA has itself waited for every signal to its barriers.)
__device__ __forceinline__ void arrive_far(uint32_t cl_addr) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(cl_addr) : "memory");
}
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.relaxed;\n\tbarrier.cluster.wait;" ::: "memory");
}

// 32 lanes x 32 bits, 16 consecutive columns
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// ================================================================================================
// pair_gemm
// ================================================================================================
constexpr int kPairs = 76;           // pairs of CTAs that tiles are split for
constexpr int kRows = 128;           // A rows, and B rows of a half, that one CTA loads
constexpr int kHalf = kRows * kBK * 2;
// The logits of the loss are summed in parts of at most kPartSteps K steps, which the epilogue adds up: the tensor core's sums of
// 16 products and what they are added to lose a quarter of the last bit on average, towards zero, so that logits of 4096
// products came out 3.9e-6 of themselves too small (of 1024, 8e-7), and their log-sum-exp 2.4e-5.  A part of 1024 takes the tensor
// core ten times as long as the epilogue takes to add it.
__host__ __device__ constexpr bool in_parts(int mode) { return mode == kStats || mode == kSlope; }
constexpr int kPartSteps = 16;
__host__ __device__ constexpr int part_steps(int n_k) {  // of all parts but the last
  const int parts = (n_k + kPartSteps - 1) / kPartSteps;
  return (n_k + parts - 1) / parts;
}
// Epilogue warps: four to a scheduler, an epilogue block being a chain of latencies; two where a thread keeps the sums of 128
// columns over the parts (168 registers instead of 96), which gives it independent work enough.
__host__ __device__ constexpr int epi_warps(int mode) { return in_parts(mode) ? 8 : 16; }
__host__ __device__ constexpr int pair_threads(int mode) { return (4 + epi_warps(mode)) * 32; }
constexpr int kGroup = 1024 / epi_warps(kStats);  // columns of a thread
constexpr int kEpiWarpBytes = 2048;  // one warp's 32 rows x 64 bytes
// The stages are cut into chunks of one operand tile (16 KiB) each: a K step takes 2 of them (one 256-column half) or 3, so
// that either way all 192 KiB are in flight (4 steps of 48 KiB would leave one half 128 KiB, which bounds it).
constexpr int kChunks = 12;
constexpr int kSteps = 8;  // barriers; more than K steps in flight
constexpr int kPairSmem = 1024 + kChunks * kHalf + epi_warps(kLayer) * kEpiWarpBytes;
static_assert(kPairSmem + 1024 <= 232448, "shared memory");

struct PairParams {
  int M, N, n_k;
  int wide;               // tiles of 512 columns, else 256
  int tiles_m, tiles_n;   // tile rows of 256, tile columns
  int group;              // tile rows of a raster group
  int whole;              // of 256-column tiles: those computed whole, in whole rounds; the others are split
  int splits, split_k;    // parts of a split tile's K steps, K steps of a part
  int halves;             // of 512-column tiles: those of the last round that are computed as two halves (pair_item)
  float* partial;         // splits > 1: fp32 sums [split tile][part][256][256]
  uint32_t idesc;
  Epilogue e;
  Ctrl* ctrl;
  Ctrl* clear;            // control block to clear, or null
  unsigned long long timeout_ns;
  int n_pairs;
  Head h;
};

struct PairSmem {
  uint64_t full[kSteps], empty[kSteps], acc_full[2], acc_empty[2], drain;
  uint32_t tmem_base;
  volatile uint32_t abort;
};

// A product's rows, K steps and tiles: the host's, or (rows that count) what the device makes of their number.
struct Extent {
  int M, n_k, wide, tiles_m, tiles_n, whole, splits, split_k, halves;  // as in PairParams, which stand for themselves (X below)
};

// What a pair computes next: `n` 256-column halves from column half tn on of tile row tm, K steps k0 .. k0 + n_k.  split: the part
// (of all split tiles') whose sums go to the partials, or -1.
struct PairItem {
  int tm, tn, n, k0, n_k, split;
};

// Tile t -> (row block, column block): groups of `group` tile rows, columns inside a group, rows fastest, so that the
// tiles in flight at once share few rows of either operand and a group's rows of A stay in L2.
template <class X>
__device__ __forceinline__ void pair_tile(const PairParams& p, const X& x, int t, int& tm, int& tn) {
  const int per = p.group * x.tiles_n, g = t / per, r = t - g * per;
  const int rows = min(p.group, x.tiles_m - g * p.group);
  tn = r / rows;
  tm = g * p.group + (r - tn * rows);
}

// Item i of a pair; false past its last: the tiles stride over the pairs.  The tiles of the last round, where no more than
// half of the pairs would have one, are dealt out as 256-column halves (256 tiles of 512 columns on 76 pairs: three rounds and
// a half, not four).  Rounds shifted by half a tile between pairs, so that some write while others multiply, were
// slower: the tile loads leave L2 no room for the outputs (4096^3 with gelu 100 to 118 us).
template <class X>
__device__ __forceinline__ bool pair_item(const PairParams& p, const X& x, int pair, int n_pairs, int i, PairItem& it) {
  const long long n = (long long)x.tiles_m * x.tiles_n, at = pair + (long long)i * n_pairs;
  it.k0 = 0;
  it.n_k = x.n_k;
  it.split = -1;
  if (!x.wide) {
    it.n = 1;
    int tile = (int)at;
    if (at >= x.whole) {
      const long long part = at - x.whole;
      if (part >= (n - x.whole) * x.splits) return false;
      tile = x.whole + (int)(part / x.splits);
      if (x.splits > 1) {
        it.split = (int)part;
        it.k0 = (int)(part % x.splits) * x.split_k;
        it.n_k = min(x.split_k, x.n_k - it.k0);
      }
    }
    pair_tile(p, x, tile, it.tm, it.tn);
    return true;
  }
  const long long whole = n - x.halves;  // tiles in whole rounds
  const int h = (int)(at - whole);
  if (h >= 2 * x.halves) return false;
  pair_tile(p, x, h < 0 ? (int)at : (int)whole + h / 2, it.tm, it.tn);
  it.tn = 2 * it.tn + (h < 0 ? 0 : h % 2);
  it.n = h < 0 && (it.tn + 1) * 256 < p.N ? 2 : 1;  // the last columns may be one half wide
  return true;
}

// One 128-row operand tile of a stage, asked for by the lanes that have `lead` set (one).
__device__ __forceinline__ void load_pair(uint32_t dst, const CUtensorMap* m, int x, int y, uint32_t bar, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];\n\t}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar), "r"(lead)
      : "memory");
}
template <bool MN>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap* m, int k, int row, uint32_t bar, uint32_t lead) {
  if constexpr (MN) {
    load_pair(dst, m, row, k, bar, lead);
    load_pair(dst + 8192, m, row + 64, k, bar, lead);
  } else {
    load_pair(dst, m, k, row, bar, lead);
  }
}

// A warp's 32 rows x 32 columns of 16-bit elements, or 32 x 16 of fp32, between global memory and its staging area: 64
// bytes of a row, whose four 16-byte chunks are XOR-swizzled by the row so that row-wise and column-wise passes are both
// free of bank conflicts.  Lane l holds chunk l % 4 of rows k * 8 + l / 4.
__device__ __forceinline__ uint4* stage_chunk(uint8_t* stage, int row, int c) {
  return reinterpret_cast<uint4*>(stage + row * 64 + ((c ^ ((row >> 1) & 3)) * 16));
}
// 16-byte columns below `chunks` of rows below `rows`.  PASS: nothing reads them soon (the loss's dw: 40 rows of 32000 columns with
// gradients 147 to 145 us).
template <bool PASS = false>
__device__ __forceinline__ void rows_out(uint8_t* stage, uint8_t* g, long long pitch, int rows, int chunks) {
  const int lane = threadIdx.x % 32, c = lane % 4;
  __syncwarp();
  g += (long long)(lane / 4) * pitch + c * 16;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int r = k * 8 + lane / 4;
    const uint4 w = *stage_chunk(stage, r, c);
    if (r < rows && c < chunks) {
      if constexpr (PASS) __stcs(reinterpret_cast<uint4*>(g), w);
      else *reinterpret_cast<uint4*>(g) = w;
    }
    g += 8 * pitch;
  }
  __syncwarp();
}
__device__ __forceinline__ void rows_in(uint4 (&w)[4], const uint8_t* g, long long pitch, int rows, int chunks) {
  const int lane = threadIdx.x % 32, c = lane % 4;
  g += (long long)(lane / 4) * pitch + c * 16;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    w[k] = make_uint4(0, 0, 0, 0);
    if (k * 8 + lane / 4 < rows && c < chunks) w[k] = *reinterpret_cast<const uint4*>(g);
    g += 8 * pitch;
  }
}
// The same for rows that are not 16-byte aligned: a row of 32 columns at a time, a column to a lane.
__device__ __forceinline__ uint16_t* stage_element(uint8_t* stage, int row, int c) {
  return reinterpret_cast<uint16_t*>(stage_chunk(stage, row, c / 8)) + c % 8;
}
__device__ __forceinline__ void rows_out_odd(uint8_t* stage, uint16_t* g, long long ld, int rows, int cols) {
  const int lane = threadIdx.x % 32;
  __syncwarp();
#pragma unroll 4
  for (int r = 0; r < rows; ++r)
    if (lane < cols) g[r * ld + lane] = *stage_element(stage, r, lane);
  __syncwarp();
}
__device__ __forceinline__ void rows_in_odd(uint8_t* stage, const uint16_t* g, long long ld, int rows, int cols) {
  const int lane = threadIdx.x % 32;
#pragma unroll 4
  for (int r = 0; r < rows; ++r)
    if (lane < cols) *stage_element(stage, r, lane) = g[r * ld + lane];
  __syncwarp();
}
__device__ __forceinline__ void add16(uint32_t* v, const uint4& b, int half) {
  const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float lo, hi;
    unpack16(w[q], half, lo, hi);
    v[2 * q] = __float_as_uint(__uint_as_float(v[2 * q]) + lo);
    v[2 * q + 1] = __float_as_uint(__uint_as_float(v[2 * q + 1]) + hi);
  }
}

// The block's 32 rows x 32 columns at (i0, j0), row `lane` in v: bias, z, activation, residual (its rows in `res`, as
// rows_in read them), y.  ACT: there may be an activation (the gradients have none).  HALF: fp16 (both
// types behind a test cost a bias or a residual 700 clocks a block, the epilogue being bound by its instructions).
template <bool ACT, bool HALF>
__device__ __forceinline__ void pair_store(const Epilogue& e, int M, int N, uint8_t* stage, int i0, int j0,
                                           uint32_t (&v)[32], const uint4 (&res)[4]) {
  const int lane = threadIdx.x % 32;
  const int rows = min(32, M - i0), cols = min(32, N - j0);
  if (rows <= 0 || cols <= 0) return;
  if (e.bias) {
    if (e.vec) {
      const uint4* b = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(e.bias) + j0);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j * 8 < cols) add16(v + 8 * j, b[j], HALF);
    } else {
#pragma unroll
      for (int c = 0; c < 32; ++c)
        if (c < cols) v[c] = __float_as_uint(__uint_as_float(v[c]) + load16(e.bias, j0 + c, HALF));
    }
  }
  auto out = [&](void* base, long long ld) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        w[q] = pack16(__uint_as_float(v[j * 8 + 2 * q]), __uint_as_float(v[j * 8 + 2 * q + 1]), HALF);
      *stage_chunk(stage, lane, j) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    uint16_t* g = static_cast<uint16_t*>(base) + (long long)i0 * ld + j0;
    if (e.vec) rows_out(stage, reinterpret_cast<uint8_t*>(g), ld * 2, rows, cols / 8);
    else rows_out_odd(stage, g, ld, rows, cols);
  };
  if (e.z) out(e.z, e.ldz);
  if constexpr (ACT) {
    auto apply = [&](auto act) {
#pragma unroll
      for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(act_fwd(decltype(act)::value, __uint_as_float(v[c])));
    };
    switch (e.act) {
      case PSR_ACT_RELU: apply(std::integral_constant<int, PSR_ACT_RELU>()); break;
      case PSR_ACT_GELU: apply(std::integral_constant<int, PSR_ACT_GELU>()); break;
      case PSR_ACT_GELU_TANH: apply(std::integral_constant<int, PSR_ACT_GELU_TANH>()); break;
      case PSR_ACT_SILU: apply(std::integral_constant<int, PSR_ACT_SILU>()); break;
      default: break;
    }
  }
  if (e.res) {
    if (e.vec) {
#pragma unroll
      for (int k = 0; k < 4; ++k) *stage_chunk(stage, k * 8 + lane / 4, lane % 4) = res[k];
      __syncwarp();
    } else {
      rows_in_odd(stage, static_cast<const uint16_t*>(e.res) + (long long)i0 * e.ldr + j0, e.ldr, rows, cols);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) add16(v + 8 * j, *stage_chunk(stage, lane, j), HALF);  // (columns past `cols` are not stored)
    __syncwarp();
  }
  out(e.y, e.ldy);
}

// The first `rows` rows of the block's fp32 sums into the part's partials, at (row, col) of the tile.
__device__ __forceinline__ void partial_store(const PairParams& p, int split, uint8_t* stage, int row, int col, int rows,
                                              const uint32_t (&v)[32]) {
  const int lane = threadIdx.x % 32;
  if (rows <= 0) return;
  float* g = p.partial + ((long long)split * 256 + row) * 256 + col;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t* w = v + h * 16 + j * 4;
      *stage_chunk(stage, lane, j) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    rows_out(stage, reinterpret_cast<uint8_t*>(g + h * 16), 1024, rows, 4);
  }
}

// Tiles of the last round that are dealt out as halves.
__host__ __device__ inline int last_halves(long long tiles, int pairs) {
  const long long rest = tiles % pairs;
  return 2 * rest <= pairs ? (int)rest : 0;
}

// The product as the device knows it: with the number of rows that count.  (Not a changed copy of the parameters: one kept the row
// count that the host had given.)  dx, whose tiles are few and whose sums are long, has its tiles chosen here, as wide_tiles and split_of
// choose others on the host: 512 columns, or 256 with those of the last round split along K.
template <int MODE>
__device__ __forceinline__ Extent extent_of(const PairParams& p, int n_pairs) {
  Extent x = {p.M, p.n_k, p.wide, p.tiles_m, p.tiles_n, p.whole, p.splits, p.split_k, p.halves};
  if (!p.h.rows) return x;
  const int rows = *p.h.rows;
  if (MODE == kWeight) {
    x.n_k = (rows + kBK - 1) / kBK;
    return x;
  }
  x.M = rows;
  x.tiles_m = (rows + 255) / 256;
  if (MODE == kSum) {
    const int ones = x.tiles_m * ((p.N + 255) / 256), twos = x.tiles_m * ((p.N + 511) / 512), rest = ones % kPairs;
    const int halves = last_halves(twos, n_pairs), most = x.n_k / 8;
    // in tenths of a clock, whole numbers: pair_gemm and pair_join, compiled apart, decide alike where two ways cost the same
    const long long k = p.n_k * (long long)kBK, step = 93 * k;
    int parts = rest ? min(kPairs / rest, most) : 1;
    const long long join = 55000 + 1800 * rest * parts;
    if (parts < 2 || 86 * k * (parts - 1) < join * parts) parts = 1;
    const long long one = parts > 1 ? ones / kPairs * step + step / parts + join : (ones + n_pairs - 1) / n_pairs * step;
    const long long two = (twos / n_pairs + (halves || twos % n_pairs == 0 ? 0 : 1)) * (160 * k + 156000) + (halves ? step + 78000 : 0);
    x.wide = two <= one;
    x.tiles_n = x.wide ? (p.N + 511) / 512 : (p.N + 255) / 256;
    x.whole = x.wide ? twos : ones - (parts > 1 ? rest : 0);
    x.split_k = (x.n_k + parts - 1) / parts;
    x.splits = x.wide ? 1 : (x.n_k + x.split_k - 1) / x.split_k;  // none of them empty
    x.halves = x.wide ? halves : 0;
    return x;
  }
  const int tiles = x.tiles_m * x.tiles_n;
  if (x.wide) x.halves = last_halves(tiles, n_pairs);
  else x.whole = min(x.whole, tiles);
  return x;
}

template <int MODE>
__device__ __forceinline__ decltype(auto) pair_extent(const PairParams& p, int n_pairs) {
  if constexpr (MODE == kLayer) return (p);
  else return extent_of<MODE>(p, n_pairs);
}

// What a thread keeps of its row over the blocks of its columns.
struct HeadRow {
  int target;  // column (kSum: row of dx)
  float4 coef;
  ExpSum e;
  float sum;
};
template <int MODE>
__device__ __forceinline__ void head_row(const PairParams& p, int M, int i, HeadRow& r) {
  r.target = -1;
  r.coef = make_float4(0.f, 0.f, 0.f, 0.f);
  if (i >= M) return;
  if constexpr (MODE == kStats || MODE == kSlope) r.target = p.h.target[i] - p.h.col0;
  if constexpr (MODE == kSlope) r.coef = p.h.coef[i];
  if constexpr (MODE == kSum) r.target = p.h.index[i];
}

// (the first to leave L2: nothing reads it soon)
__device__ __forceinline__ void store_tile(const CUtensorMap* m, int x, int y, uint32_t src) {
  asm volatile(
      "{\n\t.reg .b64 p;\n\t"
      "createpolicy.fractional.L2::evict_first.b64 p, 1.0;\n\t"
      "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group.L2::cache_hint [%0, {%1, %2}], [%3], p;\n\t}\n" ::"l"(reinterpret_cast<uint64_t>(m)),
      "r"(x), "r"(y), "r"(src)
      : "memory");
}

// What pair_gemm has besides.  kWeight: up to kCopySteps K steps, where dw's stores bound it, a block goes out by one copy from the
// staging area, whose swizzle is that of 64-byte rows (dw of 40 rows, 32000 x 2048, 33 to 26 us, 4.0 to 5 TB/s; the stores of the same
// by threads keep the shared memory pipe 72 % busy).  With more steps the copies hold up the operands' (400 rows with both gradients 164
// and 169 us).
constexpr int kCopySteps = 2;
template <int MODE>
struct Out {};
template <>
struct Out<kWeight> {
  CUtensorMap map;
  int copies;
};

// The block's 32 rows from i0 on, row `lane` in v, to e.y in 16 bits; kSum: to the row `to` of each.
template <int MODE, bool HALF>
__device__ __forceinline__ void head_out(const Epilogue& e, const Out<MODE>& out, int to, uint8_t* stage, int i0, int j0, int rows, int cols,
                                         const uint32_t (&v)[32]) {
  const int lane = threadIdx.x % 32;
  if constexpr (MODE == kWeight) {  // the copy of the last block has read it
    if (out.copies && lane == 0) bulk_wait_read<0>();
    __syncwarp();
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      w[q] = pack16(__uint_as_float(v[j * 8 + 2 * q]), __uint_as_float(v[j * 8 + 2 * q + 1]), HALF);
    *stage_chunk(stage, lane, j) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if constexpr (MODE == kWeight) {
    if (out.copies) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        store_tile(&out.map, j0, i0, smem_u32(stage));
        bulk_commit();
      }
      return;
    }
  }
  uint16_t* g = static_cast<uint16_t*>(e.y) + j0;
  if constexpr (MODE != kSum) {
    g += (long long)i0 * e.ldy;
    if (e.vec) rows_out<MODE == kWeight>(stage, reinterpret_cast<uint8_t*>(g), e.ldy * 2, rows, (cols + 7) / 8);
    else rows_out_odd(stage, g, e.ldy, rows, cols);
    return;
  }
  __syncwarp();
  if (e.vec) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = k * 8 + lane / 4, c = lane % 4;
      const long long row = __shfl_sync(0xffffffffu, to, r);
      const uint4 w = *stage_chunk(stage, r, c);
      if (r < rows && c * 8 < cols) *reinterpret_cast<uint4*>(g + row * e.ldy + c * 8) = w;
    }
  } else {
    for (int r = 0; r < rows; ++r) {
      const long long row = __shfl_sync(0xffffffffu, to, r);
      if (lane < cols) g[row * e.ldy + lane] = *stage_element(stage, r, lane);
    }
  }
  __syncwarp();
}

// Block b of a warp's columns: 32 rows x 32 columns of sums at (i0, j0), row `lane` in v.
template <int MODE, bool HALF>
__device__ __forceinline__ void head_store(const PairParams& p, const Out<MODE>& out, int M, uint8_t* stage, int i0, int j0, int b, HeadRow& row,
                                           uint32_t (&v)[32]) {
  const int lane = threadIdx.x % 32, i = i0 + lane, cols = min(32, p.N - j0);
  if constexpr (MODE == kStats) {
    if (b == 0) {
      row.e = {-FLT_MAX, 0.f};
      row.sum = 0.f;
    }
    if (cols > 0) {
      if (p.h.sums) {
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (c < cols) row.sum += __uint_as_float(v[c]);
      }
      if (cols < 32) {
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (c >= cols) v[c] = 0xFF800000u;
      }
      float m[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) m[c] = __uint_as_float(v[c]);
#pragma unroll
      for (int c = 4; c < 32; ++c) m[c % 4] = fmaxf(m[c % 4], __uint_as_float(v[c]));
      const float ref = exp_ref(row.e.r, fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])));
      float s[4] = {row.e.s * ex2_approx(row.e.r - ref), 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 32; ++c) s[c % 4] += ex2_approx(fmaf(__uint_as_float(v[c]), kLog2e, -ref));
      row.e = {ref, (s[0] + s[1]) + (s[2] + s[3])};
      const int at = row.target - j0;
      const bool here = at >= 0 && at < cols;
      if (__any_sync(0xffffffffu, here)) {
        uint32_t l = 0;
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (c == at) l = v[c];
        if (here) p.h.at[i] = __uint_as_float(l);
      }
    }
    const int group = j0 / kGroup;
    if (b == kGroup / 32 - 1 && i < M && group * kGroup < p.N) {
      const long long to = group * p.h.group_at + i * p.h.row_at;
      p.h.stats[to] = make_float2(row.e.r, row.e.s);
      if (p.h.sums) p.h.sums[to] = row.sum;
    }
  } else if constexpr (MODE == kSlope) {
    // zeros for the rows up to the K step of dw's product that the last one is in
    const int rows = min(32, (M + kBK - 1) / kBK * kBK - i0);
    if (rows <= 0 || cols <= 0) return;
    const bool counts = i < M;
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      const float q = ex2_approx(fmaf(__uint_as_float(v[c]), kLog2e, -row.coef.x));
      v[c] = counts ? __float_as_uint(fmaf(row.coef.y, q, -row.coef.z)) : 0u;
    }
    const int at = row.target - j0;
    if (__any_sync(0xffffffffu, at >= 0 && at < cols)) {
#pragma unroll
      for (int c = 0; c < 32; ++c)
        if (c == at) v[c] = __float_as_uint(__uint_as_float(v[c]) - row.coef.w);
    }
    head_out<MODE, HALF>(p.e, out, 0, stage, i0, j0, rows, cols, v);
  } else {
    const int rows = min(32, M - i0);
    if (rows <= 0 || cols <= 0) return;
    if constexpr (MODE == kSum) {
      uint8_t* g = reinterpret_cast<uint8_t*>(p.h.acc + (long long)i0 * p.h.ldacc + j0);
      const long long pitch = p.h.ldacc * 4;
      if (!p.h.first) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint4 w[4];
          rows_in(w, g + h * 64, pitch, rows, (cols - 16 * h + 3) / 4);
#pragma unroll
          for (int k = 0; k < 4; ++k) *stage_chunk(stage, k * 8 + lane / 4, lane % 4) = w[k];
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 a = *stage_chunk(stage, lane, j);
            uint32_t* to = v + 16 * h + 4 * j;
            to[0] = __float_as_uint(__uint_as_float(to[0]) + __uint_as_float(a.x));
            to[1] = __float_as_uint(__uint_as_float(to[1]) + __uint_as_float(a.y));
            to[2] = __float_as_uint(__uint_as_float(to[2]) + __uint_as_float(a.z));
            to[3] = __float_as_uint(__uint_as_float(to[3]) + __uint_as_float(a.w));
          }
          __syncwarp();
        }
      }
      if (!p.h.last) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t* w = v + h * 16 + j * 4;
            *stage_chunk(stage, lane, j) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          rows_out(stage, g + h * 64, pitch, rows, (cols - 16 * h + 3) / 4);
        }
        return;
      }
    }
    const float unit = *p.h.unit;
#pragma unroll
    for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) * unit);
    head_out<MODE, HALF>(p.e, out, row.target, stage, i0, j0, rows, cols, v);
  }
}

template <bool AMN, bool BMN, bool HALF, int MODE = kLayer>
__global__ void __launch_bounds__(pair_threads(MODE), 1)
    pair_gemm(const __grid_constant__ PairParams p, const __grid_constant__ CUtensorMap ma,
              const __grid_constant__ CUtensorMap mb, const __grid_constant__ Out<MODE> out) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ PairSmem sc;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t smem_base = (raw + 1023u) & ~1023u;
  uint8_t* epi = smem_raw + (smem_base - raw) + kChunks * kHalf;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;  // (uniform, for the compiler)
  uint32_t n_rank;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n_rank));
  if (n_rank != 2u) {  // no caller launches it without pairs
    if (threadIdx.x == 0) raise_error(p, SITE_LAUNCH);
    return;
  }
  const uint32_t rank = __shfl_sync(0xffffffffu, cluster_ctarank(), 0);
  clear_ctrl(p.clear);
  launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kSteps; ++s) {
      mbar_init(&sc.full[s], 1);
      mbar_init(&sc.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sc.acc_full[b], 1);
      mbar_init(&sc.acc_empty[b], 2 * epi_warps(MODE));
    }
    mbar_init(&sc.drain, 1);
    sc.abort = 0;
    fence_barrier_init();
    prefetch_tmap(&ma);
    prefetch_tmap(&mb);
  }
  if (warp == 1) {
    tmem_alloc_cg<2>(&sc.tmem_base, 512);
    tmem_relinquish_cg<2>();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();

  const int pair = blockIdx.x / 2, n_pairs = gridDim.x / 2;
  if constexpr (MODE != kLayer) wait_previous();  // the loss's kernels begin while the one before ends
  auto&& x = pair_extent<MODE>(p, n_pairs);
  const uint32_t full0 = __shfl_sync(0xffffffffu, mapa_shared(smem_u32(&sc.full[0]), 0), 0);  // of the pair's first CTA
  PairItem it;
  if (warp == 0) {  // the whole warp, for the same reason as the next one
    uint32_t head = 0, tail = 0, chunk = 0, used = 0, wide = 0;  // steps issued and known read, chunks, step sizes
    bool ok = true;
    for (int i = 0; ok && pair_item(p, x, pair, n_pairs, i, it); ++i) {
      const int arow = it.tm * 256 + (int)rank * kRows, brow = it.tn * 256 + (int)rank * kRows;
      const uint32_t n = 1 + it.n;
      for (int ks = it.k0; ks < it.k0 + it.n_k; ++ks) {
        while (used + n > kChunks) {  // the oldest step gives its chunks back (at most 6 are in flight)
          const uint32_t s = tail % kSteps;
          ok = __all_sync(0xffffffffu, wait_own(&sc.empty[s], (tail / kSteps) & 1u, p, &sc, SITE_EMPTY));
          if (!ok) break;
          used -= 2 + (wide >> s & 1u);
          ++tail;
        }
        if (!ok) break;
        const uint32_t s = head % kSteps;
        wide = (wide & ~(1u << s)) | ((n - 2) << s);
        if (rank == 0 && lane == 0) mbar_expect_tx(&sc.full[s], 2 * n * kHalf);  // both CTAs' bytes
        const uint32_t bar = full0 + s * 8;
        auto next = [&]() {
          const uint32_t at = smem_base + chunk * kHalf;
          chunk = chunk + 1 == kChunks ? 0 : chunk + 1;
          return at;
        };
        load_operand<AMN>(next(), &ma, ks * kBK, arow, bar, lane == 0);
        load_operand<BMN>(next(), &mb, ks * kBK, brow, bar, lane == 0);
        if (it.n == 2) load_operand<BMN>(next(), &mb, ks * kBK, brow + 256, bar, lane == 0);
        used += n;
        ++head;
      }
    }
    for (; ok && tail < head; ++tail)  // every signal to this CTA's barriers has come before it may leave
      ok = __all_sync(0xffffffffu, wait_own(&sc.empty[tail % kSteps], (tail / kSteps) & 1u, p, &sc, SITE_EMPTY));
    if (!ok) sc.abort = 1;
  } else if (warp == 1) {
    if (rank == 0) {  // the whole warp, so that addresses and descriptors stay in uniform registers; lane 0 issues
      const uint32_t tmem = sc.tmem_base;
      const uint32_t a0 = operand_lo<AMN>(smem_base, 0), b0 = operand_lo<BMN>(smem_base, 0);
      uint32_t c = 0, chunk = 0, u = 0;  // steps and chunks consumed, accumulator halves begun
      bool ok = true;
      auto next = [&]() {
        const uint32_t at = chunk * (kHalf / 16);
        chunk = chunk + 1 == kChunks ? 0 : chunk + 1;
        return at;
      };
      for (int i = 0; ok && pair_item(p, x, pair, n_pairs, i, it); ++i) {
        if constexpr (in_parts(MODE)) {  // tiles of 256 columns, a part to an accumulator
          const int steps = part_steps(it.n_k);
          for (int k0 = 0; k0 < it.n_k && ok; k0 += steps, ++u) {
            const uint32_t slot = u % 2;
            if (u >= 2) ok = __all_sync(0xffffffffu, wait_own<true>(&sc.acc_empty[slot], (u / 2 - 1) & 1u, p, &sc, SITE_ACC_EMPTY));
            if (!ok) break;
            tc_fence_after();
            for (int ks = k0; ks < min(it.n_k, k0 + steps); ++ks, ++c) {
              const uint32_t s = c % kSteps;
              ok = __all_sync(0xffffffffu, wait_own(&sc.full[s], (c / kSteps) & 1u, p, &sc, SITE_FULL));
              if (!ok) break;
              tc_fence_after();
              const uint32_t a = a0 + next(), b = b0 + next();
              mma_step<true, AMN, BMN>(tmem + slot * 256, a, b, p.idesc, ks > k0, lane == 0);
              commit_pair(&sc.empty[s], lane == 0);
            }
            if (ok) commit_pair(&sc.acc_full[slot], lane == 0);
          }
        } else {
          for (int ks = 0; ks < it.n_k && ok; ++ks, ++c) {
            const uint32_t s = c % kSteps;
            ok = __all_sync(0xffffffffu, wait_own(&sc.full[s], (c / kSteps) & 1u, p, &sc, SITE_FULL));
            if (!ok) break;
            tc_fence_after();
            const uint32_t a = a0 + next();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (h >= it.n) break;
              const uint32_t slot = (u + h) % 2, b = b0 + next();
              if (ks == 0) {  // the half's previous sums have been read back
                if (u + h >= 2)
                  ok = __all_sync(0xffffffffu, wait_own<true>(&sc.acc_empty[slot], ((u + h) / 2 - 1) & 1u, p, &sc, SITE_ACC_EMPTY));
                if (!ok) break;
                tc_fence_after();
              }
              mma_step<true, AMN, BMN>(tmem + slot * 256, a, b, p.idesc, ks > 0, lane == 0);
            }
            if (!ok) break;
            commit_pair(&sc.empty[s], lane == 0);
          }
          if (!ok) break;
          if (MODE == kWeight && it.n_k == 0) continue;
          for (int h = 0; h < it.n; ++h) commit_pair(&sc.acc_full[(u + h) % 2], lane == 0);
          u += it.n;
        }
      }
      for (uint32_t h = u > 2 ? u - 2 : 0; ok && h < u; ++h)  // the other CTA's last arrivals have come
        ok = __all_sync(0xffffffffu, wait_own<true>(&sc.acc_empty[h % 2], (h / 2) & 1u, p, &sc, SITE_ACC_EMPTY));
      if (!ok) sc.abort = 1;
    }
  } else if (warp >= 4) {
    uint8_t* stage = epi + (warp - 4) * kEpiWarpBytes;
    const int quarter = warp % 4, cgroup = (warp - 4) / 4;  // lanes 32 quarter .., columns 64 cgroup .. of a half
    const Epilogue& e = p.e;
    const bool res = MODE == kLayer && e.res && e.vec;
    uint32_t u = 0;
    bool ok = true;
    for (int i = 0; ok && pair_item(p, x, pair, n_pairs, i, it); ++i) {
      const int i0 = it.tm * 256 + (int)rank * kRows + quarter * 32;
      HeadRow row;
      if constexpr (MODE != kLayer) head_row<MODE>(p, x.M, i0 + lane, row);
      if (MODE == kWeight && it.n_k == 0) {  // sums over no rows: nothing is multiplied, nothing signalled
        for (int b = 0; b < 2 * it.n; ++b) {
          uint32_t v[32] = {};
          head_store<MODE, HALF>(p, out, x.M, stage, i0, it.tn * 256 + (b / 2) * 256 + cgroup * 64 + (b % 2) * 32, 0, row, v);
        }
        continue;
      }
      if constexpr (in_parts(MODE)) {
        uint32_t sum[kGroup / 32][32];
        for (int k0 = 0; k0 < p.n_k; k0 += part_steps(p.n_k), ++u) {
          ok = __all_sync(0xffffffffu, wait_own(&sc.acc_full[u % 2], (u / 2) & 1u, p, &sc, SITE_ACC));
          if (!ok) break;
          tc_fence_after();
          const uint32_t from = sc.tmem_base + ((uint32_t)(quarter * 32) << 16) + u % 2 * 256 + cgroup * kGroup;
          if (k0 == 0) {
#pragma unroll
            for (int q = 0; q < kGroup / 32; ++q) tmem_ld32(from + q * 32, sum[q]);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int q = 0; q < kGroup / 16; ++q) {
              uint32_t v[16];
              tmem_ld16(from + q * 16, v);
              tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < 16; ++c) {
                uint32_t& to = sum[q / 2][q % 2 * 16 + c];
                to = __float_as_uint(__uint_as_float(to) + __uint_as_float(v[c]));
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (rank == 0) mbar_arrive(&sc.acc_empty[u % 2]);
            else arrive_far(mapa_shared(smem_u32(&sc.acc_empty[u % 2]), 0));
          }
        }
        if (!ok) break;
#pragma unroll
        for (int q = 0; q < kGroup / 32; ++q)
          head_store<MODE, HALF>(p, out, x.M, stage, i0, it.tn * 256 + cgroup * kGroup + q * 32, q, row, sum[q]);
      } else {
#pragma unroll 1
        for (int b = 0; b < 2 * it.n && ok; ++b) {
          const uint32_t slot = u % 2;
          const int j0 = it.tn * 256 + (b / 2) * 256 + cgroup * 64 + (b % 2) * 32;
          uint4 rr[4];
          if (res && it.split < 0)  // in flight while the sums are waited for
            rows_in(rr, static_cast<const uint8_t*>(e.res) + ((long long)i0 * e.ldr + j0) * 2, e.ldr * 2, x.M - i0, (p.N - j0) / 8);
          if (b % 2 == 0) {
            ok = __all_sync(0xffffffffu, wait_own(&sc.acc_full[slot], (u / 2) & 1u, p, &sc, SITE_ACC));
            if (!ok) break;
            tc_fence_after();
          }
          uint32_t v[32];
          tmem_ld32(sc.tmem_base + ((uint32_t)(quarter * 32) << 16) + slot * 256 + cgroup * 64 + (b % 2) * 32, v);
          tmem_ld_wait();
          if (b % 2 == 1) {  // this warp's share of the half is in registers
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if (rank == 0) mbar_arrive(&sc.acc_empty[slot]);
              else arrive_far(mapa_shared(smem_u32(&sc.acc_empty[slot]), 0));
            }
            ++u;
          }
          if (it.split >= 0)
            partial_store(p, it.split, stage, (int)rank * kRows + quarter * 32, cgroup * 64 + (b % 2) * 32, x.M - i0, v);
          else if constexpr (MODE == kLayer) pair_store<!BMN, HALF>(e, x.M, p.N, stage, i0, j0, v, rr);
          else head_store<MODE, HALF>(p, out, x.M, stage, i0, j0, 0, row, v);
        }
      }
    }
    if (MODE == kWeight && lane == 0) bulk_wait<0>();  // dw has been written
    if (!ok) sc.abort = 1;
  }
  // Every tcgen05 op has completed before tensor memory is released.  Every load has landed then too, the products having
  // waited for it; after a wait that gave up, the loads in flight get two milliseconds.
  if (warp == 1 && lane == 0 && rank == 0) {
    mma_commit_cg<2>(&sc.drain, 1);
    wait_last(&sc.drain, 0);
  }
  __syncthreads();
  if (sc.abort && threadIdx.x == 0) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) nanosleep_ns(1000);
  }
  tc_fence_before();
  __syncthreads();
  cluster_meet();  // neither CTA leaves while the other may still signal it
  tc_fence_after();
  if (warp == 1) tmem_dealloc_cg<2>(sc.tmem_base, 512);
}

// ================================================================================================
// stream_gemm
// ================================================================================================
constexpr int kStreamThreads = 256;
constexpr int kStreamArea = 216 * 1024;  // shared memory of the stages
constexpr int kStreamMaxStages = 12;
// A stage, and a K step of this kernel, is two boxes of kBK columns: 256 adjacent bytes of each row of W at a time (32 x 4096
// x 4096 14.5 to 13.5 us, 16 x 4096 x 11008 24.1 to 22.7; with four 12.9 and 21.9, but 24 x 28672 x 8192 85.7 to 90.4: too
// few stages).
constexpr int kSub = 2;
constexpr int kStreamSmem = 1024 + kStreamArea;

struct StreamParams {
  int M, N;        // tokens, output columns (the rows of W)
  int n_k;         // K steps of kSub * kBK
  int tb;          // columns of a tile: M rounded up to a multiple of 16
  int n_tiles;     // ceil(N / 128)
  int per_cta;     // units (tile, K step) of a CTA, in order
  int stages;
  uint32_t tmem_cols;
  uint32_t accs;   // accumulators of a tile, which take the K steps in turn (the loss's logits: four, see kPartSteps)
  int segment;     // K steps of a tile that go into its accumulators at most (the loss's logits): the sums of more stand in the partials meanwhile
  uint32_t idesc;
  float* partial;  // [2 gridDim.x][tb][128]: the tiles that a CTA begins and ends with, if it has not all of their K steps
  Epilogue e;
  Ctrl* ctrl;
  Ctrl* clear;
  unsigned long long timeout_ns;
  Head h;
  const void* w;   // odd rows: W itself
  long long ldw;
  int w_rows, w_cols;
};

constexpr int kSumPitch = 33;  // a token's row, read by column and by row

struct StreamSmem {
  uint64_t full[kStreamMaxStages], empty[kStreamMaxStages], acc_full[2], acc_empty[2], drain;
  uint32_t tmem_base;
  volatile uint32_t abort;
  alignas(16) float sums[4][16][kSumPitch];  // epilogue warp, token, lane
};
static_assert(kStreamSmem + sizeof(StreamSmem) <= 232448, "shared memory");

// The loss's modes: a warp's 32 columns from j0 on, a lane to each, and the sums v of the n tokens from i0 on.  kStats reduces them
// with two lanes to a token, through `rows` ([16][kSumPitch] floats of the warp's, on a 16-byte boundary).
template <int MODE>
__device__ __forceinline__ void head_tokens(const StreamParams& p, int i0, int n, int j0, const uint32_t (&v)[16], float* rows) {
  const int lane = threadIdx.x % 32, j = j0 + lane;
  if constexpr (MODE == kStats) {
    const int cols = min(32, p.N - j0);
    if (cols <= 0) return;
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 16; ++e) rows[e * kSumPitch + lane] = lane < cols ? __uint_as_float(v[e]) : -INFINITY;
    __syncwarp();
    const int i = lane % 16, c0 = lane / 16 * 16;
    const float* row = rows + i * kSumPitch;
    float f[16], m = -INFINITY, sum = 0.f, s[2] = {};
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      f[c] = row[c0 + c];
      m = fmaxf(m, f[c]);
      if (c0 + c < cols) sum += f[c];
    }
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
    const float ref = exp_ref(-FLT_MAX, m);
#pragma unroll
    for (int c = 0; c < 16; ++c) s[c % 2] += ex2_approx(fmaf(f[c], kLog2e, -ref));
    s[0] += s[1];
    s[0] += __shfl_xor_sync(0xffffffffu, s[0], 16);
    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
    if (lane < n) {  // (n: at most 16)
      const long long to = j0 / 32 * p.h.group_at + (i0 + i) * p.h.row_at;
      p.h.stats[to] = make_float2(ref, s[0]);
      if (p.h.sums) p.h.sums[to] = sum;
      const uint64_t target = (uint64_t)p.h.ids[(i0 + i) * p.h.step] - (uint64_t)(p.h.col0 + j0);
      if (target < (uint64_t)cols) p.h.at[i0 + i] = row[target];
    }
  } else if constexpr (MODE == kSlope) {
    __syncwarp();
    if (lane < n) {  // the tokens' coefficients and targets, 16 bytes and 4 to each
      reinterpret_cast<float4*>(rows)[lane] = p.h.coef[i0 + lane];
      reinterpret_cast<int*>(rows)[64 + lane] = p.h.target[i0 + lane];
    }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float4 c = reinterpret_cast<const float4*>(rows)[e];
      const int target = reinterpret_cast<const int*>(rows)[64 + e];
      float f = fmaf(c.y, ex2_approx(fmaf(__uint_as_float(v[e]), kLog2e, -c.x)), -c.z);
      if (target == p.h.col0 + j) f -= c.w;
      if (e < n && j < p.N) store16(p.e.y, (i0 + e) * p.e.ldy + j, p.e.half, target < 0 ? 0.f : f);
    }
  } else {
    const float unit = *p.h.unit;
    const uint32_t in = __ballot_sync(0xffffffffu, lane < n && p.h.target[i0 + min(lane, n - 1)] >= 0);
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (e < n && j < p.N) store16(p.e.y, (i0 + e) * p.e.ldy + j, p.e.half, in >> e & 1u ? __uint_as_float(v[e]) * unit : 0.f);
  }
}

// ------------------------------------------------------------------------------------------------
// Rows off 16-byte boundaries
// ------------------------------------------------------------------------------------------------
// The sixteen bytes from byte `off` (even, below 16) of two vectors on.
__device__ __forceinline__ uint4 shift8(const uint4& lo, const uint4& hi, uint32_t off) {
  uint32_t w[7] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z};
  uint32_t v[6];
#pragma unroll
  for (int j = 0; j < 5; ++j) v[j] = off & 8 ? w[j + 2] : w[j];
  v[5] = off & 8 ? hi.w : w[5];
#pragma unroll
  for (int j = 0; j < 5; ++j) w[j] = off & 4 ? v[j + 1] : v[j];
  const uint32_t bits = off % 4 * 8;
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits), __funnelshift_r(w[2], w[3], bits),
                    __funnelshift_r(w[3], w[4], bits));
}

// W's rows where no tensor map takes them: warps of stream_gemm's own read a stage's 128 rows of 256 bytes, in aligned vectors that
// hold them, shift those to their place and store them where the copies would.  A thread has vector c of every 32nd row from r on;
// steps and tiles are 128 rows or columns, so that all of a thread's vectors are shifted alike.  48 x 128000 x 4100 in 307 us, 3.4 TB/s,
// where a copy of W on aligned rows and the product of that took 560.  The warps wait for their loads most of the time (DRAM and L1 43 %,
// issue slots 47 % busy), but more in flight (a whole stage, or rows asked into L2 some steps ahead) is slower, and eight warps instead of
// sixteen are.
constexpr int kOddWarps = 16, kOddRows = 2 * kOddWarps, kOddHalf = 64 / kOddRows;  // rows at a time, and a thread's vectors of half a stage
struct OddRows {
  const uint8_t *first, *past;  // the matrix
  long long pitch;              // bytes from row to row
  int rows, cols;
  int r, c;
  uint32_t off;                 // where this thread's vectors begin, behind a 16-byte boundary
};
// An aligned vector that begins before the matrix or ends behind it: the elements inside.
static __device__ __noinline__ uint4 odd_vector(const uint8_t* at, const uint8_t* first, const uint8_t* past) {
  uint32_t e[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    e[j] = at + 2 * j >= first && at + 2 * j < past ? *reinterpret_cast<const uint16_t*>(at + 2 * j) : 0;
  return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
}
// Rows r + 64 half + kOddRows j of the box at (row0, col0).
__device__ __forceinline__ void odd_fetch(const OddRows& w, int row0, int col0, int half, uint4 (&lo)[kOddHalf],
                                          uint4 (&hi)[kOddHalf]) {
  const int row = row0 + w.r + 64 * half, col = col0 + 8 * w.c;
  const uint8_t* at = w.first + row * w.pitch + 2ll * col - w.off;
  if (row0 + 128 < w.rows && col0 + 128 <= w.cols && (row0 > 0 || col0 > 0)) {  // all of them lie in the matrix
#pragma unroll
    for (int j = 0; j < kOddHalf; ++j) {
      lo[j] = __ldg(reinterpret_cast<const uint4*>(at + kOddRows * j * w.pitch));
      hi[j] = make_uint4(0, 0, 0, 0);
      if (w.off) hi[j] = __ldg(reinterpret_cast<const uint4*>(at + kOddRows * j * w.pitch) + 1);
    }
    return;
  }
  const int n = col < w.cols ? min(kOddHalf, (w.rows - row + kOddRows - 1) / kOddRows) : 0;  // (rows: row may be past them)
#pragma unroll
  for (int j = 0; j < kOddHalf; ++j) {
    const uint8_t* from = at + kOddRows * j * w.pitch;
    lo[j] = hi[j] = make_uint4(0, 0, 0, 0);
    if (j < n && from >= w.first && from + 16 <= w.past) lo[j] = __ldg(reinterpret_cast<const uint4*>(from));
    if (j < n && w.off && from + 32 <= w.past) hi[j] = __ldg(reinterpret_cast<const uint4*>(from) + 1);
  }
  if (at < w.first || at + kOddRows * (n - 1) * w.pitch + 32 > w.past) {  // at the matrix's first or last element
#pragma unroll
    for (int j = 0; j < kOddHalf; ++j) {
      const uint8_t* from = at + kOddRows * j * w.pitch;
      if (j < n && (from < w.first || from + 16 > w.past)) lo[j] = odd_vector(from, w.first, w.past);
      if (j < n && w.off && from + 32 > w.past) hi[j] = odd_vector(from + 16, w.first, w.past);
    }
  }
}
// K-major W (the box's rows are W's), or the two 64-column boxes of each 64 rows.
template <bool MN>
__device__ __forceinline__ void odd_store(const OddRows& w, int col0, int half, uint8_t* stage, const uint4 (&lo)[kOddHalf],
                                          const uint4 (&hi)[kOddHalf]) {
  const int n = w.cols - (col0 + 8 * w.c);  // elements of the row from the vector on
  uint8_t* to = stage + w.c / 8 * (MN ? 8192 : kHalf) + half * (MN ? kHalf : 8192) + w.r * 128 + ((w.c % 8) ^ (w.r % 8)) * 16;
#pragma unroll
  for (int j = 0; j < kOddHalf; ++j) {
    uint4 v = shift8(lo[j], hi[j], w.off);
    if (n < 8) {
      uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) e[q] = n > 2 * q + 1 ? e[q] : n > 2 * q ? e[q] & 0xffffu : 0u;
      v = make_uint4(e[0], e[1], e[2], e[3]);
    }
    *reinterpret_cast<uint4*>(to + j * (kOddRows * 128)) = v;
  }
}

// The slopes' product goes through W backwards: what the last one, the loss's, read at its end is still in L2.
template <int MODE>
__device__ __forceinline__ int backwards(int i, int n) { return MODE == kSlope ? n - 1 - i : i; }

__host__ __device__ constexpr int stream_threads(bool odd) { return kStreamThreads + (odd ? kOddWarps * 32 : 0); }

// A sum that is read back after another segment of W has gone through L2, as the last to leave it (logits of 64 x 32000 x 16384 in 177 us, of
// 40 x 32000 x 8192 in 98, as without segments; with plain stores 189 and 102).
__device__ __forceinline__ void store_kept(float* at, float v) {
  asm volatile(
      "{\n\t.reg .b64 p;\n\t"
      "createpolicy.fractional.L2::evict_last.b64 p, 1.0;\n\t"
      "st.global.L2::cache_hint.f32 [%0], %1, p;\n\t}\n" ::"l"(at), "f"(v)
      : "memory");
}

// K steps of a tile that a CTA sums at a time, of those left to it.
template <int MODE>
__device__ __forceinline__ int segment_of(const StreamParams& p, int left) {
  if constexpr (in_parts(MODE)) return min(left, p.segment);
  else return left;
}

// ODD: W's rows are off 16-byte boundaries.
template <bool AMN, int MODE = kLayer, bool ODD = false>
__global__ void __launch_bounds__(stream_threads(ODD), 1)
    stream_gemm(const __grid_constant__ StreamParams p, const __grid_constant__ CUtensorMap mw,
                const __grid_constant__ CUtensorMap mx) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ StreamSmem sc;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t smem_base = (raw + 1023u) & ~1023u;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;  // (uniform, for the compiler)
  const uint32_t x_bytes = (uint32_t)p.tb * kBK * 2, stage_bytes = kSub * (kHalf + x_bytes);
  const uint32_t n_st = (uint32_t)p.stages;
  clear_ctrl(p.clear);
  launch_dependents();
  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < n_st; ++s) {
      mbar_init(&sc.full[s], ODD ? 1 + kOddWarps : 1);
      mbar_init(&sc.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sc.acc_full[b], 1);
      mbar_init(&sc.acc_empty[b], 4);
    }
    mbar_init(&sc.drain, 1);
    sc.abort = 0;
    fence_barrier_init();
    if (!ODD) prefetch_tmap(&mw);
    prefetch_tmap(&mx);
  }
  if (warp == 1) {
    tmem_alloc(&sc.tmem_base, p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if constexpr (MODE != kLayer) wait_previous();

  const long long total = (long long)p.n_tiles * p.n_k;
  const long long u0 = (long long)blockIdx.x * p.per_cta;
  const long long u1 = u0 + p.per_cta < total ? u0 + p.per_cta : total;
  uint32_t fills = 0;
  if (warp == 0) {  // this warp and the next converged, as in pair_gemm
    int tile = (int)(u0 / p.n_k), ks = (int)(u0 % p.n_k);
    uint32_t s = 0, phase = 0;
    for (long long u = u0; u < u1; ++u) {
      if (fills >= n_st && !__all_sync(0xffffffffu, wait_own(&sc.empty[s], phase ^ 1u, p, &sc, SITE_EMPTY))) {
        sc.abort = 1;
        break;
      }
      if (lane == 0) mbar_expect_tx(&sc.full[s], ODD ? kSub * x_bytes : stage_bytes);
      const uint32_t base = smem_base + s * stage_bytes;
      const int wrow = backwards<MODE>(tile, p.n_tiles) * kRows, step = backwards<MODE>(ks, p.n_k);
#pragma unroll
      for (int h = 0; h < kSub; ++h) {
        const int k = (step * kSub + h) * kBK;
        const uint32_t dst = base + h * kHalf;
        if constexpr (ODD) {
        } else if constexpr (AMN) {
          load_one(dst, &mw, wrow, k, &sc.full[s], lane == 0);
          load_one(dst + 8192, &mw, wrow + 64, k, &sc.full[s], lane == 0);
        } else {
          load_one(dst, &mw, k, wrow, &sc.full[s], lane == 0);
        }
      }
#pragma unroll
      for (int h = 0; h < kSub; ++h)
        load_one(base + kSub * kHalf + h * x_bytes, &mx, (step * kSub + h) * kBK, 0, &sc.full[s], lane == 0);
      ++fills;
      if (++s == n_st) {
        s = 0;
        phase ^= 1u;
      }
      if (++ks == p.n_k) {
        ks = 0;
        ++tile;
      }
    }
  } else if (warp == 1) {
    const uint32_t tmem = sc.tmem_base;
    const uint32_t a0 = operand_lo<AMN>(smem_base, 0), b0 = operand_lo<false>(smem_base + kSub * kHalf, 0);
    uint32_t s = 0, phase = 0, seg = 0;
    bool ok = true;
    for (long long u = u0; u < u1 && ok; ++seg) {
      const int left = p.n_k - (int)(u % p.n_k);
      const int n = segment_of<MODE>(p, (int)(u1 - u < left ? u1 - u : left));
      const uint32_t slot = seg % 2;
      if (seg >= 2) ok = __all_sync(0xffffffffu, wait_own(&sc.acc_empty[slot], (seg / 2 - 1) & 1u, p, &sc, SITE_ACC_EMPTY));
      if (!ok) break;
      tc_fence_after();
      for (int ks = 0; ks < n; ++ks) {
        ok = __all_sync(0xffffffffu, wait_own(&sc.full[s], phase, p, &sc, SITE_FULL));
        if (!ok) break;
        tc_fence_after();
        const uint32_t at = s * (stage_bytes / 16);
#pragma unroll
        for (int h = 0; h < kSub; ++h)
          mma_step<false, AMN, false>(in_parts(MODE) ? tmem + (slot * p.accs + ks % p.accs) * p.tb : tmem + slot * p.tb,
                                      a0 + at + h * (kHalf / 16), b0 + at + h * (x_bytes / 16), p.idesc,
                                      (in_parts(MODE) ? ks >= (int)p.accs : ks > 0) || h > 0, lane == 0);
        commit_one(&sc.empty[s], lane == 0);
        if (++s == n_st) {
          s = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      commit_one(&sc.acc_full[slot], lane == 0);
      u += n;
    }
    if (!ok) sc.abort = 1;
  } else if (ODD && warp >= kStreamThreads / 32) {
    static_assert(kSub * kBK == 128 && kRows == 128, "a stage's box");
    const int t = threadIdx.x - kStreamThreads;
    OddRows w;
    w.first = static_cast<const uint8_t*>(p.w);
    w.past = w.first + ((p.w_rows - 1) * p.ldw + p.w_cols) * 2;
    w.pitch = p.ldw * 2;
    w.rows = p.w_rows;
    w.cols = p.w_cols;
    w.r = t / 16;
    w.c = t % 16;
    w.off = (uint32_t)(reinterpret_cast<uintptr_t>(w.first + w.r * w.pitch) % 16);
    int tile = (int)(u0 / p.n_k), ks = (int)(u0 % p.n_k), row0 = 0, col0 = 0;
    auto place = [&]() {
      const int at_tile = backwards<MODE>(tile, p.n_tiles) * kRows, at_step = backwards<MODE>(ks, p.n_k) * kSub * kBK;
      row0 = AMN ? at_step : at_tile;
      col0 = AMN ? at_tile : at_step;
    };
    uint4 lo[2][kOddHalf], hi[2][kOddHalf];  // the two halves of a stage, one in flight while the other is stored
    place();
    if (u0 < u1) odd_fetch(w, row0, col0, 0, lo[0], hi[0]);
    uint32_t s = 0, phase = 0;
    for (long long u = u0; u < u1; ++u) {
      const int col = col0;
      odd_fetch(w, row0, col0, 1, lo[1], hi[1]);
      if (u - u0 >= n_st && !__all_sync(0xffffffffu, wait_own(&sc.empty[s], phase ^ 1u, p, &sc, SITE_EMPTY))) {
        sc.abort = 1;
        break;
      }
      uint8_t* stage = smem_raw + (smem_base - raw) + s * stage_bytes;
      odd_store<AMN>(w, col, 0, stage, lo[0], hi[0]);
      if (++ks == p.n_k) {
        ks = 0;
        ++tile;
      }
      place();
      if (u + 1 < u1) odd_fetch(w, row0, col0, 0, lo[0], hi[0]);
      odd_store<AMN>(w, col, 1, stage, lo[1], hi[1]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sc.full[s]);
      if (++s == n_st) {
        s = 0;
        phase ^= 1u;
      }
    }
  } else if (warp >= 4) {
    const int quarter = warp % 4, row = quarter * 32 + lane;
    uint32_t seg = 0;
    bool ok = true;
    for (long long u = u0; u < u1; ++seg) {
      const int tile = (int)(u / p.n_k), first = (int)(u % p.n_k);
      const int left = (int)(u1 - u < p.n_k - first ? u1 - u : p.n_k - first), n = segment_of<MODE>(p, left);
      // this CTA's K steps of the tile: whether there were some before, whether more come, whether they are all
      const bool more = n < left;
      const int had = in_parts(MODE) ? (int)(u - u0 < first ? u - u0 : first) : 0;
      const uint32_t slot = seg % 2;
      ok = __all_sync(0xffffffffu, wait_own(&sc.acc_full[slot], (seg / 2) & 1u, p, &sc, SITE_ACC));
      if (!ok) break;
      tc_fence_after();
      const int first_row = backwards<MODE>(tile, p.n_tiles) * kRows, j = first_row + row;
      const bool whole = had + left == p.n_k;
      const float bias = whole && p.e.bias && j < p.N ? load16(p.e.bias, j, p.e.half) : 0.f;
      // (the second is free until the last tile: a whole one's sums may stand there)
      float* part = p.partial + (2ll * blockIdx.x + (u - had == u0 && !whole ? 0 : 1)) * p.tb * kRows + row;
      const uint32_t tacc = sc.tmem_base + ((uint32_t)(quarter * 32) << 16) + slot * p.tb * (in_parts(MODE) ? p.accs : 1);
#pragma unroll 1
      for (int c = 0; c < p.M; c += 16) {
        uint32_t v[16];
        __syncwarp();  // the load is the whole warp's: no lane is still in the last tokens' epilogue
        tmem_ld16(tacc + c, v);
        tmem_ld_wait();
        if constexpr (in_parts(MODE)) {
          for (uint32_t a = 1; a < p.accs && (int)a < n; ++a) {
            uint32_t w[16];
            tmem_ld16(tacc + a * p.tb + c, w);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) + __uint_as_float(w[e]));
          }
        }
        const int n_c = min(16, p.M - c);
        if constexpr (in_parts(MODE)) {
          if (had) {  // what this thread has stored there
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (e < n_c) v[e] = __float_as_uint(part[(c + e) * kRows] + __uint_as_float(v[e]));
          }
          if (more) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (e < n_c) store_kept(&part[(c + e) * kRows], __uint_as_float(v[e]));
            continue;
          }
        }
        if (!whole) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (e < n_c) part[(c + e) * kRows] = __uint_as_float(v[e]);
          continue;
        }
        if constexpr (MODE != kLayer) {
          head_tokens<MODE>(p, c, n_c, first_row + quarter * 32, v, &sc.sums[quarter][0][0]);
          continue;
        }
        // four tokens at a time, their residuals in flight together; each lane reads its own sums back
        float* own = &sc.sums[quarter][0][lane];
#pragma unroll
        for (int e = 0; e < 16; ++e) own[e * kSumPitch] = __uint_as_float(v[e]);
        if (j < p.N) {
#pragma unroll 1
          for (int e = 0; e < n_c; e += 4) {
            float f[4], r[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const long long i = c + e + q;
              f[q] = own[(e + q) * kSumPitch] + bias;
              r[q] = p.e.res && e + q < n_c ? load16(p.e.res, i * p.e.ldr + j, p.e.half) : 0.f;
            }
            float4 y = make_float4(f[0], f[1], f[2], f[3]);
            if (p.e.act) y = act_call4(p.e.act, y);
            const float g[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              if (e + q >= n_c) break;
              const long long i = c + e + q;
              if (p.e.z) store16(p.e.z, i * p.e.ldz + j, p.e.half, f[q]);
              store16(p.e.y, i * p.e.ldy + j, p.e.half, g[q] + r[q]);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sc.acc_empty[slot]);
      u += n;
    }
    if (!ok) sc.abort = 1;
  }
  // every MMA has completed and every load has landed before the CTA leaves
  if (warp == 1 && lane == 0) {
    mma_commit(&sc.drain);
    wait_last(&sc.drain, 0);
  }
  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < n_st && s < fills; ++s) {
      const uint32_t m = s + ((fills - 1 - s) / n_st) * n_st;
      wait_last(&sc.full[s], (m / n_st) & 1u);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(sc.tmem_base, p.tmem_cols);
}

// Joins the partials of the tiles whose K range is split, in the order of the CTAs that hold them: a thread for each
// output column, a block for each token of a tile.
template <int MODE = kLayer>
__global__ void __launch_bounds__(128) stream_join(const __grid_constant__ StreamParams p) {
  const int tile = blockIdx.x;
  const long long b = (long long)tile * p.n_k, e = b + p.n_k;
  const int c0 = (int)(b / p.per_cta), c1 = (int)((e - 1) / p.per_cta);
  const int j = tile * kRows + threadIdx.x, i = blockIdx.y;
  wait_previous();  // before any exit: what follows on the stream may rely on the products' kernel too
  if (c0 == c1) return;
  float sum = 0.f;
#pragma unroll 4
  for (int g = c0; g <= c1; ++g) {
    const int slot = 2 * g + ((long long)g * p.per_cta >= b ? 0 : 1);  // the tile that CTA g begins or ends with
    sum += p.partial[((long long)slot * p.tb + i) * kRows + threadIdx.x];
  }
  if (j < p.N) finish(p.e, i, j, sum);
}

constexpr int kJoinTokens = 4;  // of a block of head_join that has nothing to reduce
// The same for the loss's modes: a block for sixteen or four tokens of the tile in which CTA blockIdx.x of the product began, if it is the first
// to begin inside of it.  (A block for each token of every tile took 20 us at 48 tokens and 1000 tiles, of which 150 are split.)
template <int MODE>
__global__ void __launch_bounds__(128) head_join(const __grid_constant__ StreamParams p) {
  __shared__ __align__(16) float rows[4][16][kSumPitch];
  const long long u = (long long)blockIdx.x * p.per_cta;
  const int tile = (int)(u / p.n_k), warp = threadIdx.x / 32;
  constexpr int kTokens = MODE == kStats ? 16 : kJoinTokens;
  const int i0 = blockIdx.y * kTokens, n = min(kTokens, p.M - i0);
  wait_previous();
  if (u % p.n_k == 0 || u - p.per_cta > (long long)tile * p.n_k) return;
  const long long b = (long long)tile * p.n_k;
  const int c0 = (int)(b / p.per_cta), c1 = (int)((b + p.n_k - 1) / p.per_cta);
  constexpr int kAhead = MODE == kStats ? 2 : 4;  // parts in flight
  float sum[16] = {};
#pragma unroll kAhead
  for (int g = c0; g <= c1; ++g) {
    const int slot = 2 * g + ((long long)g * p.per_cta >= b ? 0 : 1);
    const float* part = p.partial + ((long long)slot * p.tb + i0) * kRows + threadIdx.x;
#pragma unroll
    for (int e = 0; e < kTokens; ++e) sum[e] += e < n ? part[e * kRows] : 0.f;
  }
  uint32_t v[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(sum[e]);
  head_tokens<MODE>(p, i0, n, backwards<MODE>(tile, p.n_tiles) * kRows + warp * 32, v, &rows[warp][0][0]);
}

// Four columns of dx from the parts of a split tile: the sums of earlier pieces, these, and the row's place in dx.
__device__ __forceinline__ void sum_parts(const PairParams& p, const float* part, int splits, long long i, int j) {
  const Epilogue& e = p.e;
  float f[4] = {};
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const float4 v = *reinterpret_cast<const float4*>(part + s * 65536ll);
    f[0] += v.x; f[1] += v.y; f[2] += v.z; f[3] += v.w;
  }
  float* acc = p.h.acc + i * p.h.ldacc + j;
  if (!p.h.first) {
    const float4 a = *reinterpret_cast<const float4*>(acc);
    f[0] += a.x; f[1] += a.y; f[2] += a.z; f[3] += a.w;
  }
  if (!p.h.last) {
    *reinterpret_cast<float4*>(acc) = make_float4(f[0], f[1], f[2], f[3]);
    return;
  }
  const float unit = *p.h.unit;
  const long long to = p.h.index[i] * e.ldy + j;
  if (e.vec) {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(e.y) + to) =
        make_uint2(pack16(f[0] * unit, f[1] * unit, e.half), pack16(f[2] * unit, f[3] * unit, e.half));
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (j + c < p.N) store16(e.y, to + c, e.half, f[c] * unit);
  }
}

// Joins the parts of the split tiles in order: four columns to a thread, 64 blocks to a tile.
template <int MODE = kLayer>
__global__ void __launch_bounds__(256) pair_join(const __grid_constant__ PairParams p) {
  const int at = blockIdx.x * 256 + threadIdx.x, row = at / 64, col = at % 64 * 4;
  int tm, tn;
  if constexpr (MODE == kSum) {  // as many tiles as the device made of the rows that count
    wait_previous();
    const Extent x = extent_of<MODE>(p, p.n_pairs);
    if (x.splits == 1) return;
    for (int t = blockIdx.y; x.whole + t < x.tiles_m * x.tiles_n; t += gridDim.y) {
      pair_tile(p, x, x.whole + t, tm, tn);
      const long long i = tm * 256ll + row;
      const int j = tn * 256 + col;
      if (i < x.M && j < p.N) sum_parts(p, p.partial + (long long)t * x.splits * 65536 + row * 256 + col, x.splits, i, j);
    }
    return;
  }
  pair_tile(p, p, p.whole + blockIdx.y, tm, tn);
  const long long i = tm * 256ll + row;
  const int j = tn * 256 + col;
  wait_previous();
  if (i >= p.M || j >= p.N) return;
  const float* part = p.partial + (long long)blockIdx.y * p.splits * 65536 + row * 256 + col;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s) {
    const float4 v = *reinterpret_cast<const float4*>(part + s * 65536ll);
    sum.x += v.x; sum.y += v.y; sum.z += v.z; sum.w += v.w;
  }
  const Epilogue& e = p.e;
  float f[4] = {sum.x, sum.y, sum.z, sum.w};
  if (!e.vec) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (j + c < p.N) finish(e, i, j + c, f[c]);
    return;
  }
  auto add = [&](const void* base, long long at) {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + at);
    float lo, hi;
    unpack16(w.x, e.half, lo, hi);
    f[0] += lo; f[1] += hi;
    unpack16(w.y, e.half, lo, hi);
    f[2] += lo; f[3] += hi;
  };
  auto put = [&](void* base, long long at) {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + at) = make_uint2(pack16(f[0], f[1], e.half), pack16(f[2], f[3], e.half));
  };
  if (e.bias) add(e.bias, j);
  if (e.z) put(e.z, i * e.ldz + j);
#pragma unroll
  for (int c = 0; c < 4; ++c) f[c] = act_fwd(e.act, f[c]);
  if (e.res) add(e.res, i * e.ldr + j);
  put(e.y, i * e.ldy + j);
}

// ================================================================================================
// Host side
// ================================================================================================
constexpr int kStreamCtas = 152;  // most CTAs of stream_gemm (one per SM); bounds the partials

// A 16-bit matrix of `outer` rows of `inner` elements, boxes of 64 x box_outer, 128-byte swizzle.  The element type
// only names the width: the copies do no arithmetic and the fill is zero.
inline bool tmap16(CUtensorMap* m, const void* base, int inner, int outer, long long ld, int box_outer) {
  const auto encode = gemm::encode_tiled_fn();
  if (!encode) return false;
  if (outer == 1) ld = (inner + 7ll) / 8 * 8;
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
  cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)box_outer};
  cuuint32_t es[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same for stores of 32 x 32, 64-byte swizzle.
inline bool tmap16_out(CUtensorMap* m, void* base, int inner, int outer, long long ld) {
  const auto encode = gemm::encode_tiled_fn();
  if (!encode) return false;
  if (outer == 1) ld = (inner + 7ll) / 8 * 8;
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
  cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  cuuint32_t box[2] = {32, 32};
  cuuint32_t es[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The matrix's rows all start on 16-byte boundaries (what a tensor map needs).
inline bool mappable(const void* base, int rows, long long ld) {
  return aligned_to(base, 16) && (rows <= 1 || (ld % 8 == 0 && ld * 2 < (1ll << 40)));
}

// Shared memory and co-resident pairs of one pair_gemm instantiation on the current device; 0 on error.
template <bool AMN, bool BMN, bool HALF, int MODE = kLayer>
inline int pairs_of(int dev, int n_sm) {
  static std::mutex mu;
  static int known[64] = {};
  std::lock_guard<std::mutex> lk(mu);
  if (dev >= 0 && dev < 64 && known[dev]) return known[dev];
  auto kern = pair_gemm<AMN, BMN, HALF, MODE>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(n_sm / 2 * 2));
  cfg.blockDim = dim3(pair_threads(MODE));
  cfg.dynamicSmemBytes = kPairSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (n > n_sm / 2) n = n_sm / 2;
  if (dev >= 0 && dev < 64) known[dev] = n;
  return n;
}

// Where a call's kernels run and what they share.
struct Launch {
  int dev, n_sm;
  Ctrl* ctrl;
  Ctrl* clear;     // the control block until a kernel has cleared it, then null
  float* partial;  // fp32 sums of split products
  size_t partial_bytes;
  unsigned long long timeout_ns;
  cudaStream_t st;
};

struct Operands {
  const void* a;
  long long lda;
  const void* b;
  long long ldb;
  int M, N, K;  // C is [M][N]
};

// 256-column tiles that are computed whole, and parts of each of the others along K.
struct Split {
  long long whole, rest;
  int parts;
  double clocks;  // that the parts' way through memory and the join take
};

// The tiles that would leave pairs without one in the last round are split along K, into as many parts as still fit at once, of at
// least 8 K steps, where that saves more clocks than it costs: 8.6 for each K that a pair is spared against 5500 and 180 for
// each part (256 KiB written and read), as measured (768 x 8192 x 4096, 96 tiles: 45 to 40 us; 2048 x 2560 x 4096, 80 tiles: 44 to 36;
// 2600 x 2304 x 2600, 99 tiles, would go from 34 to 38).
inline Split split_of(int M, int N, int K) {
  const long long tiles = ((M + 255ll) / 256) * ((N + 255ll) / 256), rest = tiles % kPairs;
  if (rest == 0) return {tiles, 0, 1, 0.0};
  long long parts = kPairs / rest;
  const long long most = ((K + kBK - 1) / kBK) / 8;
  if (parts > most) parts = most;
  const double clocks = 5500.0 + 180.0 * rest * parts * (M < 256 ? M : 256) / 256.0;
  if (parts < 2 || 8.6 * K * (1.0 - 1.0 / parts) < clocks) return {tiles, 0, 1, 0.0};
  return {tiles - rest, rest, (int)parts, clocks};
}

// Whether a product takes tiles of 512 columns.  Tiles of 256 columns take 9 clocks for each K and tile (a little more with an operand
// that is MN-major), or as long as the epilogue, which runs beside the next tile's products, if that is longer.  Tiles of 512
// columns take 16 and move less, but their epilogue has the accumulators to itself: nothing runs beside it.  Rows that do not start on
// 128-byte boundaries take the loads half as long again.  `more`: the epilogue's clocks beyond a plain store.  Clocks as measured at
// 16384 x 4096 x 512 (one / two: 48 / 71 us, with gelu, bias, residual and z 112 / 132), 4096 x 4096 x 4096 (78 / 87, 87 / 107),
// 1531 x 5000 x 1736 (31 / 28) and, under lasting load, where the power limit counts what is moved, 8192 x 8192 x 8192 (668 /
// 639, its dx 672 / 639) and 4100 x 8192 x 4096 (174 / 181).
template <bool AMN, bool BMN>
inline bool wide_tiles(const Operands& o, double more, const Split& split, long long n_pairs) {
  const long long rows = (o.M + 255ll) / 256;
  const bool ragged = o.lda % 64 || o.ldb % 64;
  const double k1 = ragged ? 12.8 : 9.0 + 0.3 * (AMN + BMN), k2 = ragged ? 18.4 : 16.0;
  const long long ones = rows * ((o.N + 255) / 256), tiles = rows * ((o.N + 511) / 512), halves = last_halves(tiles, (int)n_pairs);
  const double round = std::max(k1 * o.K, 5500.0 + more);  // of 256-column tiles
  const double one = split.rest ? split.whole / n_pairs * round + k1 * o.K / split.parts + split.clocks + more / 2
                                : (double)((ones + n_pairs - 1) / n_pairs) * round;
  const double two = (double)(tiles / n_pairs + (halves || tiles % n_pairs == 0 ? 0 : 1)) * (k2 * o.K + 2 * (4800.0 + more)) +
                     (halves ? k1 * o.K + 4800.0 + more : 0.0);
  return two <= one;
}

template <bool AMN, bool BMN, bool HALF, int MODE = kLayer>
inline int launch_pair(const Operands& o, const Epilogue& e, bool wide, const Split& split, Launch& l, const Head& head = {}) {
  const int n_pairs = pairs_of<AMN, BMN, HALF, MODE>(l.dev, l.n_sm), cols = wide ? 512 : 256;
  if (n_pairs < 1) return PSR_ERR_CUDA;
  PairParams p = {};
  p.h = head;
  p.n_pairs = n_pairs;
  p.M = o.M;
  p.N = o.N;
  p.n_k = (o.K + kBK - 1) / kBK;
  p.tiles_m = (o.M + 255) / 256;
  p.wide = wide;
  p.tiles_n = (o.N + cols - 1) / cols;
  long long items = (long long)p.tiles_m * p.tiles_n;
  if (items >= (1ll << 30)) return PSR_ERR_UNSUPPORTED;
  p.group = 16;  // (8192 x 28672 x 4096 in 967 us; 8, 12, 24, 32 rows: 987, 976, 984, 1010)
  p.whole = (int)items;
  p.splits = 1;
  p.partial = l.partial;  // (dx: for kPairs parts, whatever the device makes of its tiles)
  if (MODE == kSum && (size_t)kPairs * 65536 * 4 > l.partial_bytes) return PSR_ERR_ARG;
  if (!wide && split.rest > 0) {
    p.whole = (int)split.whole;
    p.split_k = (p.n_k + split.parts - 1) / split.parts;
    p.splits = (p.n_k + p.split_k - 1) / p.split_k;  // none of them empty
    if ((size_t)split.rest * p.splits * 65536 * 4 > l.partial_bytes) return PSR_ERR_ARG;
    items = split.whole + split.rest * p.splits;
  }
  p.idesc = idesc16(256, 256, AMN, BMN, e.half != 0);
  p.e = e;
  p.ctrl = l.ctrl;
  p.clear = l.clear;
  p.timeout_ns = l.timeout_ns;
  CUtensorMap ma, mb;
  const bool ok_a = AMN ? tmap16(&ma, o.a, o.M, o.K, o.lda, 64) : tmap16(&ma, o.a, o.K, o.M, o.lda, kRows);
  const bool ok_b = BMN ? tmap16(&mb, o.b, o.N, o.K, o.ldb, 64) : tmap16(&mb, o.b, o.K, o.N, o.ldb, kRows);
  if (!ok_a || !ok_b) return PSR_ERR_CUDA;
  Out<MODE> out = {};
  if constexpr (MODE == kWeight) {
    out.copies = e.vec && p.n_k <= kCopySteps;
    if (out.copies && !tmap16_out(&out.map, e.y, o.N, o.M, e.ldy)) return PSR_ERR_CUDA;
  }
  if (wide) {
    p.halves = last_halves(items, n_pairs);
    items += p.halves;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * (items < n_pairs && !(MODE == kSum && head.rows) ? items : n_pairs)));
  cfg.blockDim = dim3(pair_threads(MODE));
  cfg.dynamicSmemBytes = kPairSmem;
  cfg.stream = l.st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = MODE == kLayer ? 1 : 2;
  if (cudaLaunchKernelEx(&cfg, pair_gemm<AMN, BMN, HALF, MODE>, p, ma, mb, out) != cudaSuccess) {
    cudaGetLastError();
    return PSR_ERR_CUDA;
  }
  l.clear = nullptr;
  if (MODE == kSum) return launch_after(pair_join<MODE>, dim3(64, 8), 256, p, l.st);
  if (p.splits == 1) return PSR_OK;
  return launch_after(pair_join<MODE>, dim3(64, (unsigned)split.rest), 256, p, l.st);
}

// Whether stream_gemm takes a product with M rows of A: up to 64, and up to 128 where neither a single step, which leaves the whole
// epilogue to one CTA, nor many columns, whose tokens' epilogue adds up, make the tiles of 256 rows faster (streaming / tiles: 128 x
// 1024 x 1024 8.0 / 12.0 us, 128 x 4096 x 4096 17.7 / 18.5, 72 x 4096 x 8192 19.1 / 22.9; 128 x 1024 x 64 14.9 / 8.1, 128 x 8192 x
// 1024 15.5 / 13.8, 128 x 28672 x 4096 81 / 54).
inline bool streams(int M, int N, int K) { return M <= 64 || (M <= 128 && K >= 512 && N <= 4096); }

// Bytes of fp32 partials that a product with C [M][N] may leave (weights: A's rows are not tokens, so it never streams).
inline size_t partial_bytes(int M, int N, int K, bool weights) {
  if (!weights && streams(M, N, K)) return (size_t)2 * kStreamCtas * ((M + 15) / 16 * 16) * kRows * 4;
  const Split s = split_of(M, N, K);
  return (size_t)s.rest * s.parts * 65536 * 4;
}

// o.a: the tokens [M][K], o.b: W, K-major [N][K] or (WMN) [K][N].
template <bool WMN, int MODE = kLayer, bool ODD = false>
inline int launch_stream(const Operands& o, const Epilogue& e, Launch& l, const Head& head = {}) {
  const int dev = l.dev, n_sm = l.n_sm;
  static std::mutex mu;
  static bool known[64] = {};
  {
    std::lock_guard<std::mutex> lk(mu);
    if (dev < 0 || dev >= 64 || !known[dev]) {
      if (cudaFuncSetAttribute(stream_gemm<WMN, MODE, ODD>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamSmem) != cudaSuccess) {
        cudaGetLastError();
        return PSR_ERR_CUDA;
      }
      if (dev >= 0 && dev < 64) known[dev] = true;
    }
  }
  StreamParams p = {};
  p.h = head;
  p.M = o.M;
  p.N = o.N;
  p.n_k = (o.K + kSub * kBK - 1) / (kSub * kBK);
  p.tb = (o.M + 15) / 16 * 16;
  p.n_tiles = (o.N + kRows - 1) / kRows;
  const int most = n_sm < kStreamCtas ? n_sm : kStreamCtas;
  const long long units = (long long)p.n_tiles * p.n_k;
  long long per = (units + most - 1) / most;
  // Short rows of many tiles stay whole, with nothing to join (64 x 16384 x 1024: 15.3 us, split 17.5).  Otherwise a tile is split
  // into up to eight parts where SMs would be idle, and more if the parts are of four steps: few tiles finish sooner through the
  // join, which has a thread for each output (64 x 1024 x 1024: 6.2 us, whole 11.4; 32 x 1024 x 4096: 7.0, with parts of a step 9.1).
  if (p.n_k <= 8 && 2 * p.n_tiles >= most) per = (per + p.n_k - 1) / p.n_k * p.n_k;
  else per = std::max(per, (long long)std::max(1, std::min(4, p.n_k / 8)));
  if (per >= (1ll << 31)) return PSR_ERR_UNSUPPORTED;
  p.per_cta = (int)per;
  const int stage = kSub * (kHalf + p.tb * kBK * 2);
  p.stages = kStreamArea / stage < kStreamMaxStages ? kStreamArea / stage : kStreamMaxStages;
  p.accs = in_parts(MODE) ? 4 : 1;  // (of at most 64 columns)
  p.segment = (int)p.accs * kPartSteps / kSub;
  p.tmem_cols = 32;
  while (p.tmem_cols < 2u * p.tb * p.accs) p.tmem_cols *= 2;
  p.idesc = idesc16(128, p.tb, WMN, false, e.half != 0);
  p.partial = l.partial;
  p.e = e;
  p.ctrl = l.ctrl;
  p.clear = l.clear;
  p.timeout_ns = l.timeout_ns;
  p.w = o.b;
  p.ldw = o.ldb;
  p.w_rows = WMN ? o.K : o.N;
  p.w_cols = WMN ? o.N : o.K;
  CUtensorMap mw = {}, mx;
  const bool ok_w = ODD ? true : WMN ? tmap16(&mw, o.b, o.N, o.K, o.ldb, 64) : tmap16(&mw, o.b, o.K, o.N, o.ldb, kRows);
  if (!ok_w || !tmap16(&mx, o.a, o.K, o.M, o.lda, p.tb)) return PSR_ERR_CUDA;
  const unsigned grid = (unsigned)((units + per - 1) / per);
  if constexpr (MODE == kLayer) {
    stream_gemm<WMN, MODE, ODD><<<grid, kStreamThreads, kStreamSmem, l.st>>>(p, mw, mx);
    const int rc = launch_status();
    l.clear = nullptr;
    if (rc != PSR_OK || per % p.n_k == 0) return rc;
    return launch_after(stream_join<MODE>, dim3((unsigned)p.n_tiles, (unsigned)o.M), 128, p, l.st);
  } else {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(stream_threads(ODD));
    cfg.dynamicSmemBytes = kStreamSmem;
    cfg.stream = l.st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = l.clear ? 0 : 1;  // (the call's first kernel clears the control block)
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, stream_gemm<WMN, MODE, ODD>, p, mw, mx) != cudaSuccess) {
      cudaGetLastError();
      return PSR_ERR_CUDA;
    }
    l.clear = nullptr;
    if (per % p.n_k == 0) return PSR_OK;
    constexpr int tokens = MODE == kStats ? 16 : kJoinTokens;
    return launch_after(head_join<MODE>, dim3(grid, (unsigned)((o.M + tokens - 1) / tokens)), 128, p, l.st);
  }
}

// ------------------------------------------------------------------------------------------------
// An operand with rows of any stride, from any address, into rows on 16-byte boundaries
// ------------------------------------------------------------------------------------------------
// Eight elements from any (even) address, `n` of them in the row; zeros for the others.  Two aligned vectors that hold them all are
// shifted to their place where those lie in the matrix, which has its bytes from `first` to `past`; at its two ends, and at the end of a
// row, the elements are read one by one.
__device__ __forceinline__ uint4 load8(const uint16_t* p, int n, const uint8_t* first, const uint8_t* past) {
  const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) % 16);
  const uint8_t* base = reinterpret_cast<const uint8_t*>(p) - off;
  if (n >= 8 && base >= first && base + 32 <= past) {
    const uint4 lo = *reinterpret_cast<const uint4*>(base);
    uint4 hi = make_uint4(0, 0, 0, 0);
    if (off) hi = *reinterpret_cast<const uint4*>(base + 16);
    return shift8(lo, hi, off);
  }
  uint32_t e[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) e[j] = j < n ? p[j] : 0;
  return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
}

// Memory bound.
template <class T>
__global__ void __launch_bounds__(256)
    align_kernel(const T* __restrict__ x, long long ld, uint4* __restrict__ y, int rows, int cols, Ctrl* clear) {
  clear_ctrl(clear);
  constexpr int kAhead = 4;
  const uint32_t per = (cols + 7) / 8;
  const long long n = (long long)rows * per, step = gridDim.x * 256ll;
  const uint8_t* first = reinterpret_cast<const uint8_t*>(x);
  const uint8_t* past = reinterpret_cast<const uint8_t*>(x + (rows - 1ll) * ld + cols);
  for (long long i0 = blockIdx.x * 256ll + threadIdx.x; i0 < n; i0 += kAhead * step) {
    uint4 v[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const long long i = i0 + a * step;
      if (i >= n) break;
      const long long r = n < 1ll << 32 ? (uint32_t)i / per : i / per;
      const int c = (int)(i - r * per) * 8;
      v[a] = load8(x + r * ld + c, cols - c, first, past);
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (i0 + a * step < n) y[i0 + a * step] = v[a];
  }
}

// The operand's aligned copy, if it needs one: x and ld then name that.
inline int align(const void*& x, long long& ld, size_t at, int rows, int cols, void* workspace, Launch& l) {
  if (!at || rows == 0) return PSR_OK;
  uint4* y = reinterpret_cast<uint4*>(static_cast<uint8_t*>(workspace) + at);
  const long long blocks = ((long long)rows * ((cols + 7) / 8) + 255) / 256;
  align_kernel<uint16_t><<<(unsigned)(blocks < l.n_sm * 16 ? blocks : l.n_sm * 16), 256, 0, l.st>>>(static_cast<const uint16_t*>(x), ld, y,
                                                                                        rows, cols, l.clear);
  l.clear = nullptr;
  x = y;
  ld = (cols + 7ll) / 8 * 8;
  return launch_status();
}

}  // namespace linear
}  // namespace psr
