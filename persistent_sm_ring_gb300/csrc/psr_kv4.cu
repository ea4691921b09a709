// KV cache in 4 bits on sm_103a: quantise and append, read back, and the attention of new tokens over the pages.
//
// The cache is laid out in blocks of 16 tokens of one KV head: K codes, V codes, then the (scale, offset) pairs,
// 16 (d + 8) bytes in one piece, so that whatever the page size a block is one contiguous 16-byte aligned copy.
// One scale and offset for a row (not for groups of columns) keeps them out of the products: with c the codes,
//     q . k = scale (q . c) + offset sum(q),        sum_j p_j v_j = sum_j (p_j scale_j) c_j + sum_j p_j offset_j.
#include <cmath>
#include <mutex>
#include <type_traits>

#include "psr_device.cuh"
#include "psr_host.h"

namespace psr {
namespace kv4 {

constexpr int kBlk = 16;  // tokens of a block

struct Cache {
  uint8_t* base;
  const int32_t* table;
  int Hkv, d, page, n_pages, max_pages;
  int shift;  // page = 1 << shift
};

// The block that holds position pos of sequence b for KV head h, or null if the table has no usable page there.
template <int D>
__device__ __forceinline__ uint8_t* block_of(const Cache& c, int b, int h, long long pos) {
  if (pos < 0 || pos >> c.shift >= c.max_pages) return nullptr;
  const int pg = c.table[(long long)b * c.max_pages + (int)(pos >> c.shift)];
  if ((uint32_t)pg >= (uint32_t)c.n_pages) return nullptr;
  const int per = c.page / kBlk;
  return c.base + (((long long)pg * c.Hkv + h) * per + (int)(pos & (c.page - 1)) / kBlk) * (kBlk * (D + 8));
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// ------------------------------------------------------------------------------------------------
// Append and read
// ------------------------------------------------------------------------------------------------
// D / 8 lanes take a row, eight columns (16 bytes) each; a block takes kTokens tokens of one sequence and KV head, and a lane
// the K and V rows of two of them, so that four loads are in flight.  Bound by their instructions: 4 x 2000 tokens of 8 heads,
// d = 128, are appended in 16.8 us (70 % of the issue slots, 200 instructions for a lane's part of a row) and read in 9.8, where
// the bytes would take 6 each.
constexpr int kEach = 2;  // tokens of a thread
constexpr int kMove = 128;  // threads of a block

template <int D>
struct Rows {
  static constexpr int kLanes = D / 8;           // of a row
  static constexpr int kTokens = kEach * kMove / kLanes;  // of a block
};

struct MoveParams {
  Cache c;
  const void* in[2];  // append
  void* out[2];       // read
  psr_strides st[2];  // of `in`
  const int32_t *start, *count;
  int S, tiles;       // rows, blocks of a sequence and head
  int vec;            // `in`'s rows are 16-byte aligned
};

template <class T>
struct alignas(16) Eight {
  T e[8];
};
template <class T>
struct Pair {
  using type = __nv_bfloat162;
  static __device__ __forceinline__ type zero() { return __float2bfloat162_rn(0.f); }
};
template <>
struct Pair<__half> {
  using type = __half2;
  static __device__ __forceinline__ type zero() { return __float2half2_rn(0.f); }
};

// two fp32 operations at once
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(*reinterpret_cast<unsigned long long*>(&r))
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(*reinterpret_cast<unsigned long long*>(&r))
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return r;
}

// The step of a row, (max - min) / 15 rounded once to bf16.  Correct rounding without a division: the product with 1/15 is at most
// 2.1 units of its last place off (the reciprocal one, the product half of one, the span's own rounding 8/15), so only one that
// near to the middle of two bf16 numbers can round the wrong way.  There the sign of max - min - 15 middle decides: the product is
// exact (9 bits by 4), the difference cancels exactly, and what the span lost is smaller than a unit of it.
template <class T>
__device__ __forceinline__ __nv_bfloat16 step_of(float mn, float mx) {
  float span = __fsub_rn(mx, mn), back = 1.f;
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    if (span == INFINITY) {  // the span passes the largest fp32 number, which its fifteenth does not
      mx *= 0.0625f;
      mn *= 0.0625f;
      span = __fsub_rn(mx, mn);
      back = 16.f;
    }
  }
  uint32_t q = __float_as_uint(__fmul_rn(span, 1.f / 15.f));
  if (((q + 0x8004u) & 0xFFFFu) <= 8u) {
    q = (q & 0xFFFF0000u) | 0x8000u;
    const float part = __fsub_rn(mx, span);  // what of the span's rounding mx and mn have each
    const float lost = __fsub_rn(__fsub_rn(mx, __fadd_rn(span, part)), __fsub_rn(mn, part));
    const float rest = __fadd_rn(__fmaf_rn(-15.f, __uint_as_float(q), span), lost);
    if (rest != 0.f) q += rest > 0.f ? 1 : -1;
  }
  return __float2bfloat16_rn(__uint_as_float(q) * back);
}

template <class T, int D>
__global__ void __launch_bounds__(kMove) append_kernel(const __grid_constant__ MoveParams p) {
  using R = Rows<D>;
  const int bh = blockIdx.x / p.tiles, b = bh / p.c.Hkv, h = bh - b * p.c.Hkv;
  const int part = threadIdx.x % R::kLanes;
  const int first = (blockIdx.x - bh * p.tiles) * R::kTokens + threadIdx.x / R::kLanes;
  const int end = p.count ? min(p.S, p.count[b]) : p.S;
  const long long start = p.start[b];
  Eight<T> raw[kEach][2];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const T* x = static_cast<const T*>(p.in[kv]) + (b * p.st[kv].b + h * p.st[kv].h) + first * p.st[kv].s + part * 8;
#pragma unroll
    for (int n = 0; n < kEach; ++n) {
      if (first + n * (R::kTokens / kEach) >= end) continue;
      const T* y = x + n * (R::kTokens / kEach) * p.st[kv].s;
      if (p.vec) raw[n][kv] = *reinterpret_cast<const Eight<T>*>(y);
      else
#pragma unroll
        for (int e = 0; e < 8; ++e) raw[n][kv].e[e] = y[e];
    }
  }
  uint8_t* blk[kEach];  // looked up while the rows are on their way
#pragma unroll
  for (int n = 0; n < kEach; ++n) {
    const int i = first + n * (R::kTokens / kEach);
    blk[n] = i < end ? block_of<D>(p.c, b, h, start + i) : nullptr;
  }
  // minimum and negated maximum of each row side by side, NaN if there is one; a missing row is all zeros
  using T2 = typename Pair<T>::type;
  T2 low[kEach][2];
#pragma unroll
  for (int n = 0; n < kEach; ++n)
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      T2 w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = blk[n] ? reinterpret_cast<const T2*>(&raw[n][kv])[e] : Pair<T>::zero();
      const T2 a = __hmin2_nan(__hmin2_nan(w[0], w[1]), __hmin2_nan(w[2], w[3]));
      const T2 b = __hneg2(__hmax2_nan(__hmax2_nan(w[0], w[1]), __hmax2_nan(w[2], w[3])));
      T2 left, right;
      left.x = a.x; left.y = b.x;
      right.x = a.y; right.y = b.y;
      T2 v = __hmin2_nan(left, right);
#pragma unroll
      for (int o = R::kLanes / 2; o; o >>= 1) v = __hmin2_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
      low[n][kv] = v;
    }
  // The scale and offset of the lanes' 2 kEach rows, each worked out by one lane in four.
  static_assert(kEach == 2 && R::kLanes >= 4, "a row's lanes take its four (token, K or V) in turn");
  uint32_t pair;
  float inv;
  {
    const T2 v = part & 2 ? (part & 1 ? low[1][1] : low[1][0]) : (part & 1 ? low[0][1] : low[0][0]);
    const float mn = to_f32(v.x), mx = -to_f32(v.y);
    __nv_bfloat162 so;
    so.x = step_of<T>(mn, mx);
    so.y = __float2bfloat16_rn(mn);
    if (!(fabsf(mn) < INFINITY && fabsf(mx) < INFINITY)) so.x = so.y = __ushort_as_bfloat16(0x7FFF);
    inv = __fdividef(1.f, __bfloat162float(so.x));
    pair = *reinterpret_cast<uint32_t*>(&so);
  }
#pragma unroll
  for (int n = 0; n < kEach; ++n) {
    const int row = (int)((start + first + n * (R::kTokens / kEach)) & (kBlk - 1));
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint32_t so = __shfl_sync(0xffffffffu, pair, 2 * n + kv, R::kLanes);
      const float by = __shfl_sync(0xffffffffu, inv, 2 * n + kv, R::kLanes);
      if (!blk[n]) continue;
      const float s = __uint_as_float(so << 16), o = __uint_as_float(so & 0xFFFF0000u);
      uint32_t codes = 0;
      if (s > 0.f) {  // (not NaN)
        // The code is the rounded quotient rounded to an integer (adding 1.5 2^23 does that, half to even, and leaves it in the
        // low bits).  A product with the reciprocal is within 2^-21 of a quotient below 16: only one that near to a half needs
        // the division.
        const float magic = 12582912.f;
        float v[8], far = s > 1e-37f && s < 1e37f ? 0.f : 1.f;  // how far from an integer; the reciprocal may have overflowed
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = to_f32(raw[n][kv].e[e]);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          float2 q = mul2(add2(make_float2(v[e], v[e + 1]), make_float2(-o, -o)), make_float2(by, by));
          // a bf16 row's offset is its minimum and 15 rounded steps pass its maximum by less than half of one: nothing to clamp
          if (!std::is_same<T, __nv_bfloat16>::value)
            q = make_float2(fminf(fmaxf(q.x, 0.f), 15.f), fminf(fmaxf(q.y, 0.f), 15.f));
          const float2 r = add2(q, make_float2(magic, magic)), t = add2(r, make_float2(-magic, -magic));
          const float2 d = add2(q, make_float2(-t.x, -t.y));
          far = fmax3(far, fabsf(d.x), fabsf(d.y));
          codes = __funnelshift_r(codes, __float_as_uint(r.x), 4);  // the code enters at the top
          codes = __funnelshift_r(codes, __float_as_uint(r.y), 4);
        }
        if (far > 0.49997f) {
          codes = 0;
          const float f = s < 1e37f ? 1.f : 0.0625f;  // a distance from the offset may pass the largest fp32 number
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float q = fminf(fmaxf(__fdiv_rn(__fsub_rn(v[e] * f, o * f), s * f), 0.f), 15.f);
            codes |= (__float_as_uint(__fadd_rn(q, magic)) & 15u) << (4 * e);
          }
        }
      }
      *reinterpret_cast<uint32_t*>(blk[n] + kv * kBlk * (D / 2) + row * (D / 2) + part * 4) = codes;
      if (part == 0) *reinterpret_cast<uint32_t*>(blk[n] + kBlk * D + kv * kBlk * 4 + row * 4) = so;
    }
  }
}

template <class T, int D>
__global__ void __launch_bounds__(kMove) read_kernel(const __grid_constant__ MoveParams p) {
  using R = Rows<D>;
  const int bh = blockIdx.x / p.tiles, b = bh / p.c.Hkv, h = bh - b * p.c.Hkv;
  const int part = threadIdx.x % R::kLanes;
  const int first = (blockIdx.x - bh * p.tiles) * R::kTokens + threadIdx.x / R::kLanes;
  const int end = p.count ? min(p.S, p.count[b]) : p.S;
  const long long start = p.start[b];
  uint32_t codes[kEach][2] = {};
  float s[kEach][2], o[kEach][2];
#pragma unroll
  for (int n = 0; n < kEach; ++n) {
    const int i = first + n * (R::kTokens / kEach), row = (int)((start + i) & (kBlk - 1));
    const uint8_t* blk = i < end ? block_of<D>(p.c, b, h, start + i) : nullptr;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      s[n][kv] = 0.f;
      o[n][kv] = i < end ? NAN : 0.f;
      if (!blk) continue;
      codes[n][kv] = *reinterpret_cast<const uint32_t*>(blk + kv * kBlk * (D / 2) + row * (D / 2) + part * 4);
      const __nv_bfloat162 pair = *reinterpret_cast<const __nv_bfloat162*>(blk + kBlk * D + kv * kBlk * 4 + row * 4);
      s[n][kv] = __bfloat162float(pair.x);
      o[n][kv] = __bfloat162float(pair.y);
    }
  }
#pragma unroll
  for (int n = 0; n < kEach; ++n) {
    const int i = first + n * (R::kTokens / kEach);
    if (i >= p.S) continue;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      Eight<T> w;
#pragma unroll
      for (int e = 0; e < 8; ++e) w.e[e] = from_f32<T>(fmaf((float)((codes[n][kv] >> (4 * e)) & 15u), s[n][kv], o[n][kv]));
      *reinterpret_cast<Eight<T>*>(static_cast<T*>(p.out[kv]) + ((long long)bh * p.S + i) * D + part * 8) = w;
    }
  }
}

// ------------------------------------------------------------------------------------------------
// Attention
// ------------------------------------------------------------------------------------------------
// Bound by reading the cache once, and by the instructions that it takes: 8 sequences of about 110k positions, 32 query and 8 KV
// heads, d = 128, in 164 us (6.05 TB/s; 79 % of DRAM's peak, 61 % of the integer pipe's, 56 % of the issue slots).  A unit is two
// blocks (32 tokens) of one KV head and a tile of up to 8 NT query rows (the group's heads times the new tokens); the units of
// all sequences stand in a line, segment by segment (a segment: sequence, head, row tile), and each warp takes an equal stretch
// of it, so ragged batches and single long sequences load every SM alike.  A segment that lies within one stretch is finished
// there; the pieces of one that does not meet in combine_kernel through fp32 partial results and their running maxima and sums, as
// the ring's chunks do.  A segment stands in the line behind kPad places without work, so that a stretch of many short ones is
// not the longest (48 ragged sequences with 4 draft tokens, d = 64: 77 us without, 68 with).  Each row tile is a segment of its
// own and reads the cache again: with 16 query rows to a KV head those 8 sequences take 251 us, with 32 and 64 (two and four
// tiles) 451 and 881.
//
// Each warp has its own ring of stages, filled a unit or more ahead with 16-byte asynchronous copies by all of its lanes (one
// lane's bulk copy and a barrier cost a third of a unit's time at d = 64), and its own softmax state.
//   S^T[token][row] = K codes . q      (mma.m16n8k16: tokens on its 16 rows, query rows on its 8 columns)
//   O^T[column][row] += V codes^T . P  (columns of V on the 16 rows, tokens in the contraction)
// The issue slots are what is scarce.  So:
//  * a code needs no conversion: its four bits, masked in place, are a subnormal fp16 number, c 2^-24 in bits 0..3 and
//    16 c 2^-24 in bits 4..7, exact, and the matrix product takes it so.  One shift and four masks give eight codes.
//  * q becomes fp16 for it, each row scaled by a power of two that puts its largest element below 2^15 (exact for bf16
//    down to 2^-25 of that); the scales 2^24, 1/16 and that power go to the sums.
//  * P becomes fp16 times its row's scale, divided by a power of two of its own for each query row, which follows the
//    largest product of a weight and a scale, so that no ratio of the scales of different tokens costs P its digits.  An mma
//    more for 16 tokens multiplies it with a constant code 8: what is wanted is the sum of P (c - 8), as large as the output,
//    and the two sums' roundings go together (the sum of P c alone has those of terms that cancel: 2.1e-3 of the output in a
//    long context, against 1.7e-3).
//  * any order of the contraction will do, so K's fragments are read straight from the stage, 16 adjacent bytes of a row to a
//    lane.  V's come through transposing matrix loads of 16-bit elements (four columns of a token), whose pieces the copies
//    have swizzled over the banks.  P leaves the first product in the layout that movmatrix turns into the second one's operand.
//  * up to four query rows fill half of the eight columns.  SPLIT then gives columns 0..3 the first block of a unit and columns
//    4..7 the second, as rows of their own that meet at the end: a lane has half as many weights to work out (8 sequences of
//    about 110k positions, 4 rows: 174 us without, 166 with).  Both products stay as many.
//  * the maximum and that power are only raised when a weight or a product passes kRaise: the check is one vote.
constexpr int kWarps = 8;
template <int D>
constexpr int kStages = D == 128 ? 2 : 3;
constexpr int kUnit = 2 * kBlk;     // tokens of a unit
constexpr int kPad = 2;             // units that a segment counts for besides its own: loading q and writing results
constexpr int kMaxPlaces = 2130706432;  // 2^31 - 2^24: a place plus a stretch stays an int
constexpr int kMaxCtas = 2 * 152;   // bounds the partial results
template <int D>
constexpr int kPart = D + 4;        // floats of a row's partial result: sums, maximum, weight
constexpr float kRaise = 256.f;
constexpr float kLowest = -1e30f;   // a maximum that nothing has raised
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

struct AttnParams {
  Cache c;
  const void* q;
  void* o;
  float* lse;
  const int32_t* lens;
  psr_strides sq, so;
  int B, Hq, S, group, n_rt;  // group = Hq / Hkv; row tiles of group * S rows
  int page_shift;             // log2(page / 16)
  int vec;                    // q's rows are 16-byte aligned
  float scale;
  int vec_o;                  // o's rows are 16-byte aligned
  float* part;                // [2 kMaxCtas kWarps][rows of a tile][kPart]
  Ctrl* ctrl;
};

// Blocks of sequence b: 0 if it is empty or its length is out of range.  Two make a unit.
__device__ __forceinline__ int blocks_of(const AttnParams& p, int b) {
  const int n = p.lens[b];
  return n < 0 || n > (long long)p.c.max_pages * p.c.page ? 0 : (n + kBlk - 1) / kBlk;
}

// Places that a segment of so many blocks takes in the line.
__device__ __forceinline__ int places(int blocks) { return blocks ? (blocks + 1) / 2 + kPad : 0; }

// A segment of the line (fewer than kMaxPlaces places: checked on the host).
struct Cursor {
  int b, h, rt, blocks;
  int start;  // its first place
  __device__ __forceinline__ int end() const { return start + places(blocks); }
  __device__ __forceinline__ void advance(const AttnParams& p, int u) {
    while (u >= end()) {
      start = end();
      if (++rt == p.n_rt) {
        rt = 0;
        if (++h == p.c.Hkv) {
          h = 0;
          blocks = blocks_of(p, ++b);
        }
      }
    }
  }
};

// One warp: the places of the sequences before `end`.
__device__ __forceinline__ int units_before(const AttnParams& p, int end) {
  const int lane = threadIdx.x % 32;
  int sum = 0;
#pragma unroll 4
  for (int b = lane; b < end; b += 32) sum += places(blocks_of(p, b));
  return __reduce_add_sync(0xffffffffu, sum) * p.c.Hkv * p.n_rt;
}

// One warp: the segment that holds a place (of those there are).  mine: the blocks of sequence `lane`, already at hand.
__device__ __forceinline__ Cursor segment_at(const AttnParams& p, int target, int mine) {
  const int lane = threadIdx.x % 32;
  const int per = p.c.Hkv * p.n_rt;
  Cursor cur = {};
  int base = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int n = b0 == 0 ? mine : b0 + lane < p.B ? blocks_of(p, b0 + lane) : 0;
    const int own = places(n) * per;
    int sum = own;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    const int all = __shfl_sync(0xffffffffu, sum, 31);
    if (target < base + all) {
      const int at = __ffs(__ballot_sync(0xffffffffu, target < base + sum)) - 1;
      const int first = base + __shfl_sync(0xffffffffu, sum - own, at);
      cur.blocks = __shfl_sync(0xffffffffu, n, at);
      const int len = places(cur.blocks), seg = (target - first) / len;
      cur.b = b0 + at;
      cur.h = seg / p.n_rt;
      cur.rt = seg % p.n_rt;
      cur.start = first + seg * len;
      break;
    }
    base += all;
  }
  return cur;
}

// Places of a warp's stretch: an equal share.
__device__ __forceinline__ int share(int total, int ctas) {
  const int per = (total + ctas * kWarps - 1) / (ctas * kWarps);
  return per < 1 ? 1 : per;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lo_bf16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

template <int D>
struct AttnSmem {
  static constexpr int kBytes = kBlk * (D + 8);
  alignas(128) uint8_t ring[kWarps][kStages<D>][2 * kBytes];
  // Of tile nt's columns 2t and 2t + 1: what a score is taken times, the sum of q, and the last position that they see.  (In
  // registers they made d = 128 spill.)
  float4 rows[kWarps][2][4];
  int2 last[kWarps][2][4];
};

// 16 bytes, global to shared memory, past L1; groups of them complete in order
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {  // all but the N newest groups of this thread
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Four transposed 8 x 8 matrices of 16-bit elements, whose rows' addresses the lanes give: lane (g, t) gets elements (2t, g) and
// (2t + 1, g) of each.
__device__ __forceinline__ void load_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

template <class T, int D, int NT, bool SPLIT>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? 2 : 1) attn_kernel(const __grid_constant__ AttnParams p) {
  static_assert(!SPLIT || NT == 1, "four rows are one tile");
  using Sm = AttnSmem<D>;
  constexpr int NI = SPLIT ? 2 : 4;  // tokens of a unit whose weights a lane has
  constexpr int kRows = 8 * NT, kBytes = Sm::kBytes, kHalf = kBlk * D / 2;  // bytes of a block, of its K or V codes
  constexpr int KW = D / 32;  // words of K codes a lane takes of a row
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Sm& sm = *reinterpret_cast<Sm*>(smem_raw);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane / 4, t = lane % 4;
  const int slot = warp * gridDim.x + blockIdx.x;  // neighbouring stretches on different SMs
  constexpr int S = kStages<D>;
  clear_ctrl(p.ctrl);
  launch_dependents();
  const int mine = lane < p.B ? blocks_of(p, lane) : 0;
  int total = places(mine);
  for (int b = lane + 32; b < p.B; b += 32) total += places(blocks_of(p, b));
  total = __reduce_add_sync(0xffffffffu, total) * p.c.Hkv * p.n_rt;
  const int per = share(total, gridDim.x);
  if (total == 0 || slot > (total - 1) / per) return;
  const int u0 = slot * per, u1 = min(u0 + per, total);
  Cursor seg = segment_at(p, u0, mine);

  // ---- the ring: the stretch's unit k goes to stage k % S; a unit's pages are looked up one unit ahead of its copy -----------
  Cursor pre = seg;
  int next = u0, pre_end = seg.end(), pg0 = 0, pg1 = 0, off = 0, filled = 0;
  const int32_t* row = p.c.table + (long long)seg.b * p.c.max_pages;
  const int in_page = (1 << p.page_shift) - 1, per_page = p.c.Hkv << p.page_shift;  // blocks of a page, and of all heads
  const uint8_t* lane_base = p.c.base + lane * 16;
  // A stage holds K's codes of both blocks, then V's, then the scales.  V's 16-byte pieces are XOR-swizzled by their rows, so that
  // eight rows of a piece fall on different banks.
  constexpr int kSwz = D == 128 ? 3 : 1;
  const uint32_t lane_ring = smem_u32(sm.ring[warp]) + lane * 16;
  const uint32_t lane_v = smem_u32(sm.ring[warp]) + 2 * kHalf + (lane ^ (lane >> 3 & kSwz)) * 16;
  uint32_t bad = 0;  // bit s: a block of stage s has no page
  auto look_up = [&]() {
    if (next >= pre_end) {
      pre.advance(p, next);
      pre_end = pre.end();
      row = p.c.table + (long long)pre.b * p.c.max_pages;
    }
    next = max(next, pre.start + kPad);
    const int blk = 2 * (next - pre.start - kPad);  // (past the stretch's end: a block of the segment all the same)
    pg0 = row[blk >> p.page_shift];
    off = (pre.h << p.page_shift) + (blk & in_page);
    pg1 = 0;  // any page: a last block without a second one reads what is there, and masks it
    if (p.page_shift == 0 && blk + 1 < pre.blocks) pg1 = row[blk + 1];
  };
  auto fill = [&]() {
    if (next < u1) {
      const int s = filled++ % S;
      if ((uint32_t)pg0 < (uint32_t)p.c.n_pages && (uint32_t)pg1 < (uint32_t)p.c.n_pages) {
        // (fewer than 2^31 blocks: checked on the host)
        const uint8_t* src[2];
        src[0] = lane_base + (unsigned long long)(uint32_t)(pg0 * per_page + off) * kBytes;
        src[1] = src[0] + kBytes;  // the second block follows the first where a page holds two
        if (p.page_shift == 0) src[1] = lane_base + (unsigned long long)(uint32_t)(pg1 * per_page + off) * kBytes;
        const uint32_t dst = lane_ring + s * (2 * kBytes), dst_v = lane_v + s * (2 * kBytes);
#pragma unroll
        for (int c = 0; c < 2 * kHalf; c += 512) copy16(dst + c, src[c / kHalf] + c % kHalf);
#pragma unroll
        for (int c = 0; c < 2 * kHalf; c += 512) copy16(dst_v + c, src[c / kHalf] + kHalf + c % kHalf);
        if (lane < 16) copy16(dst + 4 * kHalf, (lane < 8 ? src[0] : src[1] - 128) + 2 * kHalf);
      } else {
        bad |= 1u << s;
      }
      if (++next < u1) look_up();
    }
    copy_commit();  // a group for every unit, empty or not: they are counted
  };
  look_up();
  for (int s = 0; s < S; ++s) fill();

  int used = 0;
  for (int lo = u0, hi; lo < u1; lo = hi) {
    seg.advance(p, lo);
    const int begin = seg.start + kPad, from = max(lo, begin);
    hi = min(seg.end(), u1);
    if (from >= hi) continue;
    const int n = p.lens[seg.b];
    const int R = p.group * p.S;  // query rows of the KV head: row = new token * group + head of the group
    // the query row of column c of tile nt
    auto row_of = [&](int nt, int c) { return seg.rt * kRows + nt * 8 + (SPLIT ? c % 4 : c); };
    // ---- query fragments: column g of each tile, columns of q in the order of the K codes' words -----
    uint32_t qf[NT][KW][4];
    float up[NT], down[NT];  // the power of two that q's row g is taken times, and its inverse
    uint4 raw[NT][KW];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = row_of(nt, g);
      const T* q = static_cast<const T*>(p.q) + (long long)seg.b * p.sq.b +
                   (long long)(seg.h * p.group + row % p.group) * p.sq.h + (long long)(row / p.group) * p.sq.s + t * (D / 4);
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        raw[nt][w] = make_uint4(0, 0, 0, 0);
        if (row < R) {
          if (p.vec) {
            raw[nt][w] = *reinterpret_cast<const uint4*>(q + w * 8);
          } else {
            const uint16_t* e = reinterpret_cast<const uint16_t*>(q) + w * 8;
            raw[nt][w] = make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16, e[4] | (uint32_t)e[5] << 16,
                                    e[6] | (uint32_t)e[7] << 16);
          }
        }
      }
    }
    auto element = [](const uint4& v, int i) {
      const uint32_t e = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
      uint16_t h = (uint16_t)(i % 2 ? e >> 16 : e);
      return to_f32(*reinterpret_cast<T*>(&h));
    };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float big = 0.f;
#pragma unroll
      for (int w = 0; w < KW; ++w)
#pragma unroll
        for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(element(raw[nt][w], i)));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
      // 2^(14 - exponent of the row's largest); 1 if that is zero, subnormal or not finite
      const int ex = (int)(__float_as_uint(big) >> 23);
      const uint32_t power = ex == 0 || ex == 255 ? 127 : min(253, 127 + 14 - (ex - 127));  // (from 14 on)
      up[nt] = __uint_as_float(power << 23);
      down[nt] = __uint_as_float((254 - power) << 23);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          f[i] = element(raw[nt][w], i);
          sum += f[i];
          f[i] *= i % 2 ? up[nt] * 0.0625f : up[nt];  // the codes of odd columns stand 16 times too high
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) qf[nt][w][i] = pack_f16x2(f[i], f[i + 4]);
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      // (the last segment's units ended with all lanes' reads of these, and this one's begin behind a __syncwarp)
      if (t == 0) {
        float* to = reinterpret_cast<float*>(&sm.rows[warp][nt][g / 2]) + g % 2;
        to[0] = p.scale * kLog2e * 16777216.f * down[nt];
        to[2] = p.scale * kLog2e * sum;
        reinterpret_cast<int*>(&sm.last[warp][nt][g / 2])[g % 2] = n - p.S + row_of(nt, g) / p.group;
      }
    }
    float acc[NT][D / 16][4], eight[NT][4], m[NT][2], di[NT][2], l[NT][2], corr[NT][2];
    bool fresh = true;  // no unit yet: the first one sets the maxima (a column that sees nothing of it sees nothing later)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) acc[nt][i][0] = acc[nt][i][1] = acc[nt][i][2] = acc[nt][i][3] = 0.f;
      eight[nt][0] = eight[nt][1] = eight[nt][2] = eight[nt][3] = 0.f;
      m[nt][0] = m[nt][1] = 0.f;
      di[nt][0] = di[nt][1] = 1.f;
      l[nt][0] = l[nt][1] = corr[nt][0] = corr[nt][1] = 0.f;
    }
    // one unit: MASKED where some row does not see all of its tokens
    auto unit = [&](const uint8_t* stage, int j0, auto masked_tag) {
      constexpr bool MASKED = decltype(masked_tag)::value;
      // mma row g holds token g / 2 + 4 (g % 2) of a block, row g + 8 that plus 8
      const int tok = g / 2 + 4 * (g % 2);
      float xb[NT][8];  // block, token half, column
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 8; ++e) xb[nt][e] = 0.f;
      uint32_t ka[2][KW], kb[2][KW];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const uint8_t* blk = stage + b * kHalf;
        if constexpr (D == 128) {
          const uint4 a = *reinterpret_cast<const uint4*>(blk + tok * 64 + t * 16);
          const uint4 c = *reinterpret_cast<const uint4*>(blk + (tok + 8) * 64 + t * 16);
          ka[b][0] = a.x; ka[b][1] = a.y; ka[b][2] = a.z; ka[b][3] = a.w;
          kb[b][0] = c.x; kb[b][1] = c.y; kb[b][2] = c.z; kb[b][3] = c.w;
        } else {
          const uint2 a = *reinterpret_cast<const uint2*>(blk + tok * 32 + t * 8);
          const uint2 c = *reinterpret_cast<const uint2*>(blk + (tok + 8) * 32 + t * 8);
          ka[b][0] = a.x; ka[b][1] = a.y;
          kb[b][0] = c.x; kb[b][1] = c.y;
        }
      }
#pragma unroll
      for (int w = 0; w < KW; ++w)  // the two blocks' chains of products side by side
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const uint32_t a8 = half ? ka[b][w] >> 8 : ka[b][w], b8 = half ? kb[b][w] >> 8 : kb[b][w];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16(*reinterpret_cast<float(*)[4]>(&xb[nt][4 * b]), a8 & 0x000F000Fu, b8 & 0x000F000Fu, a8 & 0x00F000F0u,
                      b8 & 0x00F000F0u, qf[nt][w][2 * half], qf[nt][w][2 * half + 1]);
          }
      // x: scores in powers of two above m; w: weights; y: weights times V's scale, in units of 1 / di
      float x[NT][2 * NI], w[NT][2 * NI], y[NT][2 * NI], vo[NI], top = 0.f, kscale[NT][2], qsum[NT][2];
      int last[NT][2] = {};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float4 v = sm.rows[warp][nt][t];
        kscale[nt][0] = v.x; kscale[nt][1] = v.y;
        qsum[nt][0] = v.z; qsum[nt][1] = v.w;
        if (MASKED) {
          const int2 at = sm.last[warp][nt][t];
          last[nt][0] = at.x; last[nt][1] = at.y;
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2 * NI; ++e) x[nt][e] = SPLIT && t >= 2 ? xb[nt][(e + 4) % 8] : xb[nt][e];
      // the lane's token i: block, half; with SPLIT half of the lane's block
      const uint8_t* own = stage + 4 * kHalf + (SPLIT ? t / 2 * 128 : 0);
      const int own_tok = tok + (SPLIT ? t / 2 * kBlk : 0);
      auto pair_of = [&](int i, int kv) {
        return reinterpret_cast<const uint32_t*>(own + i / 2 * 128)[kv * 16 + tok + 8 * (i % 2)];
      };
      auto unseen = [&](int i, int nt, int c) { return MASKED && j0 + 16 * (i / 2) + 8 * (i % 2) + own_tok > last[nt][c]; };
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const uint32_t kp = pair_of(i, 0), vp = pair_of(i, 1);
        const float ks = lo_bf16(kp), ko = hi_bf16(kp), vs = lo_bf16(vp);
        vo[i] = fmaf(8.f, vs, hi_bf16(vp));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int e = 2 * i + c;
            x[nt][e] = fmaf(ks * kscale[nt][c], x[nt][e], fmaf(ko, qsum[nt][c], -m[nt][c]));
            if (unseen(i, nt, c)) x[nt][e] = -INFINITY;  // such a row may hold anything
            w[nt][e] = ex2_approx(x[nt][e]);
            y[nt][e] = unseen(i, nt, c) ? 0.f : w[nt][e] * (vs * di[nt][c]);
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2 * NI; ++e) top = fmax3(top, w[nt][e], y[nt][e]);
      if (__any_sync(0xffffffffu, fresh || top > kRaise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float a = -INFINITY, b = -INFINITY;  // largest score, largest exponent of a product
#pragma unroll
            for (int i = 0; i < NI; ++i) {
              if (unseen(i, nt, c)) continue;
              a = fmaxf(a, x[nt][2 * i + c]);
              b = fmaxf(b, x[nt][2 * i + c] + lg2_approx(lo_bf16(pair_of(i, 1))));
            }
#pragma unroll
            for (int o = 4; o < 32; o *= 2) {
              a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
              b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
            }
            const float up = a == -INFINITY ? 0.f : fresh ? a : fmaxf(a, 0.f);
            // the power of two, from 2^-126 to 2^126: at least the largest product so far, and at least the old one
            const float old = fresh ? -126.f : 127.f - (float)(__float_as_uint(di[nt][c]) >> 23) - up;
            const float nd = fminf(fmaxf(fmaxf(old, -126.f), ceilf(b - up)), 126.f);
            m[nt][c] += up;
            di[nt][c] = __uint_as_float((uint32_t)(127 - (int)ceilf(nd)) << 23);
            if (!fresh) {
              const float fa = ex2_approx(-up), fb = ex2_approx(old - ceilf(nd));
              l[nt][c] *= fa;
              corr[nt][c] *= fa;
              eight[nt][c] *= fb;
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                acc[nt][i][c] *= fb;
                acc[nt][i][2 + c] *= fb;
              }
            }
#pragma unroll
            for (int i = 0; i < NI; ++i) {
              const int e = 2 * i + c;
              if (unseen(i, nt, c)) continue;
              w[nt][e] = ex2_approx(x[nt][e] - up);
              y[nt][e] = w[nt][e] * (lo_bf16(pair_of(i, 1)) * di[nt][c]);
            }
          }
        fresh = false;
      }
      // the lane's row of the matrices: token and 16-byte piece
      const int mt = lane % 8 / 2 + 4 * (lane % 2) + lane / 8 % 2 * 8, mj = lane / 16;
      const uint32_t at_v = smem_u32(stage) + 2 * kHalf + mt * (D / 2) + ((mj ^ (D == 128 ? mt / 2 & 3 : mt / 4 & 1)) * 16);
      uint32_t both[NT][2];  // P of the block; with SPLIT columns 0..3 are of the first block, 4..7 of the second
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if (!SPLIT || b == 0) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int i = SPLIT ? h : 2 * b + h;
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                l[nt][c] += w[nt][2 * i + c];
                if (!unseen(i, nt, c)) corr[nt][c] = fmaf(w[nt][2 * i + c], vo[i], corr[nt][c]);
              }
              both[nt][h] = transpose8x8(pack_f16x2(y[nt][2 * i], y[nt][2 * i + 1]));
            }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_f16(eight[nt], 0x00080008u, 0x00080008u, 0x00080008u, 0x00080008u, both[nt][0], both[nt][1]);
        }
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) pb[nt][h] = SPLIT && g / 4 != b ? 0u : both[nt][h];
        // V's codes: a 16-bit element is four columns of a token, an element of the transposed matrices those of tokens t, t + 4
        // (contraction 2t, 2t + 1) or, in the odd ones, t + 8, t + 12; the lane's columns are 32 j + 4 g + 0 .. 3
#pragma unroll
        for (int j = 0; j < D / 32; j += 2) {
          uint32_t r[4];
          load_trans(r, (at_v ^ (j * 16)) + b * kHalf);
          constexpr uint32_t L = 0x000F000Fu, H = 0x00F000F0u;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            // two columns to an mma, the even one on row g, the odd one, 16 times too high, on g + 8
            const uint32_t lo = r[2 * k], hi = r[2 * k + 1], los = lo >> 8, his = hi >> 8;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_f16(acc[nt][2 * (j + k)], lo & L, lo & H, hi & L, hi & H, pb[nt][0], pb[nt][1]);
              mma_f16(acc[nt][2 * (j + k) + 1], los & L, los & H, his & L, his & H, pb[nt][0], pb[nt][1]);
            }
          }
        }
      }
    };
    // ---- the units of the segment --------------------------------------------------------------------
    const int all_see = n - p.S;  // the last position that every row sees
    for (int u = from; u < hi; ++u) {
      const int s = used++ % S;
      copy_wait<S - 1>();
      __syncwarp();  // every lane's copies are there
      if (bad >> s & 1u) {
        bad ^= 1u << s;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) l[nt][0] = l[nt][1] = NAN;
      } else {
        const int j0 = (u - begin) * kUnit;
        if (j0 + kUnit - 1 <= all_see) unit(sm.ring[warp][s], j0, std::false_type());
        else unit(sm.ring[warp][s], j0, std::true_type());
      }
      __syncwarp();  // every lane has read the stage
      fill();
    }
    // ---- the results: o if the segment is whole, else a piece ----------------------------------------
    const bool whole = from == begin && hi == seg.end();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float sum = l[nt][c], base = corr[nt][c];
#pragma unroll
        for (int o = 4; o < 32; o *= 2) {
          sum += __shfl_xor_sync(0xffffffffu, sum, o);
          base += __shfl_xor_sync(0xffffffffu, base, o);
        }
        const float fo = 1.f / di[nt][c];
        float top = sum == 0.f ? kLowest : m[nt][c];  // kLowest: the column saw nothing
        float v[D / 8];  // the lane's columns, 32 j + 4 g + 0 .. 3
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          v[2 * i] = fmaf((acc[nt][i][c] - eight[nt][c]) * 16777216.f, fo, base);
          v[2 * i + 1] = fmaf(fmaf(-16.f, eight[nt][c], acc[nt][i][2 + c]) * 1048576.f, fo, base);
        }
        if constexpr (SPLIT) {  // the row's two columns, in lanes t and t + 2
          const float other = __shfl_xor_sync(0xffffffffu, top, 2), both = fmaxf(top, other), f = ex2_approx(top - both);
          top = both;
          sum *= f;
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            v[i] *= f;
            v[i] += __shfl_xor_sync(0xffffffffu, v[i], 2);
          }
        }
        const int r = row_of(nt, 2 * t + c);
        if (r >= R || (SPLIT && t >= 2)) continue;
        if (whole) {
          const long long hq = seg.h * p.group + r % p.group, i = r / p.group;
          T* out = static_cast<T*>(p.o) + seg.b * p.so.b + hq * p.so.h + i * p.so.s + g * 4;
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            struct alignas(8) Four { T e[4]; } w;
#pragma unroll
            for (int e = 0; e < 4; ++e) w.e[e] = from_f32<T>(sum == 0.f ? 0.f : v[j * 4 + e] * inv);
            if (p.vec_o) {
              *reinterpret_cast<Four*>(out + j * 32) = w;
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) out[j * 32 + e] = w.e[e];
            }
          }
          if (g == 0) p.lse[(seg.b * (long long)p.Hq + hq) * p.S + i] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
        } else {
          float* part = p.part + ((2ll * slot + (lo == u0 ? 0 : 1)) * kRows + r - seg.rt * kRows) * kPart<D>;
#pragma unroll
          for (int q = 0; q < D / 32; ++q)
            *reinterpret_cast<float4*>(part + q * 32 + g * 4) = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
          if (g == 0) {
            part[D] = top;
            part[D + 1] = sum;
          }
        }
      }
  }
}

// The query rows of the segments that lie in several stretches, or in none: a row to a warp where segments are many, or to a
// block, whose warps take every 32nd piece.  Many segments have few pieces each on average only: one sequence of 131072
// positions among 63 of 16 has hundreds, which its rows' warps join one after another (110 us, where its bytes take 21).
template <class T, int D, int NT>
__global__ void __launch_bounds__(1024) combine_kernel(const __grid_constant__ AttnParams p, int ctas, int rows) {
  constexpr int kRows = 8 * NT, E = D / 32;
  __shared__ float so[32][D], sl[32], st[32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const bool by_block = blockDim.x == 1024;
  const int R = p.group * p.S;
  const int at = by_block ? blockIdx.x : blockIdx.x * (blockDim.x / 32) + warp;
  const int row = at % R, h = at / R % p.c.Hkv, b = min(at / R / p.c.Hkv, p.B - 1);
  const int rt = row / kRows, hq = h * p.group + row % p.group, i = row / p.group;
  // where the segment begins, and how many units there are
  const int blocks = blocks_of(p, b), len = (blocks + 1) / 2;
  const int per = share(units_before(p, p.B), ctas);
  const int start = units_before(p, b) + (h * p.n_rt + rt) * places(blocks), first = start + kPad;
  // No warp leaves before the kernel that writes the pieces has ended: what follows on the stream may rely on both.
  wait_previous();
  if (at >= rows) return;
  T* o = static_cast<T*>(p.o) + b * p.so.b + hq * p.so.h + i * p.so.s;
  float* lse = p.lse + ((long long)b * p.Hq + hq) * p.S + i;
  if (len == 0) {
    if (by_block && warp) return;
    const bool empty = p.lens[b] == 0;
#pragma unroll
    for (int e = 0; e < E; ++e) o[lane + 32 * e] = from_f32<T>(empty ? 0.f : NAN);
    if (lane == 0) *lse = empty ? -INFINITY : NAN;
    return;
  }
  const int c0 = first / per, c1 = (first + len - 1) / per;
  if (c0 == c1) return;
  float top = kLowest, sum = 0.f, acc[E] = {};
#pragma unroll 4
  for (int c = by_block ? c0 + warp : c0; c <= c1; c += by_block ? 32 : 1) {
    const float* part = p.part + ((2ll * c + (c * per >= start ? 0 : 1)) * kRows + row % kRows) * kPart<D>;
    const float mc = part[D], lc = part[D + 1];
    float v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = part[lane + 32 * e];
    const float t = fmaxf(top, mc), f = ex2_approx(top - t), w = ex2_approx(mc - t);
    top = t;
    sum = sum * f + lc * w;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * f + v[e] * w;
  }
  if (by_block) {
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane + 32 * e] = acc[e];
    if (lane == 0) {
      st[warp] = top;
      sl[warp] = sum;
    }
    __syncthreads();
    if (warp) return;
    top = warp_max(st[lane]);
    const float f = ex2_approx(st[lane] - top);
    sum = sl[lane] * f;
#pragma unroll
    for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int w = 0; w < 32; ++w) {
      const float fw = __shfl_sync(0xffffffffu, f, w);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += so[w][lane + 32 * e] * fw;
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) o[lane + 32 * e] = from_f32<T>(sum == 0.f ? 0.f : acc[e] / sum);
  if (lane == 0) *lse = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

// ------------------------------------------------------------------------------------------------
// Host side
// ------------------------------------------------------------------------------------------------
static int check_shape(const psr_kv4_shape* sh) {
  if (!sh) return PSR_ERR_ARG;
  if (sh->B < 0 || sh->S < 0 || sh->Hq < 1 || sh->Hkv < 1 || sh->n_pages < 1 || sh->max_pages < 1) return PSR_ERR_ARG;
  if (sh->type != PSR_BF16 && sh->type != PSR_F16) return PSR_ERR_ARG;
  if (sh->S > 1 << 28) return PSR_ERR_UNSUPPORTED;
  if (sh->Hq % sh->Hkv != 0 || (sh->d != 64 && sh->d != 128)) return PSR_ERR_UNSUPPORTED;
  if ((double)sh->n_pages * sh->Hkv * sh->page / 16 >= 2147483648.0) return PSR_ERR_UNSUPPORTED;
  if (sh->page < 16 || sh->page > 256 || (sh->page & (sh->page - 1)) != 0) return PSR_ERR_UNSUPPORTED;
  if ((long long)sh->max_pages * sh->page >= (1LL << 31)) return PSR_ERR_UNSUPPORTED;
  return PSR_OK;
}

static int log2_of(int page) {
  int n = 0;
  while (1 << n < page) ++n;
  return n;
}

static Cache cache_of(const psr_kv4_shape* sh, const void* cache, const int32_t* table) {
  return {const_cast<uint8_t*>(static_cast<const uint8_t*>(cache)), table, sh->Hkv, sh->d, sh->page, sh->n_pages,
          sh->max_pages, log2_of(sh->page)};
}

template <class Go>
static int by_type(const psr_kv4_shape* sh, Go&& go) {
  if (sh->type == PSR_BF16)
    return sh->d == 64 ? go(__nv_bfloat16(), std::integral_constant<int, 64>())
                       : go(__nv_bfloat16(), std::integral_constant<int, 128>());
  return sh->d == 64 ? go(__half(), std::integral_constant<int, 64>()) : go(__half(), std::integral_constant<int, 128>());
}

template <class T, int D, int NT, bool SPLIT>
static int launch_attn(AttnParams& p, int dev, int n_sm, cudaStream_t st) {
  static std::mutex mu;
  static bool known[64] = {};
  constexpr int smem = (int)sizeof(AttnSmem<D>);
  static_assert(2 * (smem + 1024) <= 233472, "shared memory");
  {
    std::lock_guard<std::mutex> lk(mu);
    if (dev < 0 || dev >= 64 || !known[dev]) {
      if (cudaFuncSetAttribute(attn_kernel<T, D, NT, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
        cudaGetLastError();
        return PSR_ERR_CUDA;
      }
      if (dev >= 0 && dev < 64) known[dev] = true;
    }
  }
  const long long R = (long long)p.group * p.S;
  p.n_rt = (int)((R + 8 * NT - 1) / (8 * NT));
  const int ctas = (n_sm < 152 ? n_sm : 152) * (NT == 1 ? 2 : 1);
  attn_kernel<T, D, NT, SPLIT><<<ctas, kWarps * 32, smem, st>>>(p);
  if (launch_status() != PSR_OK) return PSR_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  // a block to a row where the stretches are more than 16 to a segment on average
  const int rows = (int)(p.B * p.c.Hkv * R);
  const bool by_block = (long long)p.B * p.c.Hkv * p.n_rt * 16 < (long long)ctas * kWarps;
  cfg.gridDim = dim3((unsigned)(by_block ? rows : (rows + 7) / 8));
  cfg.blockDim = dim3(by_block ? 1024 : 256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, combine_kernel<T, D, NT>, p, ctas, rows) != cudaSuccess) {
    cudaGetLastError();
    return PSR_ERR_CUDA;
  }
  return PSR_OK;
}

// Blocks of an append or a read; 0 if there are too many.
static unsigned move_blocks(const psr_kv4_shape* sh, MoveParams& p) {
  const int tokens = sh->d == 64 ? Rows<64>::kTokens : Rows<128>::kTokens;
  p.S = sh->S;
  p.tiles = (sh->S + tokens - 1) / tokens;
  const double n = (double)sh->B * sh->Hkv * p.tiles;
  return n < 2147483648.0 ? (unsigned)(sh->B * sh->Hkv * p.tiles) : 0u;
}

// Every row of a strided tensor starts on a 16-byte boundary.
static bool rows_aligned(const void* x, const psr_strides* st, int B, int H, int S) {
  auto even = [](long long stride, int n) { return n <= 1 || stride % 8 == 0; };
  return aligned_to(x, 16) && even(st->b, B) && even(st->h, H) && even(st->s, S);
}

}  // namespace kv4
}  // namespace psr

using namespace psr;
using namespace psr::kv4;

extern "C" {

size_t psr_kv4_cache_bytes(const psr_kv4_shape* sh) {
  if (check_shape(sh) != PSR_OK) return 0;
  return (size_t)sh->n_pages * sh->Hkv * sh->page * (sh->d + 8);
}

int psr_kv4_append(const psr_kv4_shape* sh, const void* k, const psr_strides* ks, const void* v, const psr_strides* vs,
                   void* cache, const int32_t* table, const int32_t* start, const int32_t* count, void* stream) {
  if (!sh || !k || !ks || !v || !vs || !cache || !table || !start) return PSR_ERR_ARG;
  if (!aligned_to(k, 2) || !aligned_to(v, 2) || !aligned_to(cache, 16) || !aligned_to(table, 4) ||
      !aligned_to(start, 4) || !aligned_to(count, 4))
    return PSR_ERR_ARG;
  int rc = check_shape(sh);
  if (rc != PSR_OK) return rc;
  if ((rc = check_device(nullptr)) != PSR_OK) return rc;
  if (sh->B == 0 || sh->S == 0) return PSR_OK;
  MoveParams p = {};
  p.c = cache_of(sh, cache, table);
  p.in[0] = k; p.in[1] = v;
  p.st[0] = *ks; p.st[1] = *vs;
  p.start = start; p.count = count;
  p.vec = rows_aligned(k, ks, sh->B, sh->Hkv, sh->S) && rows_aligned(v, vs, sh->B, sh->Hkv, sh->S);
  const unsigned blocks = move_blocks(sh, p);
  if (!blocks) return PSR_ERR_UNSUPPORTED;
  return by_type(sh, [&](auto t, auto d) {
    append_kernel<decltype(t), decltype(d)::value><<<blocks, kMove, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return launch_status();
  });
}

int psr_kv4_read(const psr_kv4_shape* sh, const void* cache, const int32_t* table, const int32_t* start,
                 const int32_t* count, void* k, void* v, void* stream) {
  if (!sh || !k || !v || !cache || !table || !start) return PSR_ERR_ARG;
  if (!aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(cache, 16) || !aligned_to(table, 4) ||
      !aligned_to(start, 4) || !aligned_to(count, 4))
    return PSR_ERR_ARG;
  int rc = check_shape(sh);
  if (rc != PSR_OK) return rc;
  if ((rc = check_device(nullptr)) != PSR_OK) return rc;
  if (sh->B == 0 || sh->S == 0) return PSR_OK;
  MoveParams p = {};
  p.c = cache_of(sh, cache, table);
  p.out[0] = k; p.out[1] = v;
  p.start = start; p.count = count;
  const unsigned blocks = move_blocks(sh, p);
  if (!blocks) return PSR_ERR_UNSUPPORTED;
  return by_type(sh, [&](auto t, auto d) {
    read_kernel<decltype(t), decltype(d)::value><<<blocks, kMove, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return launch_status();
  });
}

size_t psr_kv4_attn_workspace_bytes(const psr_kv4_shape* sh) {
  if (check_shape(sh) != PSR_OK) return 0;
  // a tile of 16 rows runs one CTA to an SM, one of 8 rows two
  return 256 + (size_t)2 * kMaxCtas * kWarps * 8 * (sh->d + 4) * 4;
}

int psr_kv4_attn(const psr_kv4_shape* sh, const void* q, const psr_strides* qs, const void* cache, const int32_t* table,
                 const int32_t* lens, void* o, const psr_strides* os, float* lse, void* workspace, size_t ws_bytes,
                 void* stream) {
  if (!sh || !q || !qs || !cache || !table || !lens || !o || !os || !lse || !workspace) return PSR_ERR_ARG;
  if (!aligned_to(q, 2) || !aligned_to(o, 2) || !aligned_to(lse, 4) || !aligned_to(cache, 16) ||
      !aligned_to(table, 4) || !aligned_to(lens, 4) || !aligned_to(workspace, 256))
    return PSR_ERR_ARG;
  int rc = check_shape(sh);
  if (rc != PSR_OK) return rc;
  if (ws_bytes < psr_kv4_attn_workspace_bytes(sh) || !std::isfinite(sh->scale)) return PSR_ERR_ARG;
  const long long rows = (long long)sh->B * sh->Hq * sh->S;
  const long long tiles = ((long long)sh->Hq / sh->Hkv * sh->S + 7) / 8;
  if (rows >= (1LL << 30) || (double)sh->B * sh->Hkv * tiles * ((double)sh->max_pages * sh->page / kUnit + 1 + kPad) >= kMaxPlaces)
    return PSR_ERR_UNSUPPORTED;
  int n_sm = 0, dev = 0;
  if ((rc = check_device(&n_sm)) != PSR_OK) return rc;
  if (cudaGetDevice(&dev) != cudaSuccess) return PSR_ERR_CUDA;
  if (rows == 0) {  // the control block still tells of a call that went well
    if (cudaMemsetAsync(workspace, 0, sizeof(Ctrl), static_cast<cudaStream_t>(stream)) == cudaSuccess) return PSR_OK;
    cudaGetLastError();
    return PSR_ERR_CUDA;
  }
  AttnParams p = {};
  p.c = cache_of(sh, cache, table);
  p.q = q; p.o = o; p.lse = lse; p.lens = lens;
  p.sq = *qs; p.so = *os;
  p.B = sh->B; p.Hq = sh->Hq; p.S = sh->S;
  p.group = sh->Hq / sh->Hkv;
  p.page_shift = p.c.shift - 4;
  p.vec = rows_aligned(q, qs, sh->B, sh->Hq, sh->S);
  p.vec_o = rows_aligned(o, os, sh->B, sh->Hq, sh->S);
  p.scale = sh->scale > 0.f ? sh->scale : 1.f / sqrtf((float)sh->d);
  p.ctrl = static_cast<Ctrl*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + 256);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return by_type(sh, [&](auto t, auto d) {
    constexpr int D = decltype(d)::value;
    const long long rows = (long long)sh->Hq / sh->Hkv * sh->S;  // of a KV head
    return rows <= 4   ? launch_attn<decltype(t), D, 1, true>(p, dev, n_sm, st)
           : rows <= 8 ? launch_attn<decltype(t), D, 1, false>(p, dev, n_sm, st)
                       : launch_attn<decltype(t), D, 2, false>(p, dev, n_sm, st);
  });
}

}  // extern "C"
