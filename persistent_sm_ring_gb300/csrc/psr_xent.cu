// Softmax cross entropy of the output projection l = x w^T over a large vocabulary, and its gradients, on sm_103a.  The logits are
// never kept:
//
//   loss_i = lse_i - (1 - s) l_i[t_i] - s mean(l_i) + z lse_i^2,   lse_i = log sum_j exp l_ij
//   slope  d_ij = g_i (p_ij (1 + 2 z lse_i) - s/V - (1 - s) [j = t_i]),  p = exp(l - lse),   dx = d w,  dw = d^T x
//
// Forward: the logits' product reduces its sums to (r, s), sum exp(l) = s 2^r, for every kGroup columns; a second kernel joins
// them.  Backward: by pieces of the vocabulary, the logits again, turned into slopes of 16 bits on their way out of
// tensor memory; dw's rows of the piece; and the piece's share of dx, summed in fp32 over the pieces.
//
// Rows without a target are left out: the others are packed first, which costs a copy of x and saves their share of the products, and
// keeps whatever stands in the rows left out (NaN, say) from dw.  Up to kFew rows, where the products read W and hardly multiply,
// they stay in place as zeros, and so that a weight that is not finite reaches neither their slopes nor their dx, those are set to zeros.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "psr_control.cuh"
#include "psr_host.h"
#include "psr_linear_mma.cuh"

namespace psr {
namespace xent {

using namespace linear;

constexpr int kFew = 64;

// ------------------------------------------------------------------------------------------------
// Rows that count
// ------------------------------------------------------------------------------------------------
struct RowParams {
  const uint16_t* x;
  long long ldx;
  uint16_t* xc;  // the rows that count, 16-byte aligned, zeros to the next multiple of kBK
  long long ldxc;
  int M, V, K, vec;  // vec: x's rows are 16-byte aligned
  int per;           // rows of a block, at most 256
  // of each block's rows: those that count, the largest |g| and |g (1 + 2 z lse)|; null: each block looks at all rows itself
  float4* sums;
  int packed;        // else every row stays where it is, and those that do not count are zeros
  const int64_t* targets;
  long long step, ignore;
  int* count;
  int* index;
  int* target;
  float* loss;  // forward: of the rows that do not count
  float* lse;
  // backward
  const float* dloss;
  long long dstep;
  const float* lse_in;
  float smoothing, z;
  int half;
  float4* coef;
  float* unit;
  uint16_t* dx;  // rows that do not count
  Ctrl* clear;
};

__device__ __forceinline__ int64_t target_of(const RowParams& p, long long i) { return p.targets[i * p.step]; }
__device__ __forceinline__ bool counts(const RowParams& p, int64_t t) { return t >= 0 && t < p.V && t != p.ignore; }

// A row's |g| and |g (1 + 2 z lse)|, as far as finite.
__device__ __forceinline__ void most_of(const RowParams& p, long long i, float& most, float& scaled) {
  const float g = fabsf(p.dloss[i * p.dstep]), a = fabsf(g * (1.f + 2.f * p.z * p.lse_in[i]));
  if (g <= FLT_MAX) most = fmaxf(most, g);
  if (a <= FLT_MAX) scaled = fmaxf(scaled, a);
}

// Of many rows: what each of rows_kernel's blocks has, so that none has to look at them all (M^2 / 256 targets: 4 ms at 10^6 rows).
constexpr int kScanMost = 16384;
template <bool BWD>
__global__ void __launch_bounds__(256) block_kernel(const __grid_constant__ RowParams p) {
  __shared__ float most_warp[8], scaled_warp[8];
  clear_ctrl(p.clear);
  const long long i = blockIdx.x * 256ll + threadIdx.x;
  const bool in = i < p.M && counts(p, target_of(p, i));
  float most = 0.f, scaled = 0.f;
  if (BWD && in) most_of(p, i, most, scaled);
  const int n = __syncthreads_count(in);
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    scaled = fmaxf(scaled, __shfl_xor_sync(0xffffffffu, scaled, o));
  }
  if (threadIdx.x % 32 == 0) {
    most_warp[threadIdx.x / 32] = most;
    scaled_warp[threadIdx.x / 32] = scaled;
  }
  __syncthreads();
  if (threadIdx.x) return;
  for (int w = 1; w < 8; ++w) {
    most = fmaxf(most, most_warp[w]);
    scaled = fmaxf(scaled, scaled_warp[w]);
  }
  p.sums[blockIdx.x] = make_float4((float)n, most, scaled, 0.f);
}

// The slopes are multiplied by a power of two over the largest g (1 - s) on their way into 16 bits, and the sums of products by its
// inverse: the target's share of the row with the largest g is then a power of two and rounds to itself, and fp16, which ends at
// 2^-24, holds p down to 2^-37 of it.
template <bool BWD>
__global__ void __launch_bounds__(256) rows_kernel(const __grid_constant__ RowParams p) {
  __shared__ int n_warp[8], place[256];
  __shared__ float most_warp[8], scaled_warp[8];
  clear_ctrl(p.clear);
  launch_dependents();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const long long r0 = (long long)blockIdx.x * p.per;
  const int rows = (int)min((long long)p.per, p.M - r0);
  int before = 0;
  if (p.packed) {
    if (p.sums) {
#pragma unroll 4
      for (int b = threadIdx.x; b < (int)blockIdx.x; b += 256) before += (int)p.sums[b].x;
    } else {
#pragma unroll 4
      for (long long i = threadIdx.x; i < r0; i += 256) before += counts(p, target_of(p, i));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    if (lane == 0) n_warp[warp] = before;
    __syncthreads();
    before = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) before += n_warp[w];
    __syncthreads();
  }
  const int64_t t = (int)threadIdx.x < rows ? target_of(p, r0 + threadIdx.x) : -1;
  const bool in = (int)threadIdx.x < rows && counts(p, t);
  const uint32_t ins = __ballot_sync(0xffffffffu, in);
  if (lane == 0) n_warp[warp] = __popc(ins);
  __syncthreads();
  int own = 0, at = before + __popc(ins & ((1u << lane) - 1));
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    if (w < warp) at += n_warp[w];
    own += n_warp[w];
  }
  if (!p.packed) at = (int)r0 + threadIdx.x;
  if ((int)threadIdx.x < rows) place[threadIdx.x] = in ? at : -1;
  __syncthreads();

  if constexpr (BWD) {
    float most = 0.f, scaled = 0.f;
    if (p.sums) {
#pragma unroll 4
      for (int b = threadIdx.x; b < (int)gridDim.x; b += 256) {
        const float4 f = p.sums[b];
        most = fmaxf(most, f.y);
        scaled = fmaxf(scaled, f.z);
      }
    } else {
#pragma unroll 4
      for (long long i = threadIdx.x; i < p.M; i += 256)
        if (counts(p, target_of(p, i))) most_of(p, i, most, scaled);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
      scaled = fmaxf(scaled, __shfl_xor_sync(0xffffffffu, scaled, o));
    }
    if (lane == 0) {
      most_warp[warp] = most;
      scaled_warp[warp] = scaled;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      most = fmaxf(most, most_warp[w]);
      scaled = fmaxf(scaled, scaled_warp[w]);
    }
    // (a normal number: the product may round to zero)
    const float unit = most > 0.f ? fmaxf(most * (1.f - p.smoothing), FLT_MIN) : 1.f;
    int e = 0;
    if (p.half) {
      // The three terms of a slope over the unit are at most 2^e, 2^e (of few columns much smoothed, the largest) and 1.
      frexpf(fmaxf(fmaxf(scaled / unit, 1.f), p.smoothing / p.V / (1.f - p.smoothing)), &e);
      e = max(14 - e, -100);
    }
    const float power = ldexpf(1.f, e);
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.unit = unit / power;
    if ((int)threadIdx.x < rows && (in || !p.packed)) {
      float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
      if (in) {
        const float g = p.dloss[(r0 + threadIdx.x) * p.dstep] / unit * power, lse = p.lse_in[r0 + threadIdx.x];
        c = make_float4(lse * kLog2e, g * (1.f + 2.f * p.z * lse), g * (p.smoothing / p.V), g * (1.f - p.smoothing));
      }
      p.coef[at] = c;
    }
  }
  if (p.packed && in) p.index[at] = (int)(r0 + threadIdx.x);
  if ((int)threadIdx.x < rows && (in || !p.packed)) p.target[at] = in ? (int)t : -1;
  if (!BWD && p.packed && (int)threadIdx.x < rows && !in) {
    const float f = t == p.ignore ? 0.f : __int_as_float(0x7FC00000);
    p.loss[r0 + threadIdx.x] = f;
    p.lse[r0 + threadIdx.x] = f;
  }

  const int chunks = (p.K + 7) / 8;
  auto clear_row = [&](long long r) {
    uint4* to = reinterpret_cast<uint4*>(p.xc + r * p.ldxc);
    for (int c = lane; c < chunks; c += 32) to[c] = make_uint4(0, 0, 0, 0);
  };
  for (int r = warp; r < rows; r += 8) {
    const long long i = r0 + r, to = place[r];
    if (to >= 0) {
      const uint16_t* from = p.x + i * p.ldx;
      uint4* row = reinterpret_cast<uint4*>(p.xc + to * p.ldxc);
      if (p.vec) {
#pragma unroll 4
        for (int c = lane; c < chunks; c += 32) row[c] = reinterpret_cast<const uint4*>(from)[c];
      } else {
        const uint8_t* first = reinterpret_cast<const uint8_t*>(p.x);
        const uint8_t* past = reinterpret_cast<const uint8_t*>(p.x + (p.M - 1ll) * p.ldx + p.K);
        for (int c = lane; c < chunks; c += 32) row[c] = load8(from + c * 8, p.K - c * 8, first, past);
      }
    } else {
      if (!p.packed) clear_row(i);
      if (BWD && p.dx && p.packed)
        for (int k = lane; k < p.K; k += 32) p.dx[i * p.K + k] = 0;
    }
  }
  if (p.packed && blockIdx.x == gridDim.x - 1) {
    const int total = before + own, end = (total + kBK - 1) / kBK * kBK;
    if (threadIdx.x == 0) *p.count = total;
    for (int r = total + warp; r < end; r += 8) clear_row(r);
  }
}

// ------------------------------------------------------------------------------------------------
// One row: dot products
// ------------------------------------------------------------------------------------------------
// Bound by reading W once.  A warp takes rows of W in turn, a lane 16 bytes of one at a time, and asks for the piece kDotAhead further on, in
// the next row perhaps, as it takes one; its lanes keep the sum of exponentials.  48 warps with four pieces in flight: 32000 x 4096 in 45.6
// us with the join, 5.75 TB/s; 32 with eight 47.5, 64 with two 46.9.
constexpr int kDotThreads = 256, kDotBlocks = 6, kDotAhead = 4;  // blocks of an SM, pieces of a lane in flight

struct DotParams {
  const void* x;
  const void* w;
  long long ldw;
  int V, K;
  const int64_t* target;
  float2* stats;  // of each block
  float* sums;
  float* at;
  Ctrl* clear;
};

template <class T>
__global__ void __launch_bounds__(kDotThreads, kDotBlocks) dot_kernel(const __grid_constant__ DotParams p) {
  constexpr int kAhead = kDotAhead;
  constexpr bool kHalfType = std::is_same<T, __half>::value;
  __shared__ float2 part[kDotThreads / 32];
  __shared__ float part_sum[kDotThreads / 32];
  clear_ctrl(p.clear);
  launch_dependents();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, n_warps = gridDim.x * (kDotThreads / 32);
  const int64_t target = *p.target;
  const T* x = static_cast<const T*>(p.x);
  ExpSum e = {-FLT_MAX, 0.f};
  float sum = 0.f, acc = 0.f;
  // the piece asked for next and the one taken next, each by row and first column
  int row_in = blockIdx.x * (kDotThreads / 32) + warp, k_in = lane * 8, row = row_in, k = k_in;
  uint4 v[kAhead];
  auto load = [&](int a) {
    v[a] = make_uint4(0, 0, 0, 0);
    if (row_in < p.V && k_in < p.K) v[a] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const T*>(p.w) + row_in * p.ldw + k_in));
    k_in += 256;
    if (k_in - lane * 8 >= p.K) {
      k_in = lane * 8;
      row_in += n_warps;
    }
  };
#pragma unroll
  for (int a = 0; a < kAhead; ++a) load(a);
  while (row < p.V) {
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (row >= p.V) break;
      if (k < p.K) {
        const uint4 u = *reinterpret_cast<const uint4*>(x + k);
        const uint32_t f[4] = {u.x, u.y, u.z, u.w}, g[4] = {v[a].x, v[a].y, v[a].z, v[a].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float al, ah, bl, bh;
          unpack16(f[q], kHalfType, al, ah);
          unpack16(g[q], kHalfType, bl, bh);
          acc = fmaf(al, bl, acc);
          acc = fmaf(ah, bh, acc);
        }
      }
      load(a);
      k += 256;
      if (k - lane * 8 < p.K) continue;
#pragma unroll
      for (int o = 16; o; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
      const float ref = exp_ref(e.r, acc);
      e = {ref, e.s * ex2_approx(e.r - ref) + ex2_approx(fmaf(acc, kLog2e, -ref))};
      sum += acc;
      if (row == target && lane == 0) *p.at = acc;
      acc = 0.f;
      k = lane * 8;
      row += n_warps;
    }
  }
  if (lane == 0) {
    part[warp] = make_float2(e.r, e.s);
    part_sum[warp] = sum;
  }
  __syncthreads();
  if (threadIdx.x) return;
  sum = 0.f;
  e = {-FLT_MAX, 0.f};
  for (int w = 0; w < kDotThreads / 32; ++w) {
    const float ref = fmaxf(e.r, part[w].x);
    e = {ref, e.s * ex2_approx(e.r - ref) + part[w].y * ex2_approx(part[w].x - ref)};
    sum += part_sum[w];
  }
  p.stats[blockIdx.x] = make_float2(e.r, e.s);
  if (p.sums) p.sums[blockIdx.x] = sum;
}

// ------------------------------------------------------------------------------------------------
// The losses from the groups' sums
// ------------------------------------------------------------------------------------------------
struct FinishParams {
  const float2* stats;
  const float* sums;
  long long group_at, row_at;
  int groups;
  const float* at;
  const int* count;  // packed rows
  const int* index;
  const int64_t* targets;  // else
  long long step, ignore;
  int M, V;
  int lanes;  // threads to a row: a power of two; the others of a block take the rows that follow
  float smoothing, z;
  float* loss;
  float* lse;
};

// e and the sums g, some of which may be no group's.
template <int N>
__device__ __forceinline__ void add_groups(ExpSum& e, const float2 (&g)[N]) {
  float ref = e.r, s = 0.f;
#pragma unroll
  for (int k = 0; k < N; ++k) ref = fmaxf(ref, g[k].x);
#pragma unroll
  for (int k = 0; k < N; ++k) s = fmaf(g[k].y, ex2_approx(g[k].x - ref), s);
  e = {ref, fmaf(e.s, ex2_approx(e.r - ref), s)};
}

__global__ void __launch_bounds__(256) finish_kernel(const __grid_constant__ FinishParams p) {
  __shared__ float2 part[256];
  __shared__ float part_sum[256];
  const int per = 256 / p.lanes, r = threadIdx.x % per, g0 = threadIdx.x / per;
  const long long i = (long long)blockIdx.x * per + r;
  wait_previous();
  const int rows = p.count ? *p.count : p.M;
  if ((long long)blockIdx.x * per >= rows) return;
  ExpSum e = {-FLT_MAX, 0.f};
  float sum = 0.f;
  long long to = i;  // the row's place, and the target's logit
  float at_target = 0.f;
  if (g0 == 0 && i < rows) {
    if (p.index) to = p.index[i];
    at_target = p.at[i];
  }
  if (i < rows) {
    constexpr int N = 8;  // groups in flight
    for (int first = g0; first < p.groups; first += N * p.lanes) {
      float2 g[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int at = first + k * p.lanes;
        g[k] = at < p.groups ? p.stats[at * p.group_at + i * p.row_at] : make_float2(-FLT_MAX, 0.f);
      }
      if (p.sums) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const int at = first + k * p.lanes;
          if (at < p.groups) sum += p.sums[at * p.group_at + i * p.row_at];
        }
      }
      add_groups(e, g);
    }
  }
  part[threadIdx.x] = make_float2(e.r, e.s);
  part_sum[threadIdx.x] = sum;
  __syncthreads();
  for (int n = p.lanes / 2; n; n /= 2) {  // in halves: the order of the sums does not depend on the launch
    if (g0 < n) {
      const int with = threadIdx.x + n * per;
      ExpSum a = {part[threadIdx.x].x, part[threadIdx.x].y};
      const float2 g[1] = {part[with]};
      add_groups(a, g);
      part[threadIdx.x] = make_float2(a.r, a.s);
      part_sum[threadIdx.x] += part_sum[with];
    }
    __syncthreads();
  }
  if (g0 || i >= rows) return;
  if (!p.index) {
    const int64_t t = p.targets[i * p.step];
    if (t < 0 || t >= p.V || t == p.ignore) {
      p.loss[to] = p.lse[to] = t == p.ignore ? 0.f : __int_as_float(0x7FC00000);
      return;
    }
  }
  // the difference of two numbers near one another, in 64 bits
  const float2 f = part[r];
  const double lse = ((double)f.x + log2f(f.y)) * 0.69314718055994530942;
  double loss = lse - (1.0 - p.smoothing) * at_target;
  if (p.z > 0.f) loss += p.z * lse * lse;  // (0 times infinity would be none)
  if (p.sums) loss -= p.smoothing / (double)p.V * part_sum[r];
  p.loss[to] = (float)loss;
  p.lse[to] = (float)lse;
}

// ------------------------------------------------------------------------------------------------
// Host side
// ------------------------------------------------------------------------------------------------
// Bytes of slopes that a piece of the vocabulary may have, and its least columns.
constexpr long long kPieceBytes = 512ll << 20;
constexpr int kPieceLeast = 4096;

struct Sizes {
  bool few, dot, odd;      // odd: few rows whose products read W off 16-byte boundaries
  long long ldx, ldw;      // rows of x and w, as given
  long long ldxc, ldd, ldacc;
  int groups, pieces, piece;
  Split all;               // of dx: the device's choice
  size_t sums_bytes;
  size_t head, row_sums, index, target, coef, at, stats, logit_sums, partial, x, w, slope, acc, total;
};

static int sizes(const psr_xent_shape* sh, bool backward, Sizes& s) {
  if (!sh || sh->M < 0 || sh->V < 1 || sh->K < 1) return PSR_ERR_ARG;
  if (sh->type != PSR_BF16 && sh->type != PSR_F16) return PSR_ERR_ARG;
  if (sh->odd < 0 || sh->odd > 3) return PSR_ERR_ARG;
  if (!(sh->smoothing >= 0.f && sh->smoothing < 1.f) || !(sh->z_weight >= 0.f && sh->z_weight <= FLT_MAX)) return PSR_ERR_ARG;
  if (sh->M > 1 << 24 || sh->V > 1 << 28 || sh->K > 1 << 20) return PSR_ERR_UNSUPPORTED;
  s.ldx = sh->ldx ? sh->ldx : sh->K;
  s.ldw = sh->ldw ? sh->ldw : sh->K;
  if (s.ldx < sh->K || s.ldw < sh->K) return PSR_ERR_ARG;
  const bool odd_x = (sh->odd & PSR_LINEAR_ODD_X) || (sh->M > 1 && s.ldx % 8), odd_w = (sh->odd & PSR_LINEAR_ODD_W) || (sh->V > 1 && s.ldw % 8);
  const long long M = sh->M, V = sh->V, K = sh->K, Mk = (M + kBK - 1) / kBK * kBK;
  s.few = M <= kFew;
  s.dot = !backward && M == 1 && !odd_x && !odd_w && K % 8 == 0;
  s.ldxc = (K + 63) / 64 * 64;  // (rows on 128-byte boundaries: the tile loads take half as long again from others)
  size_t off = 256;
  auto take = [&](bool want, long long bytes) {
    const size_t at = off;
    if (!want) return (size_t)0;
    off = (off + (size_t)bytes + 255) / 256 * 256;
    return at;
  };
  s.head = take(true, 256);
  s.row_sums = take(M > kScanMost, (M + 255) / 256 * 16);
  s.index = take(!s.few, M * 4);
  s.target = take(!s.few || backward, M * 4);
  s.coef = take(backward, M * 16);
  s.at = take(!backward, M * 4);
  s.groups = s.dot ? kDotBlocks * kStreamCtas : (int)(s.few ? (V + 31) / 32 : (V + kGroup - 1) / kGroup);
  s.stats = take(!backward, M * s.groups * 8);
  s.logit_sums = take(!backward && sh->smoothing > 0.f, M * s.groups * 4);
  // packed rows, or (up to kFew rows) those that count beside zeros; the products of a forward pass of few rows read x itself
  s.x = take(!s.few || backward || odd_x, Mk * s.ldxc * 2);
  s.odd = s.few && odd_w;
  s.w = take(odd_w && !s.few, V * ((K + 7) / 8 * 8) * 2);
  s.pieces = 1;
  s.piece = (int)V;
  s.sums_bytes = s.few && !s.dot ? partial_bytes((int)M, (int)V, (int)K, false) : 0;
  s.all = {((M + 255) / 256) * ((K + 255) / 256), 0, 1, 0.0};
  if (backward) {
    if (!s.few) {
      const long long most = std::max((long long)kPieceLeast, kPieceBytes / (2 * Mk) / 512 * 512);
      s.pieces = (int)((V + most - 1) / most);
      if (s.pieces > 1) s.piece = (int)(((V + s.pieces - 1) / s.pieces + 511) / 512 * 512);
      s.pieces = (int)((V + s.piece - 1) / s.piece);
      s.sums_bytes = (size_t)kPairs * 65536 * 4;  // parts of split tiles of dx: no more than pairs
    } else {
      s.sums_bytes = std::max(s.sums_bytes, partial_bytes((int)M, (int)K, (int)V, false));
    }
    s.ldd = (s.piece + 63ll) / 64 * 64;
    s.slope = take(true, Mk * s.ldd * 2);
    s.ldacc = (K + 7) / 8 * 8;
    s.acc = take(s.pieces > 1, M * s.ldacc * 4);
  }
  s.partial = take(true, (long long)s.sums_bytes);
  s.total = off;
  return PSR_OK;
}

static int launch_of(void* workspace, const Sizes& s, int timeout_ms, void* stream, Launch& l) {
  const int rc = check_device(&l.n_sm);
  if (rc != PSR_OK) return rc;
  if (cudaGetDevice(&l.dev) != cudaSuccess) return PSR_ERR_CUDA;
  l.ctrl = l.clear = static_cast<Ctrl*>(workspace);
  l.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + s.partial);
  l.partial_bytes = s.sums_bytes;
  l.timeout_ns = (unsigned long long)(timeout_ms > 0 ? timeout_ms : 2000) * 1000000ull;
  l.st = static_cast<cudaStream_t>(stream);
  return PSR_OK;
}

template <class T>
static T* in(void* workspace, size_t at) { return at ? reinterpret_cast<T*>(static_cast<uint8_t*>(workspace) + at) : nullptr; }

static int launch_rows(const psr_xent_shape* sh, const Sizes& s, RowParams& p, bool backward, const void* x, const int64_t* targets,
                       void* ws, Launch& l) {
  p.x = static_cast<const uint16_t*>(x);
  p.ldx = s.ldx;
  p.xc = in<uint16_t>(ws, s.x);
  p.ldxc = s.ldxc;
  p.M = sh->M;
  p.V = sh->V;
  p.K = sh->K;
  p.vec = sh->K % 8 == 0 && aligned_to(x, 16) && (sh->M == 1 || s.ldx % 8 == 0);
  p.per = sh->M > kScanMost ? 256 : std::max(8, (sh->M + 1023) / 1024);
  p.sums = in<float4>(ws, s.row_sums);
  p.packed = !s.few;
  p.targets = targets;
  p.step = sh->targets_step;
  p.ignore = sh->ignore;
  p.count = in<int>(ws, s.head);
  p.unit = in<float>(ws, s.head) + 1;
  p.index = in<int>(ws, s.index);
  p.target = in<int>(ws, s.target);
  p.coef = in<float4>(ws, s.coef);
  p.smoothing = sh->smoothing;
  p.z = sh->z_weight;
  p.half = sh->type == PSR_F16;
  p.clear = l.clear;
  const unsigned grid = (unsigned)((sh->M + p.per - 1) / p.per);
  if (p.sums) {
    if (backward) block_kernel<true><<<grid, 256, 0, l.st>>>(p);
    else block_kernel<false><<<grid, 256, 0, l.st>>>(p);
    p.clear = l.clear = nullptr;
    const int rc = launch_status();
    if (rc != PSR_OK) return rc;
  }
  if (backward) rows_kernel<true><<<grid, 256, 0, l.st>>>(p);
  else rows_kernel<false><<<grid, 256, 0, l.st>>>(p);
  l.clear = nullptr;
  return launch_status();
}

static int forward(const psr_xent_shape* sh, const Sizes& s, const void* x, const void* w, const int64_t* targets, float* loss,
                   float* lse, void* ws, Launch& l) {
  int rc = PSR_OK;
  Head h = {};
  h.stats = in<float2>(ws, s.stats);
  h.sums = in<float>(ws, s.logit_sums);
  h.at = in<float>(ws, s.at);
  h.group_at = s.few ? 1 : sh->M;
  h.row_at = s.few ? s.groups : 1;
  FinishParams f = {};
  f.groups = s.groups;
  long long ldx = s.ldx, ldw = s.ldw;
  Epilogue e = {};
  e.half = sh->type == PSR_F16;
  if (s.dot) {
    DotParams p = {x, w, s.ldw, sh->V, sh->K, targets, h.stats, h.sums, h.at, l.clear};
    const int blocks = std::min(kDotBlocks * std::min(l.n_sm, kStreamCtas), (sh->V + kDotThreads / 32 - 1) / (kDotThreads / 32));
    if (e.half) dot_kernel<__half><<<blocks, kDotThreads, 0, l.st>>>(p);
    else dot_kernel<__nv_bfloat16><<<blocks, kDotThreads, 0, l.st>>>(p);
    l.clear = nullptr;
    f.groups = blocks;
    rc = launch_status();
  } else if (s.few) {
    if ((rc = align(x, ldx, s.x, sh->M, sh->K, ws, l)) != PSR_OK) return rc;
    h.ids = targets;
    h.step = sh->targets_step;
    const Operands o = {x, ldx, w, ldw, sh->M, sh->V, sh->K};
    rc = s.odd ? launch_stream<false, kStats, true>(o, e, l, h) : launch_stream<false, kStats>(o, e, l, h);
  } else {
    RowParams p = {};
    p.loss = loss;
    p.lse = lse;
    if ((rc = launch_rows(sh, s, p, false, x, targets, ws, l)) != PSR_OK) return rc;
    if ((rc = align(w, ldw, s.w, sh->V, sh->K, ws, l)) != PSR_OK) return rc;
    h.rows = f.count = p.count;
    f.index = p.index;
    h.target = p.target;
    const Operands o = {p.xc, p.ldxc, w, ldw, sh->M, sh->V, sh->K};
    const Split whole = {((sh->M + 255ll) / 256) * ((sh->V + 255ll) / 256), 0, 1, 0.0};
    rc = launch_pair<false, false, false, kStats>(o, e, false, whole, l, h);
  }
  if (rc != PSR_OK) return rc;
  f.stats = h.stats;
  f.sums = h.sums;
  f.group_at = h.group_at;
  f.row_at = h.row_at;
  f.at = h.at;
  f.targets = targets;
  f.step = sh->targets_step;
  f.ignore = sh->ignore;
  f.M = sh->M;
  f.V = sh->V;
  f.smoothing = sh->smoothing;
  f.z = sh->z_weight;
  f.loss = loss;
  f.lse = lse;
  f.lanes = s.few ? 256 : 32;
  const int per = 256 / f.lanes;
  return launch_after(finish_kernel, dim3((unsigned)((sh->M + per - 1) / per)), 256, f, l.st);
}

template <bool HALF>
static int backward(const psr_xent_shape* sh, const Sizes& s, const float* dloss, const void* x, const void* w, const int64_t* targets,
                    const float* lse, void* dx, void* dw, void* ws, Launch& l) {
  RowParams p = {};
  p.dloss = dloss;
  p.dstep = sh->dloss_step;
  p.lse_in = lse;
  p.dx = static_cast<uint16_t*>(dx);
  int rc = launch_rows(sh, s, p, true, x, targets, ws, l);
  if (rc != PSR_OK) return rc;
  long long ldw = s.ldw;
  if ((rc = align(w, ldw, s.w, sh->V, sh->K, ws, l)) != PSR_OK) return rc;
  const int M = sh->M, K = sh->K;
  void* slope = in<uint8_t>(ws, s.slope);
  const bool flat = K % 8 == 0;
  for (int at = 0; at < sh->V; at += s.piece) {
    const int n = std::min(s.piece, sh->V - at);
    const uint16_t* wp = static_cast<const uint16_t*>(w) + at * ldw;
    Head h = {};
    h.rows = s.few ? nullptr : p.count;
    h.index = p.index;
    h.target = p.target;
    h.col0 = at;
    h.coef = p.coef;
    h.acc = in<float>(ws, s.acc);
    h.ldacc = s.ldacc;
    h.first = at == 0;
    h.last = at + n == sh->V;
    h.unit = p.unit;
    Epilogue e = {};
    e.half = HALF;
    e.y = slope;
    e.ldy = s.ldd;
    e.vec = 1;  // (rows of a multiple of eight elements: the last chunk may go past the piece's columns)
    const Operands logits = {p.xc, p.ldxc, wp, ldw, M, n, K};
    const Split whole = {((M + 255ll) / 256) * ((n + 255ll) / 256), 0, 1, 0.0};
    if (s.odd) rc = launch_stream<false, kSlope, true>(logits, e, l, h);
    else if (s.few) rc = launch_stream<false, kSlope>(logits, e, l, h);
    else rc = launch_pair<false, false, HALF, kSlope>(logits, e, false, whole, l, h);
    if (rc != PSR_OK) return rc;
    e.ldy = K;
    if (dx) {  // before dw, which takes W's place in L2
      e.y = dx;
      e.vec = flat && aligned_to(dx, 16);
      const Operands o = {slope, s.ldd, wp, ldw, M, K, n};
      if (s.odd) rc = launch_stream<true, kSum, true>(o, e, l, h);
      else if (s.few) rc = launch_stream<true, kSum>(o, e, l, h);
      else rc = launch_pair<false, true, HALF, kSum>(o, e, false, s.all, l, h);
      if (rc != PSR_OK) return rc;
    }
    if (dw) {
      uint16_t* to = static_cast<uint16_t*>(dw) + (long long)at * K;
      e.y = to;
      e.vec = flat && aligned_to(to, 16);
      const Operands o = {slope, s.ldd, p.xc, p.ldxc, n, K, M};
      const Split all = {((n + 255ll) / 256) * ((K + 255ll) / 256), 0, 1, 0.0};
      rc = launch_pair<true, true, HALF, kWeight>(o, e, wide_tiles<true, true>(o, 0.0, all, l.n_sm / 2), all, l, h);
      if (rc != PSR_OK) return rc;
    }
  }
  return PSR_OK;
}

}  // namespace xent
}  // namespace psr

using namespace psr;
using namespace psr::xent;

extern "C" {

size_t psr_xent_workspace_bytes(const psr_xent_shape* sh, int backward) {
  Sizes s;
  return xent::sizes(sh, backward != 0, s) == PSR_OK ? s.total : 0;
}

static int xent_arguments(const psr_xent_shape* sh, const Sizes& s, const void* x, const void* w, const int64_t* targets,
                          const void* workspace, size_t ws_bytes) {
  if (!x || !w || !targets || !workspace) return PSR_ERR_ARG;
  if (!aligned_to(x, 2) || !aligned_to(w, 2) || !aligned_to(targets, 8) || !aligned_to(workspace, 256)) return PSR_ERR_ARG;
  // operands that are read where they are start on 16-byte boundaries
  if ((!s.x && !aligned_to(x, 16)) || (!s.w && !s.odd && !aligned_to(w, 16))) return PSR_ERR_ARG;
  return ws_bytes < s.total ? PSR_ERR_ARG : PSR_OK;
}

int psr_xent(const psr_xent_shape* sh, const void* x, const void* w, const int64_t* targets, float* loss, float* lse, void* workspace,
             size_t ws_bytes, int timeout_ms, void* stream) {
  Sizes s;
  int rc = xent::sizes(sh, false, s);
  if (rc != PSR_OK) return rc;
  if (sh->M == 0) return check_device(nullptr);
  if ((rc = xent_arguments(sh, s, x, w, targets, workspace, ws_bytes)) != PSR_OK) return rc;
  if (!loss || !lse || !aligned_to(loss, 4) || !aligned_to(lse, 4)) return PSR_ERR_ARG;
  Launch l;
  if ((rc = xent::launch_of(workspace, s, timeout_ms, stream, l)) != PSR_OK) return rc;
  return forward(sh, s, x, w, targets, loss, lse, workspace, l);
}

int psr_xent_bwd(const psr_xent_shape* sh, const float* dloss, const void* x, const void* w, const int64_t* targets, const float* lse,
                 void* dx, void* dw, void* workspace, size_t ws_bytes, int timeout_ms, void* stream) {
  Sizes s;
  int rc = xent::sizes(sh, true, s);
  if (rc != PSR_OK) return rc;
  if (!aligned_to(dx, 2) || !aligned_to(dw, 2)) return PSR_ERR_ARG;
  if (sh->M == 0) {  // sums over no rows
    if ((rc = check_device(nullptr)) != PSR_OK || !dw) return rc;
    if (cudaMemsetAsync(dw, 0, (size_t)sh->V * sh->K * 2, static_cast<cudaStream_t>(stream)) == cudaSuccess) return PSR_OK;
    cudaGetLastError();
    return PSR_ERR_CUDA;
  }
  if ((rc = xent_arguments(sh, s, x, w, targets, workspace, ws_bytes)) != PSR_OK) return rc;
  if (!dloss || !lse || !aligned_to(dloss, 4) || !aligned_to(lse, 4)) return PSR_ERR_ARG;
  if (!dx && !dw) return check_device(nullptr);
  Launch l;
  if ((rc = xent::launch_of(workspace, s, timeout_ms, stream, l)) != PSR_OK) return rc;
  return sh->type == PSR_F16 ? xent::backward<true>(sh, s, dloss, x, w, targets, lse, dx, dw, workspace, l)
                             : xent::backward<false>(sh, s, dloss, x, w, targets, lse, dx, dw, workspace, l);
}

}  // extern "C"
