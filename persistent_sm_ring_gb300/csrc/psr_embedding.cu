// The embedding on sm_103a: rows of a table looked up by token and scaled, and the table's gradient.
//
// Forward: y_i = scale w[id_i].  Backward: dw_v = scale sum of dy_i over the i with id_i = v, with fp32 sums in an order that the
// tokens alone decide: they are sorted by id (stable), blocks of sorted positions are summed one after another, and the blocks' sums of a
// run of equal ids over more than two of them are added in eight interleaved series, then those.  No result depends on the order in which
// blocks run.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "psr_control.cuh"
#include "psr_device.cuh"
#include "psr_host.h"

namespace psr {
namespace embedding {

// E adjacent elements of a row
template <class T, int E>
struct alignas(sizeof(T) * E) Vec { T v[E]; };

// The same as words, two elements of 16 bits to each.
template <class T, int E>
using Raw = std::conditional_t<sizeof(T) * E % 4 == 0, Vec<uint32_t, (sizeof(T) * E + 3) / 4>, Vec<uint16_t, 1>>;
template <class T, int E>
__device__ __forceinline__ void add_to(float* acc, const Raw<T, E>& x) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += __uint_as_float(x.v[e]);
  } else if constexpr (E == 1) {
    T v;
    memcpy(&v, &x.v[0], 2);
    acc[0] += to_f32(v);
  } else {
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      if constexpr (std::is_same<T, __half>::value) {
        __half2 h;
        memcpy(&h, &x.v[e], 4);
        const float2 f = __half22float2(h);
        acc[2 * e] += f.x;
        acc[2 * e + 1] += f.y;
      } else {
        acc[2 * e] += __uint_as_float(x.v[e] << 16);
        acc[2 * e + 1] += __uint_as_float(x.v[e] & 0xFFFF0000u);
      }
    }
  }
}

// ------------------------------------------------------------------------------------------------
// Lookup
// ------------------------------------------------------------------------------------------------
// Memory bound.  A warp takes 32 * kAhead vectors of a row, all of them in flight at once (16421 tokens of 4096 bf16 columns from
// 128000 rows: 33 us, 5.8 TB/s; two vectors 35, eight 34; 32 tokens of 8192: 4 us).
constexpr int kAhead = 4;

template <class T, int E>
__global__ void __launch_bounds__(256)
    lookup_kernel(const int64_t* __restrict__ ids, long long step, const T* __restrict__ w, long long ldw, T* __restrict__ y,
                  long long ldy, int M, int V, int K, int pieces, float scale) {
  const long long item = blockIdx.x * 8ll + threadIdx.x / 32;
  const long long row = item / pieces;
  if (row >= M) return;
  const int k0 = (int)(item - row * pieces) * 32 * E * kAhead + threadIdx.x % 32 * E;
  const long long id = ids[row * step];
  const bool ok = id >= 0 && id < V;
  const T* src = w + (ok ? id : 0) * ldw;
  T* dst = y + row * ldy;
  Vec<T, E> x[kAhead];
#pragma unroll
  for (int a = 0; a < kAhead; ++a) {
    const int k = k0 + a * 32 * E;
    if (ok && k < K) x[a] = *reinterpret_cast<const Vec<T, E>*>(src + k);
  }
#pragma unroll
  for (int a = 0; a < kAhead; ++a) {
    const int k = k0 + a * 32 * E;
    if (k >= K) break;
#pragma unroll
    for (int e = 0; e < E; ++e) x[a].v[e] = from_f32<T>(ok ? to_f32(x[a].v[e]) * scale : __int_as_float(0x7FC00000));
    if constexpr (sizeof(Vec<T, E>) == 16) {
      uint4 q;
      memcpy(&q, &x[a], 16);
      __stcs(reinterpret_cast<uint4*>(dst + k), q);
    } else {
      *reinterpret_cast<Vec<T, E>*>(dst + k) = x[a];
    }
  }
}

// ------------------------------------------------------------------------------------------------
// Sort of the tokens by id
// ------------------------------------------------------------------------------------------------
// A cluster of CTAs sorts (id, position) pairs by up to nine bits a pass, least significant first.  Each warp has a
// contiguous share of the pairs and counts its digits; the counts before it (of smaller digits, of earlier CTAs and warps) are
// where its pairs go, equal digits in their order: of 32 pairs, a word of shared memory for each digit gathers the lanes that have it
// (with match.any 65539 tokens took 5 us longer).  Ids outside the table, and the padding id, become V: they end up behind all
// others.  One kernel, so that the next one's zeros begin with it: 9 us for 2049 tokens, 13 for 16384 (two passes), 13 for 65539 of
// 260 ids (one), bound by the latencies of its rounds: pairs brought into order in shared memory before they are stored, or more of them
// in flight, are no faster.  Separate kernels over all SMs took 12 for 65539, but of several kernels in a row only one begins early: 16384
// tokens into 128000 rows took 285 us where the cluster, before there were as many zero writers, took 244.
constexpr int kSortCtas = 8, kSortThreads = 1024, kSortWarps = kSortThreads / 32, kSortBits = 9, kBins = 1 << kSortBits;

struct Tokens {
  const int64_t* ids;
  long long step;
  long long padding;  // an id without gradient (negative: none)
  int M, V;
};

struct SortParams {
  Tokens t;
  uint2* a;        // the sorted pairs (key, position)
  uint2* b;        // space for them between passes
  int* n_long;     // set to zero for the sums
  int passes, bits;
  Ctrl* clear;
};

struct SortSmem {
  uint32_t hist[kSortWarps][kBins];
  uint32_t lanes[kSortWarps][kBins];  // of a warp's 32 pairs, those with each digit
  uint32_t total[kBins];  // of this CTA, by digit; read by the others
  uint32_t base[kBins];
  uint32_t warp_sum[kSortWarps];
};

__device__ __forceinline__ uint32_t key_of(const Tokens& t, long long i) {
  const long long id = t.ids[i * t.step];
  return id >= 0 && id < t.V && id != t.padding ? (uint32_t)id : (uint32_t)t.V;
}

__global__ void __launch_bounds__(kSortThreads, 1) sort_kernel(const __grid_constant__ SortParams p) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  SortSmem& sm = *reinterpret_cast<SortSmem*>(smem_raw);
  clear_ctrl(p.clear);
  launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.n_long = 0;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank(), ctas = kSortCtas;
  const long long share = (((long long)p.t.M + ctas * kSortWarps - 1) / (ctas * kSortWarps) + 31) / 32 * 32;
  const long long i0 = ((long long)rank * kSortWarps + warp) * share;
  const long long i1 = min((long long)p.t.M, i0 + share);
  const uint32_t bins = 1u << p.bits;
  constexpr int kRounds = 4;  // pairs of a lane in flight
  for (int pass = 0; pass < p.passes; ++pass) {
    const uint2* src = (p.passes - pass) % 2 ? p.b : p.a;  // the last pass writes a
    uint2* dst = (p.passes - pass) % 2 ? p.a : p.b;
    const int shift = pass * p.bits;
    for (uint32_t d = lane; d < bins; d += 32) sm.hist[warp][d] = sm.lanes[warp][d] = 0;
    __syncwarp();
    // calls f(whether there is a pair, the pair, its digit) for the warp's pairs, 32 at a time in order
    auto each = [&](auto f) {
      for (long long i = i0; i < i1; i += 32 * kRounds) {
        uint2 x[kRounds];
#pragma unroll
        for (int j = 0; j < kRounds; ++j) {
          const long long at = i + 32 * j + lane;
          x[j] = make_uint2(0, 0);
          if (at < i1) x[j] = pass == 0 ? make_uint2(key_of(p.t, at), (uint32_t)at) : src[at];
        }
#pragma unroll
        for (int j = 0; j < kRounds; ++j) {
          if (i + 32 * j >= i1) break;
          const bool in = i + 32 * j + lane < i1;
          f(in, x[j], in ? x[j].x >> shift & (bins - 1) : bins);
        }
      }
    };
    each([&](bool in, uint2, uint32_t d) {
      if (in) atomicAdd(&sm.hist[warp][d], 1u);
    });
    __syncthreads();
    uint32_t total = 0;
    if (threadIdx.x < bins) {
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t n = sm.hist[w][threadIdx.x];
        sm.hist[w][threadIdx.x] = total;
        total += n;
      }
      sm.total[threadIdx.x] = total;
    }
    cluster_sync();
    // pairs with smaller digits, and those with this one in earlier CTAs
    uint32_t all = 0, before = 0;
    if (threadIdx.x < bins) {
#pragma unroll
      for (uint32_t c = 0; c < ctas; ++c) {
        const uint32_t n = ld_shared_cluster(mapa_shared(smem_u32(&sm.total[threadIdx.x]), c));
        if (c < rank) before += n;
        all += n;
      }
    }
    uint32_t sum = all;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t n = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += n;
    }
    if (lane == 31) sm.warp_sum[warp] = sum;
    __syncthreads();
    if (threadIdx.x < bins) {
      uint32_t base = sum - all + before;
#pragma unroll
      for (int w = 0; w < kBins / 32; ++w)
        if (w < warp) base += sm.warp_sum[w];
      sm.base[threadIdx.x] = base;
    }
    __syncthreads();
    each([&](bool in, uint2 x, uint32_t d) {
      if (in) atomicOr(&sm.lanes[warp][d], 1u << lane);
      __syncwarp();
      uint32_t same = 0, n = 0;
      if (in) {
        same = sm.lanes[warp][d];
        n = sm.hist[warp][d];
        dst[sm.base[d] + n + __popc(same & ((1u << lane) - 1))] = x;
      }
      __syncwarp();
      if (in && lane == __ffs(same) - 1) {
        sm.hist[warp][d] = n + __popc(same);
        sm.lanes[warp][d] = 0;
      }
      __syncwarp();
    });
    cluster_sync();  // the next pass, or the CTAs' ends: all pairs are in place, all totals read
  }
}

// Few tokens: each finds its place by comparing itself with all others, (id, position) as one number, four threads to a token.  No
// passes and no exchange between blocks: 5 us for 2047 tokens, where the cluster takes 10 (the whole call with 1000 rows of 512 columns
// 9.8 and 13.6 us, with 10 tokens 4.3 and 9.3).  The comparisons grow as M^2, and beyond kRankMost the keys do not fit in 32 bits.
constexpr int kRankBits = 11, kRankMost = 1 << kRankBits, kRankTokens = 64;  // tokens of a block

__global__ void __launch_bounds__(4 * kRankTokens) rank_kernel(const __grid_constant__ SortParams p) {
  __shared__ __align__(16) uint32_t keys[kRankMost];
  clear_ctrl(p.clear);
  launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.n_long = 0;
  const int M = p.t.M, padded = (M + 15) / 16 * 16;
#pragma unroll 8
  for (int i = threadIdx.x; i < padded; i += 4 * kRankTokens) keys[i] = i < M ? key_of(p.t, i) << kRankBits | (uint32_t)i : 0xffffffffu;
  __syncthreads();
  const int token = blockIdx.x * kRankTokens + threadIdx.x / 4;
  const uint32_t own = token < M ? keys[token] : 0;
  int rank = 0;
#pragma unroll 4
  for (int i = threadIdx.x % 4 * 4; i < padded; i += 16) {
    const uint4 k = *reinterpret_cast<const uint4*>(keys + i);
    rank += (k.x < own) + (k.y < own) + (k.z < own) + (k.w < own);
  }
  rank += __shfl_xor_sync(0xffffffffu, rank, 1);
  rank += __shfl_xor_sync(0xffffffffu, rank, 2);
  if (token < M && threadIdx.x % 4 == 0) p.a[rank] = make_uint2(own >> kRankBits, (uint32_t)token);
}

// ------------------------------------------------------------------------------------------------
// Zeros for the rows that no token names
// ------------------------------------------------------------------------------------------------
// Memory bound.  CTAs of their own write the zeros by bulk copies, beside the sort and the sums, and mark the ids among their rows first.
// Three to an SM, as many as fit: 16384 tokens into 128000 rows of 4096 in 188 us (1.18 GB at 6.3 TB/s), with two 215, with one 244 (a fill of
// the library's writes 4.0 TB/s).  Each has every n-th 32 rows, so that what all write at a time lies together; nothing reads the zeros soon,
// so they are the first to leave L2 (2047 tokens into 50021 rows of 1736: 36.7 us instead of 39).
constexpr int kZeroCtas = 3;
constexpr int kZeroBytes = 8192;  // what one copy of zeros writes
constexpr int kMarks = 32768;     // rows that a CTA marks at a time
struct ZeroSmem {
  uint4 zeros[kZeroBytes / 16];
  uint32_t marks[kMarks / 32];
};

// `n` bytes of zeros (an even number, from an even address) by a warp; odd ends by hand.
__device__ __forceinline__ void zero_bytes(uint8_t* at, long long n, uint32_t zeros, uint64_t policy) {
  const int lane = threadIdx.x % 32;
  long long head = (16 - (long long)(reinterpret_cast<uintptr_t>(at) % 16)) % 16;
  if (head > n) head = n;
  if (2 * lane < head) *reinterpret_cast<uint16_t*>(at + 2 * lane) = 0;
  const long long body = (n - head) / 16 * 16, tail = n - head - body;
  for (long long i = lane * (long long)kZeroBytes; i < body; i += 32ll * kZeroBytes)
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group.L2::cache_hint [%0], [%1], %2, %3;" ::"l"(at + head + i), "r"(zeros),
                 "r"((uint32_t)min((long long)kZeroBytes, body - i)), "l"(policy)
                 : "memory");
  if (2 * lane < tail) *reinterpret_cast<uint16_t*>(at + n - tail + 2 * lane) = 0;
}

__device__ void zero_rows(const Tokens& t, uint8_t* dw, long long row_bytes, uint32_t cta, uint32_t n_cta, ZeroSmem& sm) {
  const uint32_t words = ((uint32_t)t.V + 31) / 32, own = cta < words ? (words - cta + n_cta - 1) / n_cta : 0;
  const uint32_t zeros = smem_u32(sm.zeros);
  for (int i = threadIdx.x; i < kZeroBytes / 16; i += 256) sm.zeros[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  uint64_t policy;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  for (uint32_t w0 = 0; w0 < own; w0 += kMarks / 32) {
    const uint32_t n = min(own - w0, (uint32_t)kMarks / 32);
    for (uint32_t i = threadIdx.x; i < n; i += 256) sm.marks[i] = 0;
    __syncthreads();
#pragma unroll 8
    for (long long i = threadIdx.x; i < t.M; i += 256) {
      const uint32_t id = key_of(t, i), q = id / 32 / n_cta, w = q - w0, bit = 1u << (id % 32);
      if (id / 32 - q * n_cta == cta && w < n && !(*(volatile uint32_t*)&sm.marks[w] & bit)) atomicOr(&sm.marks[w], bit);
    }
    __syncthreads();
    for (uint32_t w = threadIdx.x / 32; w < n; w += 8) {  // runs of rows without a mark
      const long long v = 32ll * ((w0 + w) * n_cta + cta);
      const int rows = (int)min(32ll, t.V - v);
      uint32_t left = ~sm.marks[w] & (rows == 32 ? 0xffffffffu : (1u << rows) - 1);
      while (left) {
        const int first = __ffs(left) - 1;
        const uint32_t rest = ~(left >> first);
        const int run = rest ? __ffs(rest) - 1 : 32;
        zero_bytes(dw + (v + first) * row_bytes, run * row_bytes, zeros, policy);
        left = first + run == 32 ? 0 : left >> (first + run) << (first + run);
      }
    }
    __syncthreads();
  }
  bulk_commit();
  bulk_wait<0>();
}

// ------------------------------------------------------------------------------------------------
// Sums of the rows of each id
// ------------------------------------------------------------------------------------------------
// Memory bound: 65539 rows of 1001 fp32 columns in 54 us (4.9 TB/s; rows off 16-byte boundaries, 128 bytes to a load), 16384 rows of 4096
// with the zeros of 128000 in 177 (6.7 TB/s).  A warp takes a block of sorted positions and 32 * E * U columns, reads R rows at a time and
// writes a row of dw where the id changes.  A run of equal ids that crosses one border between blocks belongs to the block where it
// begins.  A longer one is long: each of its blocks leaves its sum in a partial row of its own (the one where it begins in its second,
// the others in their first), and join_kernel adds them up.
constexpr int kBlockMost = 64;  // positions of a block

struct SumParams {
  const uint2* sorted;
  const void* dy;
  long long lddy;
  void* dw;
  float* partial;  // [blocks][2][K]
  int* n_long;     // long runs: the blocks where they begin, and their ids
  int2* longs;
  int M, V, K, block, blocks, pieces;
  int accumulate;
  int zero_ctas;   // the grid's first CTAs write zeros
  Tokens t;
  float scale;
};

template <class T, int E>
__device__ __forceinline__ void put_row(const SumParams& p, uint32_t id, int k, const float* acc) {
  Vec<T, E>* at = reinterpret_cast<Vec<T, E>*>(static_cast<T*>(p.dw) + (long long)id * p.K + k);
  Vec<T, E> v;
  if (p.accumulate) v = *at;
#pragma unroll
  for (int e = 0; e < E; ++e) v.v[e] = from_f32<T>(p.accumulate ? fmaf(acc[e], p.scale, to_f32(v.v[e])) : acc[e] * p.scale);
  *at = v;
}

template <class T, int E, int U>
__global__ void __launch_bounds__(256, E >= 4 ? 3 : 4) sum_kernel(const __grid_constant__ SumParams p) {
  constexpr int R = 4;
  __shared__ union {
    ZeroSmem zero;
    uint32_t order[8][2 * kBlockMost];
  } sm;
  if ((int)blockIdx.x < p.zero_ctas) {  // nothing here waits for the sort
    zero_rows(p.t, static_cast<uint8_t*>(p.dw), p.K * (long long)sizeof(T), blockIdx.x, p.zero_ctas, sm.zero);
    wait_previous();
    return;
  }
  const long long item = (blockIdx.x - p.zero_ctas) * 8ll + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const int blk = (int)(item / p.pieces), piece = (int)(item - (long long)blk * p.pieces);
  wait_previous();
  if (blk >= p.blocks) return;
  const uint32_t V = (uint32_t)p.V, none = 0xffffffffu, all = 0xffffffffu;
  const long long i0 = (long long)blk * p.block;
  const int n = (int)min((long long)p.block, p.M - i0);
  const uint2* s = p.sorted + i0;
  auto key_at = [&](long long r) { return i0 + r >= 0 && i0 + r < p.M ? s[r].x : none; };  // of any position
  uint2 lo = make_uint2(none, 0), hi = lo, lo2 = lo, hi2 = lo;  // the block's pairs, and those behind it
  if (lane < n) lo = s[lane];
  if (lane + 32 < n) hi = s[lane + 32];
  if (n == p.block) {
    if (lane < p.block && i0 + n + lane < p.M) lo2 = s[n + lane];
    if (lane + 32 < p.block && i0 + n + lane + 32 < p.M) hi2 = s[n + lane + 32];
  }
  const uint32_t before = key_at(-1), past = key_at(2ll * p.block), older = key_at(-1ll - p.block);
  const uint32_t first = __shfl_sync(all, lo.x, 0), last = __shfl_sync(all, n <= 32 ? lo.x : hi.x, (n - 1) % 32);
  const uint32_t next = __shfl_sync(all, lo2.x, 0);
  // positions whose id is the first's, the last's, one of the table's
  auto mask = [&](uint32_t a, uint32_t b) { return (unsigned long long)a | (unsigned long long)b << 32; };
  auto count = [](unsigned long long m) { return m == ~0ull ? 64 : __ffsll((long long)~m) - 1; };  // ones at the low end
  const int named = count(mask(__ballot_sync(all, lo.x < V), __ballot_sync(all, hi.x < V)));
  int begin = 0, end = named;
  int head = 0;  // positions of a long run that began earlier
  if (before == first && first < V) {
    const int run = count(mask(__ballot_sync(all, lo.x == first), __ballot_sync(all, hi.x == first)));
    if (older != first && (run < n || next != first)) begin = run;  // the last block's
    else head = run;
  }
  int tail = n;  // position where a long run begins that goes on
  if (named == n && next == last && head < n) {
    if (past == last) {
      const int same = 64 - __clzll((long long)~(mask(__ballot_sync(all, lo.x == last), __ballot_sync(all, hi.x == last)) << (64 - n)));
      tail = same - (64 - n);
      if (lane == 0 && piece == 0) p.longs[atomicAdd(p.n_long, 1)] = make_int2(blk, (int)last);
    } else {
      end = n + count(mask(__ballot_sync(all, lo2.x == last), __ballot_sync(all, hi2.x == last)));
    }
  }
  // where the id changes; the rows' positions in shared memory, from where four at a time come
  const uint32_t up_lo = __shfl_down_sync(all, lo.x, 1), up_hi = __shfl_down_sync(all, hi.x, 1), mid = __shfl_sync(all, hi.x, 0);
  const uint32_t to_lo = lane == 31 ? mid : up_lo, to_hi = lane == 31 ? next : up_hi;
  const unsigned long long changes = mask(__ballot_sync(all, lo.x != (lane == n - 1 ? next : to_lo)),
                                          __ballot_sync(all, hi.x != (lane + 32 == n - 1 ? next : to_hi)));
  uint32_t* rows = sm.order[threadIdx.x / 32];
  if (lane < n) rows[lane] = lo.y;
  if (lane + 32 < n) rows[lane + 32] = hi.y;
  if (n == p.block) {
    if (lane < n) rows[n + lane] = lo2.y;
    if (lane + 32 < n) rows[n + lane + 32] = hi2.y;
  }
  __syncwarp();
  const int k0 = piece * 32 * E * U + lane * E;
  const T* dy = static_cast<const T*>(p.dy) + k0;
  float acc[U * E] = {};
  for (int r = begin & ~(R - 1); r < end; r += R) {
    const uint4 at = *reinterpret_cast<const uint4*>(rows + r);
    const uint32_t row[R] = {at.x, at.y, at.z, at.w};
    Raw<T, E> x[R][U];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const bool in = r + q >= begin && r + q < end;
      const T* src = dy + (in ? row[q] : 0) * p.lddy;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        x[q][u] = Raw<T, E>();
        if (in && k0 + u * 32 * E < p.K) x[q][u] = *reinterpret_cast<const Raw<T, E>*>(src + u * 32 * E);
      }
    }
    uint32_t ends = r < 64 ? (uint32_t)(changes >> r) & (r + R <= n ? (1u << R) - 1 : (1u << max(n - r, 0)) - 1) : 0;
    if (end - 1 - r < R) ends |= 1u << (end - 1 - r);
#pragma unroll
    for (int q = 0; q < R; ++q) {
#pragma unroll
      for (int u = 0; u < U; ++u) add_to<T, E>(acc + u * E, x[q][u]);
      const int at_q = r + q;
      if (!(ends >> q & 1u) || at_q < begin || at_q >= end) continue;
      const uint32_t id = __shfl_sync(all, at_q < n && at_q < 32 ? lo.x : at_q < n ? hi.x : last, at_q % 32);
      const int slot = at_q < head ? 0 : at_q >= tail && at_q < n ? 1 : -1;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * 32 * E;
        if (k < p.K) {
          if (slot < 0) {
            put_row<T, E>(p, id, k, acc + u * E);
          } else {
            Vec<float, E> v;
#pragma unroll
            for (int e = 0; e < E; ++e) v.v[e] = acc[u * E + e];
            *reinterpret_cast<Vec<float, E>*>(p.partial + (2ll * blk + slot) * p.K + k) = v;
          }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) acc[u * E + e] = 0.f;
      }
    }
  }
}

// Long runs: a CTA adds the partial rows of one up in 32 * E * U columns, its warps every eighth and then their sums in order.  (The
// order of the list depends on the launch, the sums do not.)
// (260 runs of 252 rows in 1001 columns: 12 us in pieces of 256 columns, 16 in pieces of 128.)
template <class T, int E, int U>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ SumParams p) {
  __shared__ float sums[8][U][32 * E];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  wait_previous();
  const int pieces = (p.K + 32 * E * U - 1) / (32 * E * U);
  const long long items = (long long)*p.n_long * pieces;
  for (long long item = blockIdx.x; item < items; item += gridDim.x) {
    const int2 run = p.longs[item / pieces];
    const int blk = run.x, k0 = (int)(item % pieces) * 32 * E * U + lane * E;
    const uint32_t id = (uint32_t)run.y;
    int n = 1;  // blocks that it goes on in
    for (bool more = true; more;) {
      bool same[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const long long b = blk + 1ll + n + 32 * j + lane;
        same[j] = b < p.blocks && p.sorted[b * p.block].x == id;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t go = __ballot_sync(0xffffffffu, same[j]);
        if (more) n += go == 0xffffffffu ? 32 : __ffs(~go) - 1;
        more = more && go == 0xffffffffu;
      }
    }
    float acc[U][E] = {};
    const float* at = p.partial + 2ll * blk * p.K + k0;
    constexpr int R = 4;  // partial rows in flight
    for (int b0 = warp; b0 <= n; b0 += 8 * R) {
      Vec<float, E> v[R][U];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int b = b0 + 8 * r;
        const float* from = at + (b ? 2ll * b : 1ll) * p.K;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          v[r][u] = Vec<float, E>();
          if (b <= n && k0 + u * 32 * E < p.K) v[r][u] = *reinterpret_cast<const Vec<float, E>*>(from + u * 32 * E);
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int e = 0; e < E; ++e) acc[u][e] += v[r][u].v[e];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < E; ++e) sums[warp][u][lane * E + e] = acc[u][e];
    __syncthreads();
    if (warp >= U) continue;
    float f[E] = {};  // a warp to each 32 * E columns
    const int k = k0 + warp * 32 * E;
#pragma unroll
    for (int w = 0; w < 8; ++w)
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] += sums[w][warp][lane * E + e];
    if (k < p.K) put_row<T, E>(p, id, k, f);
  }
}

// ------------------------------------------------------------------------------------------------
// Host side
// ------------------------------------------------------------------------------------------------
static int check_shape(const psr_embedding_shape* sh) {
  if (!sh || sh->M < 0 || sh->V < 1 || sh->K < 1) return PSR_ERR_ARG;
  if (sh->type != PSR_BF16 && sh->type != PSR_F16 && sh->type != PSR_F32) return PSR_ERR_ARG;
  if (!std::isfinite(sh->scale)) return PSR_ERR_ARG;
  if (sh->M > 1 << 28 || sh->V > 1 << 30 || sh->K > 1 << 20) return PSR_ERR_UNSUPPORTED;
  if ((sh->ldw && sh->ldw < sh->K) || (sh->ldy && sh->ldy < sh->K)) return PSR_ERR_ARG;
  return PSR_OK;
}

static size_t size_of(int type) { return type == PSR_F32 ? 4 : 2; }

// Elements of the widest vector that the row lengths and addresses allow.
static int vector_of(int type, int K, long long lda, long long ldb, const void* a, const void* b) {
  const int es = (int)size_of(type);
  for (int e = 16 / es; e > 1; e /= 4)
    if (K % e == 0 && lda % e == 0 && ldb % e == 0 && aligned_to(a, (size_t)e * es) && aligned_to(b, (size_t)e * es)) return e;
  return 1;
}

// Calls f(T, E, U) for the type and vector; U vectors to a lane in the sums.
template <class F>
static int dispatch(int type, int e, F f) {
  auto with = [&](auto t) {
    using T = decltype(t);
    if constexpr (sizeof(T) == 4) {
      if (e == 4) return f(t, std::integral_constant<int, 4>(), std::integral_constant<int, 2>());
    } else {
      if (e == 8) return f(t, std::integral_constant<int, 8>(), std::integral_constant<int, 2>());
      if (e == 2) return f(t, std::integral_constant<int, 2>(), std::integral_constant<int, 4>());
    }
    return f(t, std::integral_constant<int, 1>(), std::integral_constant<int, 4>());
  };
  if (type == PSR_BF16) return with(__nv_bfloat16());
  if (type == PSR_F16) return with(__half());
  return with(float());
}

struct Sizes {
  int block, blocks;
  size_t n_long, a, b, longs, partial, total;
};

static int launch_sort(const SortParams& p, cudaStream_t st) {
  if (p.t.M <= kRankMost && p.t.V < (1 << (32 - kRankBits)) - 1) {
    rank_kernel<<<(unsigned)((p.t.M + kRankTokens - 1) / kRankTokens), 4 * kRankTokens, 0, st>>>(p);
    return launch_status();
  }
  static std::mutex mu;
  static bool known[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PSR_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (dev >= 64 || !known[dev]) {
      if (cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(SortSmem)) != cudaSuccess) {
        cudaGetLastError();
        return PSR_ERR_CUDA;
      }
      if (dev < 64) known[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kSortCtas);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = sizeof(SortSmem);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kSortCtas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, sort_kernel, p) == cudaSuccess) return PSR_OK;
  cudaGetLastError();
  return PSR_ERR_CUDA;
}

// Positions of a block: as many as leave every SM 16 warps of 512 columns, between 8 and 64.  (A number for all types and alignments, so that
// the workspace's size needs no addresses.  Rows of fp32, or off 16-byte boundaries, have two to four times the warps: 65539 rows of 1001
// fp32 columns get 32 positions, and an SM 108 warps.)  Shorter blocks cost more starts than they balance, longer ones gain no more (those rows
// in blocks of 64, 32, 16: 83, 83, 89 us).
static Sizes sizes(const psr_embedding_shape* sh) {
  Sizes s;
  const long long warps = (long long)sh->M * ((sh->K + 511) / 512);
  s.block = 8;
  while (s.block < kBlockMost && warps / (2 * s.block) >= 152 * 16) s.block *= 2;
  s.blocks = (int)(((long long)sh->M + s.block - 1) / s.block);
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  s.n_long = 256;
  s.a = 512;
  s.b = s.a + up((size_t)sh->M * 8);
  s.longs = s.b + up((size_t)sh->M * 8);
  s.partial = s.longs + up((size_t)s.blocks * 8);
  s.total = s.partial + up((size_t)s.blocks * 2 * sh->K * 4);
  return s;
}

}  // namespace embedding
}  // namespace psr

using namespace psr;
using namespace psr::embedding;

extern "C" {

int psr_embedding(const psr_embedding_shape* sh, const int64_t* ids, const void* w, void* y, void* stream) {
  int rc = check_shape(sh);
  if (rc != PSR_OK) return rc;
  if (sh->M == 0) return check_device(nullptr);
  if (!ids || !w || !y) return PSR_ERR_ARG;
  if (!aligned_to(ids, 8) || !aligned_to(w, size_of(sh->type)) || !aligned_to(y, size_of(sh->type))) return PSR_ERR_ARG;
  if ((rc = check_device(nullptr)) != PSR_OK) return rc;
  const long long ldw = sh->ldw ? sh->ldw : sh->K, ldy = sh->ldy ? sh->ldy : sh->K;
  const int e = vector_of(sh->type, sh->K, ldw, ldy, w, y);
  return dispatch(sh->type, e, [&](auto t, auto ec, auto) {
    using T = decltype(t);
    constexpr int E = decltype(ec)::value;
    const int pieces = (sh->K + 32 * E * kAhead - 1) / (32 * E * kAhead);
    const long long blocks = ((long long)sh->M * pieces + 7) / 8;
    if (blocks >= 1ll << 31) return (int)PSR_ERR_UNSUPPORTED;
    lookup_kernel<T, E><<<(unsigned)blocks, 256, 0, static_cast<cudaStream_t>(stream)>>>(
        ids, sh->ids_step, static_cast<const T*>(w), ldw, static_cast<T*>(y), ldy, sh->M, sh->V, sh->K, pieces, sh->scale);
    return launch_status();
  });
}

size_t psr_embedding_workspace_bytes(const psr_embedding_shape* sh) {
  return check_shape(sh) == PSR_OK ? sizes(sh).total : 0;
}

int psr_embedding_bwd(const psr_embedding_shape* sh, const void* dy, const int64_t* ids, void* dw, void* workspace,
                      size_t ws_bytes, void* stream) {
  int rc = check_shape(sh);
  if (rc != PSR_OK) return rc;
  if ((sh->M > 0 && (!dy || !ids)) || !dw || !workspace) return PSR_ERR_ARG;
  if (!aligned_to(ids, 8) || !aligned_to(dy, size_of(sh->type)) || !aligned_to(dw, size_of(sh->type)) ||
      !aligned_to(workspace, 256))
    return PSR_ERR_ARG;
  const Sizes s = sizes(sh);
  if (ws_bytes < s.total) return PSR_ERR_ARG;
  int n_sm = 0;
  if ((rc = check_device(&n_sm)) != PSR_OK) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const long long lddy = sh->ldy ? sh->ldy : sh->K;

  if (sh->M == 0) {
    if (cudaMemsetAsync(ws, 0, 256, st) == cudaSuccess &&
        (sh->accumulate || cudaMemsetAsync(dw, 0, (size_t)sh->V * sh->K * size_of(sh->type), st) == cudaSuccess))
      return PSR_OK;
    cudaGetLastError();
    return PSR_ERR_CUDA;
  }

  SortParams q = {};
  q.t = {ids, sh->ids_step, sh->padding, sh->M, sh->V};
  q.a = reinterpret_cast<uint2*>(ws + s.a);
  q.b = reinterpret_cast<uint2*>(ws + s.b);
  q.n_long = reinterpret_cast<int*>(ws + s.n_long);
  int bits = 1;
  while ((1ll << bits) <= sh->V) ++bits;  // of the keys 0 .. V
  q.passes = (bits + kSortBits - 1) / kSortBits;
  q.bits = (bits + q.passes - 1) / q.passes;
  q.clear = reinterpret_cast<Ctrl*>(ws);
  if ((rc = launch_sort(q, st)) != PSR_OK) return rc;

  SumParams p = {};
  p.sorted = q.a;
  p.dy = dy;
  p.lddy = lddy;
  p.dw = dw;
  p.partial = reinterpret_cast<float*>(ws + s.partial);
  p.n_long = q.n_long;
  p.longs = reinterpret_cast<int2*>(ws + s.longs);
  p.M = sh->M;
  p.V = sh->V;
  p.K = sh->K;
  p.block = s.block;
  p.blocks = s.blocks;
  p.accumulate = sh->accumulate;
  p.zero_ctas = sh->accumulate ? 0 : std::min(kZeroCtas * n_sm, (sh->V + 31) / 32);
  p.t = q.t;
  p.scale = sh->scale;
  const int e = vector_of(sh->type, sh->K, lddy, sh->K, dy, dw);
  return dispatch(sh->type, e, [&](auto t, auto ec, auto uc) {
    using T = decltype(t);
    constexpr int E = decltype(ec)::value, U = decltype(uc)::value, UJ = E >= 4 ? 1 : E == 1 ? 8 : U;
    p.pieces = (sh->K + 32 * E * U - 1) / (32 * E * U);
    const long long blocks = p.zero_ctas + ((long long)s.blocks * p.pieces + 7) / 8;
    if (blocks >= 1ll << 31) return (int)PSR_ERR_UNSUPPORTED;
    int r = launch_after(sum_kernel<T, E, U>, dim3((unsigned)blocks), 256, p, st);
    const long long most = (s.blocks - 1ll) / 2 * ((sh->K + 32 * E * UJ - 1) / (32 * E * UJ));  // a long run takes over two blocks
    if (r == PSR_OK && most > 0) r = launch_after(join_kernel<T, E, UJ>, dim3((unsigned)std::min(most, 6ll * n_sm)), 256, p, st);
    return r;
  });
}

}  // extern "C"
