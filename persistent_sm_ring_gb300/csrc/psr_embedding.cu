// The embedding on sm_103a: rows of a table looked up by token and scaled, and the table's gradient.
//
// Forward: y_i = scale w[id_i].  Backward: dw_v = scale sum of dy_i over the i with id_i = v, in the order of i, with fp32
// sums: the tokens are sorted by id (stable), blocks of sorted positions are summed, and a run of equal ids that crosses
// blocks is joined from fp32 partials in order.  No result depends on the order in which blocks run.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "psr_control.cuh"
#include "psr_device.cuh"
#include "psr_host.h"

namespace psr {
namespace embedding {

// E adjacent elements of a row
template <class T, int E>
struct alignas(sizeof(T) * E) Vec { T v[E]; };

// ------------------------------------------------------------------------------------------------
// Lookup
// ------------------------------------------------------------------------------------------------
// Memory bound.  A warp takes 32 * kAhead vectors of a row, all of them in flight at once.
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
    *reinterpret_cast<Vec<T, E>*>(dst + k) = x[a];
  }
}

// ------------------------------------------------------------------------------------------------
// Sort of the tokens by id, and zeros for the rows that no token names
// ------------------------------------------------------------------------------------------------
// A cluster of CTAs sorts (id, position) pairs by up to nine bits a pass, least significant first.  Each warp has a
// contiguous share of the pairs and counts its digits; the counts before it (of smaller digits, of earlier CTAs and warps) are
// where its pairs go, equal digits in their order.  Ids outside the table, and the padding id, become V: they end up behind all
// others.  The grid's other clusters meanwhile write the zeros, each CTA those of its own range of the table, for
// which it marks the ids that occur.
constexpr int kSortCtas = 8, kSortThreads = 1024, kSortWarps = kSortThreads / 32, kSortBits = 9, kBins = 1 << kSortBits;
constexpr int kMarks = 32768;  // table rows that a CTA marks at a time

struct SortParams {
  const int64_t* ids;
  long long step;
  long long padding;  // an id without gradient (negative: none)
  int M, V;
  uint2* a;        // the sorted pairs (key, position)
  uint2* b;        // space for them between passes
  int passes, bits;
  uint8_t* dw;     // rows to clear, or null
  long long row_bytes;
  Ctrl* clear;
};

struct SortSmem {
  uint32_t hist[kSortWarps][kBins];
  uint32_t total[kBins];  // of this CTA, by digit; read by the others
  uint32_t warp_sum[kSortWarps];
};

__device__ __forceinline__ uint32_t key_of(const SortParams& p, long long i) {
  const long long id = p.ids[i * p.step];
  return id >= 0 && id < p.V && id != p.padding ? (uint32_t)id : (uint32_t)p.V;
}

// `n` bytes of zeros (an even number, from an even address) by a warp.
__device__ __forceinline__ void zero_bytes(uint8_t* at, long long n) {
  const int lane = threadIdx.x % 32;
  long long head = (16 - (long long)(reinterpret_cast<uintptr_t>(at) % 16)) % 16;
  if (head > n) head = n;
  if (2 * lane < head) *reinterpret_cast<uint16_t*>(at + 2 * lane) = 0;
  const long long body = (n - head) / 16, tail = n - head - body * 16;
  uint4* v = reinterpret_cast<uint4*>(at + head);
  for (long long i = lane; i < body; i += 32) v[i] = make_uint4(0, 0, 0, 0);
  if (2 * lane < tail) *reinterpret_cast<uint16_t*>(at + n - tail + 2 * lane) = 0;
}

__device__ void zero_rows(const SortParams& p, uint32_t* marks) {
  const int n_cta = gridDim.x - kSortCtas, cta = blockIdx.x - kSortCtas;
  const long long per = ((long long)p.V + n_cta - 1) / n_cta;
  const long long end = min((long long)p.V, (cta + 1) * per);
  for (long long v0 = cta * per; v0 < end; v0 += kMarks) {
    const int n = (int)min((long long)kMarks, end - v0);
    for (int i = threadIdx.x; i < (n + 31) / 32; i += kSortThreads) marks[i] = 0;
    __syncthreads();
    for (long long i = threadIdx.x; i < p.M; i += kSortThreads) {
      const long long r = (long long)key_of(p, i) - v0;
      if (r >= 0 && r < n) atomicOr(&marks[r / 32], 1u << (r % 32));
    }
    __syncthreads();
    for (int r = threadIdx.x / 32; r < n; r += kSortWarps)
      if (!(marks[r / 32] >> (r % 32) & 1u)) zero_bytes(p.dw + (v0 + r) * p.row_bytes, p.row_bytes);
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kSortThreads, 1) sort_kernel(const __grid_constant__ SortParams p) {
  extern __shared__ uint8_t smem_raw[];
  SortSmem& sm = *reinterpret_cast<SortSmem*>(smem_raw);
  clear_ctrl(p.clear);
  if (blockIdx.x >= kSortCtas) {
    zero_rows(p, &sm.hist[0][0]);
    return;
  }
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const long long share = (((long long)p.M + kSortCtas * kSortWarps - 1) / (kSortCtas * kSortWarps) + 31) / 32 * 32;
  const long long i0 = ((long long)rank * kSortWarps + warp) * share;
  const long long i1 = min((long long)p.M, i0 + share);
  const uint32_t bins = 1u << p.bits;
  for (int pass = 0; pass < p.passes; ++pass) {
    const uint2* src = (p.passes - pass) % 2 ? p.b : p.a;  // the last pass writes a
    uint2* dst = (p.passes - pass) % 2 ? p.a : p.b;
    const int shift = pass * p.bits;
    auto pair = [&](long long i) { return pass == 0 ? make_uint2(key_of(p, i), (uint32_t)i) : src[i]; };
    for (uint32_t d = lane; d < bins; d += 32) sm.hist[warp][d] = 0;
    __syncwarp();
    for (long long i = i0; i < i1; i += 32) {  // (whole warps: a warp's last lanes may have no pair)
      const bool in = i + lane < i1;
      const uint32_t d = in ? pair(i + lane).x >> shift & (bins - 1) : bins;
      const uint32_t same = __match_any_sync(0xffffffffu, d);
      if (in && lane == __ffs(same) - 1) sm.hist[warp][d] += __popc(same);
      __syncwarp();
    }
    __syncthreads();
    uint32_t total = 0;
    if (threadIdx.x < bins) {
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
      for (uint32_t c = 0; c < (uint32_t)kSortCtas; ++c) {
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
      for (int w = 0; w < warp; ++w) base += sm.warp_sum[w];
      for (int w = 0; w < kSortWarps; ++w) sm.hist[w][threadIdx.x] += base;
    }
    __syncthreads();
    for (long long i = i0; i < i1; i += 32) {
      const bool in = i + lane < i1;
      uint2 x = make_uint2(0, 0);
      if (in) x = pair(i + lane);
      const uint32_t d = in ? x.x >> shift & (bins - 1) : bins;
      const uint32_t same = __match_any_sync(0xffffffffu, d);
      uint32_t at = 0;
      if (in) at = sm.hist[warp][d] + __popc(same & ((1u << lane) - 1));
      __syncwarp();
      if (in) {
        dst[at] = x;
        if (lane == __ffs(same) - 1) sm.hist[warp][d] += __popc(same);
      }
      __syncwarp();
    }
    cluster_sync();  // the next pass, or the CTAs' ends: all pairs are in place, all totals read
  }
}

// ------------------------------------------------------------------------------------------------
// Sums of the rows of each id
// ------------------------------------------------------------------------------------------------
// Memory bound.  A warp takes a block of sorted positions and 32 * E * U columns, reads four rows at a time and writes a
// row of dw where the id changes.  A run that began in an earlier block goes to the block's first partial row, one that goes
// on in the next block to its second; join_kernel adds those up.
constexpr int kBlockMost = 64;  // positions of a block

struct SumParams {
  const uint2* sorted;
  const void* dy;
  long long lddy;
  void* dw;
  float* partial;  // [blocks][2][K]
  int M, V, K, block, blocks, pieces;
  int accumulate;
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
__global__ void __launch_bounds__(256) sum_kernel(const __grid_constant__ SumParams p) {
  constexpr int R = 4;
  const long long item = blockIdx.x * 8ll + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const int blk = (int)(item / p.pieces);
  wait_previous();
  if (blk >= p.blocks) return;
  const int k0 = (int)(item - (long long)blk * p.pieces) * 32 * E * U + lane * E;
  const long long i0 = (long long)blk * p.block;
  const int n = (int)min((long long)p.block, p.M - i0);
  const uint2* s = p.sorted + i0;
  const uint32_t none = 0xffffffffu;
  uint2 lo = make_uint2(none, 0), hi = make_uint2(none, 0);
  if (lane < n) lo = s[lane];
  if (lane + 32 < n) hi = s[lane + 32];
  const uint32_t before = i0 > 0 ? s[-1].x : none, after = i0 + n < p.M ? s[n].x : none;
  auto key = [&](int r) { return __shfl_sync(0xffffffffu, r < 32 ? lo.x : hi.x, r % 32); };
  auto row = [&](int r) { return __shfl_sync(0xffffffffu, r < 32 ? lo.y : hi.y, r % 32); };
  float acc[U * E] = {};
  bool first = true;
  uint32_t id = key(0);
  for (int r = 0; r < n && id < (uint32_t)p.V; r += R) {
    Vec<T, E> x[R][U];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const bool in = r + q < n && key(min(r + q, n - 1)) < (uint32_t)p.V;
      const T* src = static_cast<const T*>(p.dy) + (long long)row(min(r + q, n - 1)) * p.lddy;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * 32 * E;
        if (in && k < p.K) x[q][u] = *reinterpret_cast<const Vec<T, E>*>(src + k);
      }
    }
#pragma unroll
    for (int q = 0; q < R; ++q) {
      if (r + q >= n || id >= (uint32_t)p.V) break;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (k0 + u * 32 * E < p.K)
#pragma unroll
          for (int e = 0; e < E; ++e) acc[u * E + e] += to_f32(x[q][u].v[e]);
      const bool last = r + q + 1 == n;
      const uint32_t next = last ? none : key(min(r + q + 1, n - 1));
      if (next == id) continue;
      const int slot = first && before == id ? 0 : last && after == id ? 1 : -1;
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
      id = next;
      first = false;
    }
  }
}

// Runs that cross blocks: the block where a run begins adds its partial rows up, in order.
template <class T, int E, int U>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ SumParams p) {
  const long long item = blockIdx.x * 8ll + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const int blk = (int)(item / p.pieces);
  wait_previous();
  if (blk >= p.blocks - 1) return;
  const long long i0 = (long long)blk * p.block, i1 = i0 + p.block;
  const uint32_t id = p.sorted[i1].x;
  if (id >= (uint32_t)p.V || p.sorted[i1 - 1].x != id) return;      // no run goes on
  if (i0 > 0 && p.sorted[i0].x == id && p.sorted[i0 - 1].x == id) return;  // it began earlier
  int n = 1;  // blocks that it goes on in
  for (bool more = true; more;) {
    const long long b = blk + 1ll + n + lane;
    const uint32_t go = __ballot_sync(0xffffffffu, b < p.blocks && p.sorted[b * p.block].x == id);
    const int run = go == 0xffffffffu ? 32 : __ffs(~go) - 1;
    n += run;
    more = run == 32;
  }
  const int k0 = (int)(item - (long long)blk * p.pieces) * 32 * E * U + lane * E;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int k = k0 + u * 32 * E;
    if (k >= p.K) break;
    const float* at = p.partial + 2ll * blk * p.K + k;
    float acc[E];
    const Vec<float, E> v = *reinterpret_cast<const Vec<float, E>*>(at + p.K);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = v.v[e];
#pragma unroll 8
    for (int b = 1; b <= n; ++b) {
      const Vec<float, E> w = *reinterpret_cast<const Vec<float, E>*>(at + 2ll * b * p.K);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += w.v[e];
    }
    put_row<T, E>(p, id, k, acc);
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
  size_t a, b, partial, total;
};

// Positions of a block: as many as leave every SM 16 warps, between 8 and 64.
static Sizes sizes(const psr_embedding_shape* sh) {
  Sizes s;
  const long long warps = (long long)sh->M * ((sh->K + 511) / 512);
  s.block = 8;
  while (s.block < kBlockMost && warps / (2 * s.block) >= 152 * 16) s.block *= 2;
  s.blocks = (int)(((long long)sh->M + s.block - 1) / s.block);
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  s.a = 256;
  s.b = s.a + up((size_t)sh->M * 8);
  s.partial = s.b + up((size_t)sh->M * 8);
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

  SortParams q = {};
  q.ids = ids;
  q.step = sh->ids_step;
  q.padding = sh->padding;
  q.M = sh->M;
  q.V = sh->V;
  q.a = reinterpret_cast<uint2*>(ws + s.a);
  q.b = reinterpret_cast<uint2*>(ws + s.b);
  int bits = 1;
  while ((1ll << bits) <= sh->V) ++bits;  // of the keys 0 .. V
  q.passes = (bits + kSortBits - 1) / kSortBits;
  q.bits = (bits + q.passes - 1) / q.passes;
  q.dw = sh->accumulate ? nullptr : static_cast<uint8_t*>(dw);
  q.row_bytes = (long long)sh->K * size_of(sh->type);
  q.clear = reinterpret_cast<Ctrl*>(ws);
  if (cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(SortSmem)) != cudaSuccess) {
    cudaGetLastError();
    return PSR_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(sh->accumulate ? kSortCtas : n_sm / kSortCtas * kSortCtas));
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
  if (cudaLaunchKernelEx(&cfg, sort_kernel, q) != cudaSuccess) {
    cudaGetLastError();
    return PSR_ERR_CUDA;
  }
  if (sh->M == 0) return PSR_OK;

  SumParams p = {};
  p.sorted = q.a;
  p.dy = dy;
  p.lddy = lddy;
  p.dw = dw;
  p.partial = reinterpret_cast<float*>(ws + s.partial);
  p.M = sh->M;
  p.V = sh->V;
  p.K = sh->K;
  p.block = s.block;
  p.blocks = s.blocks;
  p.accumulate = sh->accumulate;
  p.scale = sh->scale;
  const int e = vector_of(sh->type, sh->K, lddy, sh->K, dy, dw);
  return dispatch(sh->type, e, [&](auto t, auto ec, auto uc) {
    using T = decltype(t);
    constexpr int E = decltype(ec)::value, U = decltype(uc)::value;
    p.pieces = (sh->K + 32 * E * U - 1) / (32 * E * U);
    const long long blocks = ((long long)s.blocks * p.pieces + 7) / 8;
    if (blocks >= 1ll << 31) return (int)PSR_ERR_UNSUPPORTED;
    int r = launch_after(sum_kernel<T, E, U>, dim3((unsigned)blocks), 256, p, st);
    if (r == PSR_OK && s.blocks > 1) r = launch_after(join_kernel<T, E, U>, dim3((unsigned)blocks), 256, p, st);
    return r;
  });
}

}  // extern "C"
