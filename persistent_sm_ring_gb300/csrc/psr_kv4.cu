// KV cache in 4 bits on sm_103a: quantise and append, read back, and the attention of new tokens over the pages.
//
// The cache is laid out in blocks of 16 tokens of one KV head: K codes, V codes, then the (scale, offset) pairs,
// 16 (d + 8) bytes in one piece, so that whatever the page size a block is one contiguous 16-byte aligned copy.
// One scale and offset for a row (not for groups of columns) keeps them out of the products: with c the codes,
//     q . k = scale (q . c) + offset sum(q),        sum_j p_j v_j = sum_j (p_j scale_j) c_j + sum_j p_j offset_j.
#include <cmath>
#include <cstring>

#include "psr_control.cuh"
#include "psr_host.h"

namespace psr {
namespace kv4 {

constexpr int kBlk = 16;  // tokens of a block

struct Cache {
  uint8_t* base;
  const int32_t* table;
  int Hkv, d, page, n_pages, max_pages;
};

__device__ __forceinline__ int block_bytes(int d) { return kBlk * (d + 8); }

// The block that holds position pos of sequence b for KV head h, or null if the table has no usable page there.
__device__ __forceinline__ uint8_t* block_of(const Cache& c, int b, int h, long long pos) {
  if (pos < 0 || pos >= (long long)c.max_pages * c.page) return nullptr;
  const int pg = c.table[(long long)b * c.max_pages + (int)(pos / c.page)];
  if (pg < 0 || pg >= c.n_pages) return nullptr;
  const int per = c.page / kBlk;
  return c.base + (((long long)pg * c.Hkv + h) * per + (int)(pos % c.page) / kBlk) * block_bytes(c.d);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_min(float v) { return -warp_max(-v); }
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ------------------------------------------------------------------------------------------------
// Append: one warp quantises one row of K or V
// ------------------------------------------------------------------------------------------------
struct AppendParams {
  Cache c;
  const void* x[2];
  psr_strides st[2];
  const int32_t *start, *count;
  int B, S;
};

template <class T, int D>
__global__ void append_kernel(const AppendParams p) {
  constexpr int E = D / 32;  // elements a lane, adjacent columns
  const int lane = threadIdx.x % 32;
  const long long rows = 2LL * p.B * p.c.Hkv * p.S;
  for (long long r = (blockIdx.x * (long long)blockDim.x + threadIdx.x) / 32; r < rows;
       r += (long long)gridDim.x * blockDim.x / 32) {
    const int kv = (int)(r & 1);
    long long t = r >> 1;
    const int i = (int)(t % p.S);
    t /= p.S;
    const int h = (int)(t % p.c.Hkv), b = (int)(t / p.c.Hkv);
    if (p.count && i >= p.count[b]) continue;
    const long long pos = (long long)p.start[b] + i;
    uint8_t* blk = block_of(p.c, b, h, pos);
    if (!blk) continue;
    const T* x = static_cast<const T*>(p.x[kv]) + b * p.st[kv].b + h * p.st[kv].h + i * p.st[kv].s;
    float v[E];
    bool fine = true;
    float mn = INFINITY, mx = -INFINITY;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      v[e] = to_f32(x[lane * E + e]);
      fine = fine && isfinite(v[e]);
      mn = fminf(mn, v[e]);
      mx = fmaxf(mx, v[e]);
    }
    mn = warp_min(mn);
    mx = warp_max(mx);
    fine = __all_sync(0xffffffffu, fine);
    // max/15 - min/15: max - min can pass the largest fp32 number
    __nv_bfloat16 sc = __float2bfloat16_rn(__fsub_rn(__fdiv_rn(mx, 15.f), __fdiv_rn(mn, 15.f)));
    __nv_bfloat16 of = __float2bfloat16_rn(mn);
    const float s = __bfloat162float(sc), o = __bfloat162float(of);
    uint32_t codes = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float c = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(v[e], o), s)), 0.f), 15.f);
      if (fine && s > 0.f) codes |= (uint32_t)c << (4 * e);
    }
    if (!fine) sc = of = __ushort_as_bfloat16(0x7FFF);
    const int row = (int)(pos % kBlk);
    uint8_t* dst = blk + kv * kBlk * (D / 2) + row * (D / 2) + lane * (E / 2);
    if constexpr (E == 4) *reinterpret_cast<uint16_t*>(dst) = (uint16_t)codes;
    else *dst = (uint8_t)codes;
    if (lane == 0) {
      __nv_bfloat162 pair;
      pair.x = sc;
      pair.y = of;
      *reinterpret_cast<__nv_bfloat162*>(blk + kBlk * D + kv * kBlk * 4 + row * 4) = pair;
    }
  }
}

// ------------------------------------------------------------------------------------------------
// Read: one warp dequantises one row of K or V
// ------------------------------------------------------------------------------------------------
struct ReadParams {
  Cache c;
  void* x[2];
  const int32_t *start, *count;
  int B, S;
};

template <class T, int D>
__global__ void read_kernel(const ReadParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x % 32;
  const long long rows = 2LL * p.B * p.c.Hkv * p.S;
  for (long long r = (blockIdx.x * (long long)blockDim.x + threadIdx.x) / 32; r < rows;
       r += (long long)gridDim.x * blockDim.x / 32) {
    const int kv = (int)(r & 1);
    const long long t = r >> 1;
    const int i = (int)(t % p.S);
    const int h = (int)(t / p.S % p.c.Hkv), b = (int)(t / p.S / p.c.Hkv);
    T* x = static_cast<T*>(p.x[kv]) + t * D + lane * E;
    const bool live = !p.count || i < p.count[b];
    const long long pos = (long long)p.start[b] + i;
    const uint8_t* blk = live ? block_of(p.c, b, h, pos) : nullptr;
    float s = 0.f, o = live ? NAN : 0.f;
    uint32_t codes = 0;
    if (blk) {
      const int row = (int)(pos % kBlk);
      const __nv_bfloat162 pair = *reinterpret_cast<const __nv_bfloat162*>(blk + kBlk * D + kv * kBlk * 4 + row * 4);
      s = __bfloat162float(pair.x);
      o = __bfloat162float(pair.y);
      const uint8_t* src = blk + kv * kBlk * (D / 2) + row * (D / 2) + lane * (E / 2);
      if constexpr (E == 4) codes = *reinterpret_cast<const uint16_t*>(src);
      else codes = *src;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = from_f32<T>(fmaf((float)((codes >> (4 * e)) & 15u), s, o));
  }
}

// ------------------------------------------------------------------------------------------------
// Attention: one block for a query row, its warps over the positions
// ------------------------------------------------------------------------------------------------
struct AttnParams {
  Cache c;
  const void* q;
  void* o;
  float* lse;
  const int32_t* lens;
  psr_strides sq, so;
  int B, Hq, S;
  float scale;
};

template <class T, int D>
__global__ void __launch_bounds__(128) attn_kernel(const AttnParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  __shared__ float so[4][D], sm[4], sl[4];
  const long long row = blockIdx.x;
  const int i = (int)(row % p.S), hq = (int)(row / p.S % p.Hq), b = (int)(row / p.S / p.Hq);
  const int h = hq / (p.Hq / p.c.Hkv);
  const int n = p.lens[b];
  const T* q = static_cast<const T*>(p.q) + b * p.sq.b + hq * p.sq.h + i * p.sq.s;
  float qv[E], o[E] = {}, m = -INFINITY, l = 0.f, bad = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) qv[e] = to_f32(q[lane * E + e]) * p.scale;
  if (n < 0 || n > p.c.max_pages * (long long)p.c.page) bad = NAN;
  else
    for (int j = warp; j < n; j += 4) {
      const uint8_t* blk = block_of(p.c, b, h, j);
      if (!blk) { bad = NAN; continue; }
      if (j > n - p.S + i) continue;
      auto load = [&](int kv, float (&x)[E]) {
        const __nv_bfloat162 pair = *reinterpret_cast<const __nv_bfloat162*>(blk + kBlk * D + kv * kBlk * 4 + j % kBlk * 4);
        const uint8_t* src = blk + kv * kBlk * (D / 2) + j % kBlk * (D / 2) + lane * (E / 2);
        uint32_t codes;
        if constexpr (E == 4) codes = *reinterpret_cast<const uint16_t*>(src);
        else codes = *src;
#pragma unroll
        for (int e = 0; e < E; ++e)
          x[e] = fmaf((float)((codes >> (4 * e)) & 15u), __bfloat162float(pair.x), __bfloat162float(pair.y));
      };
      float kk[E], vv[E], x = 0.f;
      load(0, kk);
      load(1, vv);
#pragma unroll
      for (int e = 0; e < E; ++e) x += qv[e] * kk[e];
      x = warp_sum(x);
      const float mn = fmaxf(m, x);
      const float a = expf(m - mn), w = expf(x - mn);
      m = mn;
      l = l * a + w;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = o[e] * a + w * vv[e];
    }
#pragma unroll
  for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l + bad;
  }
  __syncthreads();
  if (warp) return;
  const float mm = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  float ll = 0.f, acc[E] = {};
  for (int w = 0; w < 4; ++w) {
    const float a = sm[w] == -INFINITY ? 0.f : expf(sm[w] - mm);
    ll += sm[w] == -INFINITY ? sl[w] : sl[w] * a;
    for (int e = 0; e < E; ++e) acc[e] += so[w][lane * E + e] * a;
  }
  T* out = static_cast<T*>(p.o) + b * p.so.b + hq * p.so.h + i * p.so.s;
  for (int e = 0; e < E; ++e) out[lane * E + e] = from_f32<T>(ll == 0.f ? 0.f : acc[e] / ll);
  if (lane == 0) p.lse[row] = ll == 0.f ? -INFINITY : mm + logf(ll);
}

// ------------------------------------------------------------------------------------------------
// Host side
// ------------------------------------------------------------------------------------------------
static int check_shape(const psr_kv4_shape* sh) {
  if (!sh) return PSR_ERR_ARG;
  if (sh->B < 0 || sh->S < 0 || sh->Hq < 1 || sh->Hkv < 1 || sh->n_pages < 1 || sh->max_pages < 1) return PSR_ERR_ARG;
  if (sh->type != PSR_BF16 && sh->type != PSR_F16) return PSR_ERR_ARG;
  if (sh->Hq % sh->Hkv != 0 || (sh->d != 64 && sh->d != 128)) return PSR_ERR_UNSUPPORTED;
  if (sh->page < 16 || sh->page > 256 || (sh->page & (sh->page - 1)) != 0) return PSR_ERR_UNSUPPORTED;
  if ((long long)sh->max_pages * sh->page >= (1LL << 31)) return PSR_ERR_UNSUPPORTED;
  return PSR_OK;
}

static Cache cache_of(const psr_kv4_shape* sh, const void* cache, const int32_t* table) {
  return {const_cast<uint8_t*>(static_cast<const uint8_t*>(cache)), table, sh->Hkv, sh->d, sh->page, sh->n_pages,
          sh->max_pages};
}

template <class Go>
static int by_type(const psr_kv4_shape* sh, Go&& go) {
  if (sh->type == PSR_BF16)
    return sh->d == 64 ? go(__nv_bfloat16(), std::integral_constant<int, 64>())
                       : go(__nv_bfloat16(), std::integral_constant<int, 128>());
  return sh->d == 64 ? go(__half(), std::integral_constant<int, 64>()) : go(__half(), std::integral_constant<int, 128>());
}

static unsigned row_blocks(const psr_kv4_shape* sh, int n_sm) {
  const long long rows = 2LL * sh->B * sh->Hkv * sh->S;
  const long long blocks = (rows + 7) / 8;
  return (unsigned)(blocks < n_sm * 32 ? blocks : n_sm * 32);
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
  int n_sm = 0;
  if ((rc = check_device(&n_sm)) != PSR_OK) return rc;
  if (sh->B == 0 || sh->S == 0) return PSR_OK;
  AppendParams p = {cache_of(sh, cache, table), {k, v}, {*ks, *vs}, start, count, sh->B, sh->S};
  return by_type(sh, [&](auto t, auto d) {
    append_kernel<decltype(t), decltype(d)::value><<<row_blocks(sh, n_sm), 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
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
  int n_sm = 0;
  if ((rc = check_device(&n_sm)) != PSR_OK) return rc;
  if (sh->B == 0 || sh->S == 0) return PSR_OK;
  ReadParams p = {cache_of(sh, cache, table), {k, v}, start, count, sh->B, sh->S};
  return by_type(sh, [&](auto t, auto d) {
    read_kernel<decltype(t), decltype(d)::value><<<row_blocks(sh, n_sm), 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return launch_status();
  });
}

size_t psr_kv4_attn_workspace_bytes(const psr_kv4_shape* sh) {
  if (check_shape(sh) != PSR_OK) return 0;
  return 256;
}

int psr_kv4_attn(const psr_kv4_shape* sh, const void* q, const psr_strides* qs, const void* cache, const int32_t* table,
                 const int32_t* lens, void* o, const psr_strides* os, float* lse, void* workspace, size_t ws_bytes,
                 int timeout_ms, void* stream) {
  if (!sh || !q || !qs || !cache || !table || !lens || !o || !os || !lse || !workspace) return PSR_ERR_ARG;
  if (!aligned_to(q, 2) || !aligned_to(o, 2) || !aligned_to(lse, 4) || !aligned_to(cache, 16) ||
      !aligned_to(table, 4) || !aligned_to(lens, 4) || !aligned_to(workspace, 256))
    return PSR_ERR_ARG;
  int rc = check_shape(sh);
  if (rc != PSR_OK) return rc;
  if (ws_bytes < psr_kv4_attn_workspace_bytes(sh)) return PSR_ERR_ARG;
  const long long rows = (long long)sh->B * sh->Hq * sh->S;
  if (rows >= (1LL << 31)) return PSR_ERR_UNSUPPORTED;
  if ((rc = check_device(nullptr)) != PSR_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(workspace, 0, 256, st) != cudaSuccess) return PSR_ERR_CUDA;
  if (rows == 0) return PSR_OK;
  AttnParams p = {cache_of(sh, cache, table), q, o, lse, lens, *qs, *os, sh->B, sh->Hq, sh->S,
                  sh->scale > 0.f ? sh->scale : 1.f / sqrtf((float)sh->d)};
  return by_type(sh, [&](auto t, auto d) {
    attn_kernel<decltype(t), decltype(d)::value><<<(unsigned)rows, 128, 0, st>>>(p);
    return launch_status();
  });
}

}  // extern "C"
