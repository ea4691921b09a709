// The linear layer y = act(x w^T + bias) + residual and its gradients on sm_103a.
#include <cmath>
#include <cstring>

#include "psr_control.cuh"
#include "psr_host.h"

namespace psr {
namespace linear {

// act(z) and act'(z) in fp32
template <int ACT>
__device__ __forceinline__ float act_fwd(float z) {
  if constexpr (ACT == PSR_ACT_RELU) return z > 0.f ? z : (z == z ? 0.f : z);
  if constexpr (ACT == PSR_ACT_GELU) return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
  if constexpr (ACT == PSR_ACT_GELU_TANH)
    return 0.5f * z * (1.f + tanhf(0.79788456080286536f * (z + 0.044715f * z * z * z)));
  if constexpr (ACT == PSR_ACT_SILU) return z / (1.f + expf(-z));
  return z;
}
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == PSR_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  if constexpr (ACT == PSR_ACT_GELU)
    return 0.5f * (1.f + erff(z * 0.70710678118654752f)) + z * 0.39894228040143268f * expf(-0.5f * z * z);
  if constexpr (ACT == PSR_ACT_GELU_TANH) {
    const float u = 0.79788456080286536f * (z + 0.044715f * z * z * z);
    const float t = tanhf(u);
    return 0.5f * (1.f + t) + 0.5f * z * (1.f - t * t) * 0.79788456080286536f * (1.f + 0.134145f * z * z);
  }
  if constexpr (ACT == PSR_ACT_SILU) {
    const float s = 1.f / (1.f + expf(-z));
    return s * (1.f + z * (1.f - s));
  }
  return 1.f;
}

// What becomes of an fp32 sum: z = sum + bias, y = act(z) + residual (or a plain gradient: act none, no bias).
struct Epilogue {
  const void* bias;
  const void* res;
  void* y;
  void* z;
  long long ldr, ldy, ldz;
};

template <class T, int ACT>
__device__ __forceinline__ void finish(const Epilogue& e, long long i, int j, float v) {
  if (e.bias) v += to_f32(static_cast<const T*>(e.bias)[j]);
  if (e.z) static_cast<T*>(e.z)[i * e.ldz + j] = from_f32<T>(v);
  v = act_fwd<ACT>(v);
  if (e.res) v += to_f32(static_cast<const T*>(e.res)[i * e.ldr + j]);
  static_cast<T*>(e.y)[i * e.ldy + j] = from_f32<T>(v);
}

// C[i][j] = sum_k A(i, k) B(j, k), A(i, k) = a[i lda + k] (or a[k lda + i] with AT), B alike: 64 x 64 tiles in
// shared memory, 4 x 4 sums a thread.
template <class T, int ACT, bool AT, bool BT>
__global__ void __launch_bounds__(256)
    simple_gemm(const T* __restrict__ a, long long lda, const T* __restrict__ b, long long ldb, int M, int N, int K,
                const Epilogue e) {
  __shared__ float sa[16][68], sb[16][68];
  const long long i0 = (long long)blockIdx.y * 64;
  const int j0 = blockIdx.x * 64;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < K; k0 += 16) {
    for (int t = threadIdx.x; t < 64 * 16; t += 256) {
      const int ka = AT ? t / 64 : t % 16, ia = AT ? t % 64 : t / 16;
      const bool oka = k0 + ka < K && i0 + ia < M;
      sa[ka][ia] = oka ? to_f32(AT ? a[(long long)(k0 + ka) * lda + i0 + ia] : a[(i0 + ia) * lda + k0 + ka]) : 0.f;
      const int kb = BT ? t / 64 : t % 16, jb = BT ? t % 64 : t / 16;
      const bool okb = k0 + kb < K && j0 + jb < N;
      sb[kb][jb] = okb ? to_f32(BT ? b[(long long)(k0 + kb) * ldb + j0 + jb] : b[(long long)(j0 + jb) * ldb + k0 + kb])
                       : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[r][c] += sa[k][ty * 4 + r] * sb[k][tx * 4 + c];
    __syncthreads();
  }
  for (int r = 0; r < 4; ++r)
    for (int c = 0; c < 4; ++c)
      if (i0 + ty * 4 + r < M && j0 + tx * 4 + c < N) finish<T, ACT>(e, i0 + ty * 4 + r, j0 + tx * 4 + c, acc[r][c]);
}

template <class T, int ACT, bool AT, bool BT>
static int launch_simple(const void* a, long long lda, const void* b, long long ldb, int M, int N, int K,
                         const Epilogue& e, cudaStream_t st) {
  if (M == 0) return PSR_OK;
  const dim3 grid((unsigned)((N + 63) / 64), (unsigned)((M + 63) / 64));
  if (grid.y > 65535) return PSR_ERR_UNSUPPORTED;
  simple_gemm<T, ACT, AT, BT><<<grid, 256, 0, st>>>(static_cast<const T*>(a), lda, static_cast<const T*>(b), ldb, M, N,
                                                   K, e);
  return launch_status();
}

// ------------------------------------------------------------------------------------------------
// dz = dy act'(z), and the column sums of its unrounded values over chunks of rows
// ------------------------------------------------------------------------------------------------
constexpr int kDzRows = 64;  // rows of a chunk

template <class T, int ACT>
__global__ void dz_kernel(const T* __restrict__ dy, long long ldy, const T* __restrict__ z, long long ldz, T* dz,
                          long long lddz, float* partial, int M, int N) {
  const int j = blockIdx.x * 256 + threadIdx.x;
  if (j >= N) return;
  const long long i0 = (long long)blockIdx.y * kDzRows;
  float sum = 0.f;
  for (int r = 0; r < kDzRows && i0 + r < M; ++r) {
    float v = to_f32(dy[(i0 + r) * ldy + j]);
    if constexpr (ACT != PSR_ACT_NONE) v *= act_slope<ACT>(to_f32(z[(i0 + r) * ldz + j]));
    if (dz) dz[(i0 + r) * lddz + j] = from_f32<T>(v);
    sum += v;
  }
  if (partial) partial[(long long)blockIdx.y * N + j] = sum;
}

template <class T>
__global__ void db_kernel(const float* __restrict__ partial, int chunks, int N, T* db) {
  const int j = blockIdx.x * 256 + threadIdx.x;
  if (j >= N) return;
  float sum = 0.f;
  for (int c = 0; c < chunks; ++c) sum += partial[(long long)c * N + j];
  db[j] = from_f32<T>(sum);
}

// ------------------------------------------------------------------------------------------------
// Host side
// ------------------------------------------------------------------------------------------------
struct Sizes {
  long long ldx, ldw, ldr, ldy, ldz;
  int chunks;     // row chunks of the column sums
  long long lddz; // row stride of dz in the workspace
  size_t dz, partial, total_fwd, total_bwd;
};

static size_t au(size_t x) { return (x + 255) / 256 * 256; }

static int sizes(const psr_linear_shape* sh, Sizes& s) {
  if (!sh) return PSR_ERR_ARG;
  if (sh->M < 0 || sh->N < 1 || sh->K < 1) return PSR_ERR_ARG;
  if (sh->act < PSR_ACT_NONE || sh->act > PSR_ACT_SILU) return PSR_ERR_ARG;
  if (sh->type != PSR_BF16 && sh->type != PSR_F16) return PSR_ERR_ARG;
  auto ld = [](long long given, long long contiguous) { return given == 0 ? contiguous : given; };
  s.ldx = ld(sh->ldx, sh->K); s.ldw = ld(sh->ldw, sh->K);
  s.ldr = ld(sh->ldr, sh->N); s.ldy = ld(sh->ldy, sh->N); s.ldz = ld(sh->ldz, sh->N);
  if (s.ldx < sh->K || s.ldw < sh->K || s.ldr < sh->N || s.ldy < sh->N || s.ldz < sh->N) return PSR_ERR_ARG;
  s.chunks = (sh->M + kDzRows - 1) / kDzRows;
  s.lddz = (sh->N + 7) / 8 * 8;
  size_t off = 256;  // control block
  s.total_fwd = off;
  s.dz = off;
  if (sh->act != PSR_ACT_NONE) off = au(off + (size_t)sh->M * s.lddz * 2);
  s.partial = off;
  off = au(off + (size_t)s.chunks * sh->N * 4);
  s.total_bwd = off;
  return PSR_OK;
}

template <class T, int ACT>
static int forward(const psr_linear_shape* sh, const Sizes& s, const void* x, const void* w, const Epilogue& e,
                   cudaStream_t st) {
  return launch_simple<T, ACT, false, false>(x, s.ldx, w, s.ldw, sh->M, sh->N, sh->K, e, st);
}

template <class T, int ACT>
static int make_dz(const psr_linear_shape* sh, const Sizes& s, const void* dy, const void* z, void* dz, float* partial,
                   cudaStream_t st) {
  if (sh->M == 0) return PSR_OK;
  const dim3 grid((unsigned)((sh->N + 255) / 256), (unsigned)s.chunks);
  if (grid.y > 65535) return PSR_ERR_UNSUPPORTED;
  dz_kernel<T, ACT><<<grid, 256, 0, st>>>(static_cast<const T*>(dy), s.ldy, static_cast<const T*>(z), s.ldz,
                                         static_cast<T*>(dz), s.lddz, partial, sh->M, sh->N);
  return launch_status();
}

template <class T>
static int backward(const psr_linear_shape* sh, const Sizes& s, const void* dy, const void* z, const void* x,
                    const void* w, void* dx, void* dw, void* db, uint8_t* ws, cudaStream_t st) {
  const bool act = sh->act != PSR_ACT_NONE;
  void* dz = act ? ws + s.dz : nullptr;
  float* partial = db ? reinterpret_cast<float*>(ws + s.partial) : nullptr;
  int rc = PSR_OK;
  if (act || db) {
    switch (sh->act) {
      case PSR_ACT_RELU: rc = make_dz<T, PSR_ACT_RELU>(sh, s, dy, z, dz, partial, st); break;
      case PSR_ACT_GELU: rc = make_dz<T, PSR_ACT_GELU>(sh, s, dy, z, dz, partial, st); break;
      case PSR_ACT_GELU_TANH: rc = make_dz<T, PSR_ACT_GELU_TANH>(sh, s, dy, z, dz, partial, st); break;
      case PSR_ACT_SILU: rc = make_dz<T, PSR_ACT_SILU>(sh, s, dy, z, dz, partial, st); break;
      default: rc = make_dz<T, PSR_ACT_NONE>(sh, s, dy, z, dz, partial, st);
    }
    if (rc != PSR_OK) return rc;
  }
  if (db) {
    db_kernel<T><<<(unsigned)((sh->N + 255) / 256), 256, 0, st>>>(partial, s.chunks, sh->N, static_cast<T*>(db));
    if ((rc = launch_status()) != PSR_OK) return rc;
  }
  const void* g = act ? dz : dy;
  const long long ldg = act ? s.lddz : s.ldy;
  Epilogue e = {};
  if (dx) {
    e.y = dx;
    e.ldy = sh->K;
    rc = launch_simple<T, PSR_ACT_NONE, false, true>(g, ldg, w, s.ldw, sh->M, sh->K, sh->N, e, st);
    if (rc != PSR_OK) return rc;
  }
  if (dw) {
    e.y = dw;
    e.ldy = sh->K;
    rc = launch_simple<T, PSR_ACT_NONE, true, true>(g, ldg, x, s.ldx, sh->N, sh->K, sh->M, e, st);
  }
  return rc;
}

}  // namespace linear
}  // namespace psr

using namespace psr;
using namespace psr::linear;

extern "C" {

size_t psr_linear_workspace_bytes(const psr_linear_shape* sh, int backward) {
  Sizes s;
  if (sizes(sh, s) != PSR_OK) return 0;
  return backward ? s.total_bwd : s.total_fwd;
}

int psr_linear(const psr_linear_shape* sh, const void* x, const void* w, const void* bias, const void* residual,
               void* y, void* z, void* workspace, size_t ws_bytes, int timeout_ms, void* stream) {
  if (!sh || !x || !w || !y || !workspace) return PSR_ERR_ARG;
  if (!aligned_to(workspace, 256)) return PSR_ERR_ARG;
  for (const void* ptr : {x, w, bias, residual, (const void*)y, (const void*)z})
    if (!aligned_to(ptr, 2)) return PSR_ERR_ARG;
  Sizes s;
  int rc = sizes(sh, s);
  if (rc != PSR_OK) return rc;
  if (ws_bytes < s.total_fwd) return PSR_ERR_ARG;
  if ((rc = check_device(nullptr)) != PSR_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(workspace, 0, 256, st) != cudaSuccess) return PSR_ERR_CUDA;
  const Epilogue e = {bias, residual, y, z, s.ldr, s.ldy, s.ldz};
  auto go = [&](auto tag) {
    using T = decltype(tag);
    switch (sh->act) {
      case PSR_ACT_RELU: return forward<T, PSR_ACT_RELU>(sh, s, x, w, e, st);
      case PSR_ACT_GELU: return forward<T, PSR_ACT_GELU>(sh, s, x, w, e, st);
      case PSR_ACT_GELU_TANH: return forward<T, PSR_ACT_GELU_TANH>(sh, s, x, w, e, st);
      case PSR_ACT_SILU: return forward<T, PSR_ACT_SILU>(sh, s, x, w, e, st);
      default: return forward<T, PSR_ACT_NONE>(sh, s, x, w, e, st);
    }
  };
  return sh->type == PSR_BF16 ? go(__nv_bfloat16()) : go(__half());
}

int psr_linear_bwd(const psr_linear_shape* sh, const void* dy, const void* z, const void* x, const void* w, void* dx,
                   void* dw, void* db, void* workspace, size_t ws_bytes, int timeout_ms, void* stream) {
  if (!sh || !dy || !x || !w || !workspace || (sh->act != PSR_ACT_NONE && !z)) return PSR_ERR_ARG;
  if (!aligned_to(workspace, 256)) return PSR_ERR_ARG;
  for (const void* ptr : {dy, z, x, w, (const void*)dx, (const void*)dw, (const void*)db})
    if (!aligned_to(ptr, 2)) return PSR_ERR_ARG;
  Sizes s;
  int rc = sizes(sh, s);
  if (rc != PSR_OK) return rc;
  if (ws_bytes < s.total_bwd) return PSR_ERR_ARG;
  if ((rc = check_device(nullptr)) != PSR_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(workspace, 0, 256, st) != cudaSuccess) return PSR_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  return sh->type == PSR_BF16 ? backward<__nv_bfloat16>(sh, s, dy, z, x, w, dx, dw, db, ws, st)
                              : backward<__half>(sh, s, dy, z, x, w, dx, dw, db, ws, st);
}

}  // extern "C"
