// The linear layer y = act(x w^T + bias) + residual and its gradients on sm_103a.
//
// Operands whose rows start on 16-byte boundaries go to the tcgen05 products of psr_linear_mma.cuh; others (odd
// strides, odd offsets) to a plain tiled product on the fp32 units.
#include <cmath>
#include <cstring>

#include "psr_control.cuh"
#include "psr_host.h"
#include "psr_linear_mma.cuh"

namespace psr {
namespace linear {

// C[i][j] = sum_k A(i, k) B(j, k), A(i, k) = a[i lda + k] (or a[k lda + i] with AT), B alike: 64 x 64 tiles in
// shared memory, 4 x 4 sums a thread.
template <class T, bool AT, bool BT>
__global__ void __launch_bounds__(256)
    simple_gemm(const T* __restrict__ a, long long lda, const T* __restrict__ b, long long ldb, int M, int N, int K,
                const Epilogue e) {
  __shared__ float sa[16][68], sb[16][68];
  const long long i0 = (long long)blockIdx.x * 64;
  const int j0 = blockIdx.y * 64;
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
      if (i0 + ty * 4 + r < M && j0 + tx * 4 + c < N) finish(e, i0 + ty * 4 + r, j0 + tx * 4 + c, acc[r][c]);
}

template <class T, bool AT, bool BT>
static int launch_simple(const void* a, long long lda, const void* b, long long ldb, int M, int N, int K,
                         const Epilogue& e, cudaStream_t st) {
  if (M == 0) return PSR_OK;
  const dim3 grid((unsigned)((M + 63) / 64), (unsigned)((N + 63) / 64));
  if (grid.y > 65535) return PSR_ERR_UNSUPPORTED;
  simple_gemm<T, AT, BT><<<grid, 256, 0, st>>>(static_cast<const T*>(a), lda, static_cast<const T*>(b), ldb, M, N,
                                                   K, e);
  return launch_status();
}

// ------------------------------------------------------------------------------------------------
// dz = dy act'(z), and the column sums of its unrounded values over chunks of rows
// ------------------------------------------------------------------------------------------------
constexpr int kDzRows = 64;  // rows of a chunk

template <class T>
__global__ void dz_kernel(const T* __restrict__ dy, long long ldy, const T* __restrict__ z, long long ldz, T* dz,
                          long long lddz, float* partial, int M, int N, int act) {
  const int j = blockIdx.y * 256 + threadIdx.x;
  if (j >= N) return;
  const long long i0 = (long long)blockIdx.x * kDzRows;
  float sum = 0.f;
  for (int r = 0; r < kDzRows && i0 + r < M; ++r) {
    float v = to_f32(dy[(i0 + r) * ldy + j]);
    if (act != PSR_ACT_NONE) v *= act_slope(act, to_f32(z[(i0 + r) * ldz + j]));
    if (dz) dz[(i0 + r) * lddz + j] = from_f32<T>(v);
    sum += v;
  }
  if (partial) partial[(long long)blockIdx.x * N + j] = sum;
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
  size_t stream, dz, partial, total_fwd, total_bwd;
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
  s.stream = off;
  off = au(off + stream_partial_bytes(sh->M));
  s.total_fwd = off;
  s.dz = off;
  if (sh->act != PSR_ACT_NONE) off = au(off + (size_t)sh->M * s.lddz * 2);
  s.partial = off;
  off = au(off + (size_t)s.chunks * sh->N * 4);
  s.total_bwd = off;
  return PSR_OK;
}

struct Launch {
  int dev, n_sm;
  Ctrl* ctrl;
  float* stream_partial;
  unsigned long long timeout_ns;
  cudaStream_t st;
};

// C = A B^T with A [M][K] (or AMN: [K][M]) and B [N][K] (or BMN: [K][N]).  W is the operand that streams when
// there are few rows of A.
template <class T, bool AMN, bool BMN>
static int product(const Operands& o, Epilogue e, const Launch& l) {
  if (o.M == 0) return PSR_OK;
  if (!mappable(o.a, AMN ? o.K : o.M, o.lda) || !mappable(o.b, BMN ? o.K : o.N, o.ldb))
    return launch_simple<T, AMN, BMN>(o.a, o.lda, o.b, o.ldb, o.M, o.N, o.K, e, l.st);
  auto flat = [&](const void* p, long long ld) { return !p || (aligned_to(p, 16) && (o.M == 1 || ld % 8 == 0)); };
  e.vec = o.N % 8 == 0 && flat(e.y, e.ldy) && flat(e.z, e.ldz) && flat(e.res, e.ldr) && flat(e.bias, 0);
  if constexpr (!AMN)
    if (o.M <= kStreamMaxM) return launch_stream<BMN>(o, e, l.stream_partial, l.ctrl, l.timeout_ns, l.dev, l.n_sm, l.st);
  // 512 columns feed the tensor cores best; 256 where their finer grain saves more than that
  const long long rows = (o.M + 255) / 256, n_pairs = l.n_sm / 2;
  auto waves = [&](long long cols) { return (rows * ((o.N + cols - 1) / cols) + n_pairs - 1) / n_pairs; };
  if (100 * waves(512) * 2 <= 113 * waves(256))
    return launch_pair<2, AMN, BMN>(o, e, l.ctrl, l.timeout_ns, l.dev, l.n_sm, l.st);
  return launch_pair<1, AMN, BMN>(o, e, l.ctrl, l.timeout_ns, l.dev, l.n_sm, l.st);
}

template <class T>
static int backward(const psr_linear_shape* sh, const Sizes& s, const void* dy, const void* z, const void* x,
                    const void* w, void* dx, void* dw, void* db, uint8_t* ws, const Launch& l) {
  const bool act = sh->act != PSR_ACT_NONE;
  void* dz = act ? ws + s.dz : nullptr;
  int rc = PSR_OK;
  if (sh->M > 0 && (db || (act && (dx || dw)))) {
    const dim3 grid((unsigned)s.chunks, (unsigned)((sh->N + 255) / 256));
    if (grid.y > 65535) return PSR_ERR_UNSUPPORTED;
    dz_kernel<T><<<grid, 256, 0, l.st>>>(static_cast<const T*>(dy), s.ldy, static_cast<const T*>(z), s.ldz,
                                         static_cast<T*>(dz), s.lddz,
                                         db ? reinterpret_cast<float*>(ws + s.partial) : nullptr, sh->M, sh->N, sh->act);
    if ((rc = launch_status()) != PSR_OK) return rc;
  }
  if (db) {
    db_kernel<T><<<(unsigned)((sh->N + 255) / 256), 256, 0, l.st>>>(reinterpret_cast<float*>(ws + s.partial), s.chunks,
                                                                   sh->N, static_cast<T*>(db));
    if ((rc = launch_status()) != PSR_OK) return rc;
  }
  const void* g = act ? dz : dy;
  const long long ldg = act ? s.lddz : s.ldy;
  Epilogue e = {};
  e.half = sh->type == PSR_F16;
  e.ldy = sh->K;
  if (dx) {
    e.y = dx;
    if ((rc = product<T, false, true>({g, ldg, w, s.ldw, sh->M, sh->K, sh->N}, e, l)) != PSR_OK) return rc;
  }
  if (dw) {
    e.y = dw;
    if (sh->M == 0) {
      if (cudaMemsetAsync(dw, 0, (size_t)sh->N * sh->K * 2, l.st) != cudaSuccess) return PSR_ERR_CUDA;
    } else {
      rc = product<T, true, true>({g, ldg, x, s.ldx, sh->N, sh->K, sh->M}, e, l);
    }
  }
  return rc;
}

static int launch_of(void* workspace, const Sizes& s, int timeout_ms, void* stream, Launch& l) {
  const int rc = check_device(&l.n_sm);
  if (rc != PSR_OK) return rc;
  if (cudaGetDevice(&l.dev) != cudaSuccess) return PSR_ERR_CUDA;
  l.ctrl = static_cast<Ctrl*>(workspace);
  l.stream_partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + s.stream);
  l.timeout_ns = (unsigned long long)(timeout_ms > 0 ? timeout_ms : 2000) * 1000000ull;
  l.st = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(workspace, 0, sizeof(Ctrl), l.st) != cudaSuccess) {
    cudaGetLastError();
    return PSR_ERR_CUDA;
  }
  return PSR_OK;
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
  Launch l;
  if ((rc = launch_of(workspace, s, timeout_ms, stream, l)) != PSR_OK) return rc;
  Epilogue e = {};
  e.bias = bias; e.res = residual; e.y = y; e.z = z;
  e.ldr = s.ldr; e.ldy = s.ldy; e.ldz = s.ldz;
  e.act = sh->act;
  e.half = sh->type == PSR_F16;
  const Operands o = {x, s.ldx, w, s.ldw, sh->M, sh->N, sh->K};
  return sh->type == PSR_BF16 ? product<__nv_bfloat16, false, false>(o, e, l) : product<__half, false, false>(o, e, l);
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
  Launch l;
  if ((rc = launch_of(workspace, s, timeout_ms, stream, l)) != PSR_OK) return rc;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  return sh->type == PSR_BF16 ? backward<__nv_bfloat16>(sh, s, dy, z, x, w, dx, dw, db, ws, l)
                              : backward<__half>(sh, s, dy, z, x, w, dx, dw, db, ws, l);
}

}  // extern "C"
