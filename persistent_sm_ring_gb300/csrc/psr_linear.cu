// The linear layer y = act(x w^T + bias) + residual and its gradients on sm_103a.
//
// The products are the tcgen05 kernels of psr_linear_mma.cuh.  A tensor map wants rows that start on 16-byte boundaries: an
// operand with others is copied into the workspace first (4100 columns: 0.09 ms of 0.21 at 8192 x 4096 x 4100).
#include <algorithm>
#include <cmath>
#include <cstring>

#include "psr_control.cuh"
#include "psr_host.h"
#include "psr_linear_mma.cuh"

namespace psr {
namespace linear {

// ------------------------------------------------------------------------------------------------
// One row of x, or a few with a small W: dot products on the fp32 units
// ------------------------------------------------------------------------------------------------
// Bound by reading W once.  A warp takes a row of W, a lane 16 bytes of it at a time (the warp 512 adjacent bytes), and asks for
// the next piece as it takes one, so that kAhead of them stay in flight; x comes from L1.  Against the tensor core kernels
// this has no tensor memory, barriers or partials to set up: 8192 x 8192 in 22.7 us (5.9 TB/s), where the streaming kernel takes
// 29; with groups of eight loads that are all used before the next are asked for 26.6, and 1024 x 8192 10.1 instead of 6.0.
// A few rows (a block row each) read W again from L2.  That is faster while the dot products fit on the SMs at once, up to
// kGemvDots of them and kGemvBytes of W in all (dot products / streaming: 8 x 1024 x 1024 5.2 / 5.5 us, 16 x 256 x 512 2.9 /
// 4.8; beyond, 16 x 1024 x 64 6.3 / 4.7 and 8 x 1024 x 4096 8.9 / 6.7).
constexpr long long kGemvDots = 8192, kGemvBytes = 32 << 20;

template <class T>
__global__ void __launch_bounds__(256)
    gemv_kernel(const T* __restrict__ x, long long ldx, const T* __restrict__ w, long long ldw, int N, int K,
                const __grid_constant__ Epilogue e, Ctrl* clear) {
  constexpr int kAhead = 8;
  constexpr bool kHalfType = std::is_same<T, __half>::value;
  clear_ctrl(clear);
  const int lane = threadIdx.x % 32;
  const int j = blockIdx.x * 8 + threadIdx.x / 32;
  if (j >= N) return;
  x += blockIdx.y * ldx;
  const T* row = w + (long long)j * ldw + lane * 8;
  float acc = 0.f;
  auto load = [&](int k) { return __ldcs(reinterpret_cast<const uint4*>(row + k)); };
  auto dot = [&](const uint4& v, int k) {
    const uint4 u = *reinterpret_cast<const uint4*>(x + k);
    const uint32_t a[4] = {u.x, u.y, u.z, u.w}, b[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float al, ah, bl, bh;
      unpack16(a[q], kHalfType, al, ah);
      unpack16(b[q], kHalfType, bl, bh);
      acc = fmaf(al, bl, acc);
      acc = fmaf(ah, bh, acc);
    }
  };
  int k = 0;
  if (256 * kAhead <= K) {
    uint4 v[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) v[a] = load(256 * a);
    for (; k + 512 * kAhead <= K; k += 256 * kAhead) {
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        dot(v[a], k + 256 * a + lane * 8);
        v[a] = load(k + 256 * (a + kAhead));
      }
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) dot(v[a], k + 256 * a + lane * 8);
    k += 256 * kAhead;
  }
  if (k < K) {  // the rest (K is a multiple of 8), all of it in flight at once
    uint4 v[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) v[a] = k + 256 * a + lane * 8 < K ? load(k + 256 * a) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (k + 256 * a + lane * 8 < K) dot(v[a], k + 256 * a + lane * 8);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (lane == 0) finish(e, blockIdx.y, j, acc);
}

template <class T>
static int launch_gemv(const Operands& o, const Epilogue& e, Launch& l) {
  gemv_kernel<T><<<dim3((unsigned)((o.N + 7) / 8), (unsigned)o.M), 256, 0, l.st>>>(
      static_cast<const T*>(o.a), o.lda, static_cast<const T*>(o.b), o.ldb, o.N, o.K, e, l.clear);
  l.clear = nullptr;
  return launch_status();
}

// ------------------------------------------------------------------------------------------------
// dz = dy act'(z), and the column sums of its unrounded values over chunks of rows
// ------------------------------------------------------------------------------------------------
// Memory bound (4100 x 8192 in 38 us, 5.3 TB/s).  A thread takes V adjacent columns (16 bytes where the rows allow it) of every
// eighth row of a chunk, two of them in flight (four took 2 % longer, eight 8 %: fewer blocks fit), the
// eight warps of a block join their sums in shared memory, and a second kernel joins the chunks in order: the sums do not
// depend on the order in which blocks run.
constexpr int kDzRows = 64;  // rows of a chunk

template <class T, int V>
__global__ void __launch_bounds__(256)
    dz_kernel(const T* __restrict__ dy, long long ldy, const T* __restrict__ z, long long ldz, T* __restrict__ dz,
              long long lddz, float* __restrict__ partial, int M, int N, int act, Ctrl* clear) {
  __shared__ float sums[8][32 * V];
  clear_ctrl(clear);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const uint32_t chunks = (M + kDzRows - 1) / kDzRows, cols = blockIdx.x / chunks, chunk = blockIdx.x - cols * chunks;
  const int j = (int)(cols * 32 + lane) * V;
  const long long i0 = (long long)chunk * kDzRows, i1 = i0 + kDzRows < M ? i0 + kDzRows : M;
  struct alignas(sizeof(T) * V) Vec { T v[V]; };
  float sum[V] = {};
  if (j < N) {
#pragma unroll 2
    for (long long i = i0 + warp; i < i1; i += 8) {
      Vec g = *reinterpret_cast<const Vec*>(dy + i * ldy + j), zz;
      if (act != PSR_ACT_NONE) zz = *reinterpret_cast<const Vec*>(z + i * ldz + j);
#pragma unroll
      for (int c = 0; c < V; ++c) {
        float f = to_f32(g.v[c]);
        if (act != PSR_ACT_NONE) f *= act_slope(act, to_f32(zz.v[c]));
        g.v[c] = from_f32<T>(f);
        sum[c] += f;
      }
      if (dz) *reinterpret_cast<Vec*>(dz + i * lddz + j) = g;
    }
  }
  if (!partial) return;
#pragma unroll
  for (int c = 0; c < V; ++c) sums[warp][lane * V + c] = sum[c];
  __syncthreads();
  for (int c = threadIdx.x; c < 32 * V; c += 256) {
    const int col = (int)cols * 32 * V + c;
    float f = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) f += sums[w][c];
    if (col < N) partial[(long long)chunk * N + col] = f;
  }
}

// Column sums over the chunks: eight warps take every eighth chunk of 32 columns.
template <class T>
__global__ void __launch_bounds__(256) db_kernel(const float* __restrict__ partial, int chunks, int N, T* db) {
  __shared__ float sums[8][32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, j = blockIdx.x * 32 + lane;
  float f = 0.f;
  if (j < N)
#pragma unroll 8
    for (int c = warp; c < chunks; c += 8) f += partial[(long long)c * N + j];
  sums[warp][lane] = f;
  __syncthreads();
  if (warp || j >= N) return;
  for (int w = 1; w < 8; ++w) f += sums[w][lane];
  db[j] = from_f32<T>(f);
}

// ------------------------------------------------------------------------------------------------
// Host side
// ------------------------------------------------------------------------------------------------
struct Sizes {
  long long ldx, ldw, ldr, ldy, ldz;
  int chunks;     // row chunks of the column sums
  long long lddz; // row stride of dz in the workspace
  size_t sums, sums_bytes, dz, partial, total;
  size_t x, w, dy;  // aligned copies of operands (0: the tensor's own rows are)
};

static int launch_of(void* workspace, const Sizes& s, int timeout_ms, void* stream, Launch& l) {
  const int rc = check_device(&l.n_sm);
  if (rc != PSR_OK) return rc;
  if (cudaGetDevice(&l.dev) != cudaSuccess) return PSR_ERR_CUDA;
  l.ctrl = l.clear = static_cast<Ctrl*>(workspace);
  l.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + s.sums);
  l.partial_bytes = s.sums_bytes;
  l.timeout_ns = (unsigned long long)(timeout_ms > 0 ? timeout_ms : 2000) * 1000000ull;
  l.st = static_cast<cudaStream_t>(stream);
  return PSR_OK;
}

// An operand that is not copied starts on a 16-byte boundary.
static bool placed(const void* x, size_t copy) { return copy || aligned_to(x, 16); }

// A call that launched nothing still leaves a cleared control block for psr_get_stats.
static int clear_rest(const Launch& l) {
  if (!l.clear || cudaMemsetAsync(l.clear, 0, sizeof(Ctrl), l.st) == cudaSuccess) return PSR_OK;
  cudaGetLastError();
  return PSR_ERR_CUDA;
}

static size_t au(size_t x) { return (x + 255) / 256 * 256; }

static int sizes(const psr_linear_shape* sh, bool backward, Sizes& s) {
  if (!sh) return PSR_ERR_ARG;
  if (sh->M < 0 || sh->N < 1 || sh->K < 1) return PSR_ERR_ARG;
  if (sh->act < PSR_ACT_NONE || sh->act > PSR_ACT_SILU) return PSR_ERR_ARG;
  if (sh->type != PSR_BF16 && sh->type != PSR_F16) return PSR_ERR_ARG;
  if (sh->odd < 0 || sh->odd > 7) return PSR_ERR_ARG;
  if (sh->M > 1 << 30 || sh->N > 1 << 30 || sh->K > 1 << 30) return PSR_ERR_UNSUPPORTED;
  auto ld = [](long long given, long long contiguous) { return given == 0 ? contiguous : given; };
  s.ldx = ld(sh->ldx, sh->K); s.ldw = ld(sh->ldw, sh->K);
  s.ldr = ld(sh->ldr, sh->N); s.ldy = ld(sh->ldy, sh->N); s.ldz = ld(sh->ldz, sh->N);
  if (s.ldx < sh->K || s.ldw < sh->K || s.ldr < sh->N || s.ldy < sh->N || s.ldz < sh->N) return PSR_ERR_ARG;
  s.chunks = (sh->M + kDzRows - 1) / kDzRows;
  s.lddz = (sh->N + 7) / 8 * 8;
  size_t off = 256;  // control block
  s.sums = off;      // fp32 partials of one split product at a time
  if (backward) {
    const size_t x = partial_bytes(sh->M, sh->K, sh->N, false), w = partial_bytes(sh->N, sh->K, sh->M, true);
    s.sums_bytes = x > w ? x : w;
  } else {
    s.sums_bytes = partial_bytes(sh->M, sh->N, sh->K, false);
  }
  off = au(off + s.sums_bytes);
  s.dz = s.partial = off;
  if (backward) {
    if (sh->act != PSR_ACT_NONE) off = au(off + (size_t)sh->M * s.lddz * 2);
    s.partial = off;
    off = au(off + (size_t)s.chunks * sh->N * 4);
  }
  auto copy = [&](int odd, long long ld, int rows, int cols) {
    const size_t at = off;
    if (!(sh->odd & odd) && (rows <= 1 || ld % 8 == 0)) return (size_t)0;
    off = au(off + (size_t)rows * ((cols + 7ll) / 8 * 8) * 2);
    return at;
  };
  s.x = copy(PSR_LINEAR_ODD_X, s.ldx, sh->M, sh->K);
  s.w = copy(PSR_LINEAR_ODD_W, s.ldw, sh->N, sh->K);
  s.dy = backward && sh->act == PSR_ACT_NONE ? copy(PSR_LINEAR_ODD_DY, s.ldy, sh->M, sh->N) : 0;
  s.total = off;
  return PSR_OK;
}

// C = A B^T with A [M][K] (or AMN: [K][M]) and B [N][K] (or BMN: [K][N]).  W is the operand that streams when
// there are few rows of A.
template <class T, bool AMN, bool BMN>
static int product(const Operands& o, Epilogue e, Launch& l) {
  if (o.M == 0) return PSR_OK;
  if (!mappable(o.a, AMN ? o.K : o.M, o.lda) || !mappable(o.b, BMN ? o.K : o.N, o.ldb)) return PSR_ERR_UNSUPPORTED;
  auto flat = [&](const void* p, long long ld) { return !p || (aligned_to(p, 16) && (o.M == 1 || ld % 8 == 0)); };
  e.vec = o.N % 8 == 0 && flat(e.y, e.ldy) && flat(e.z, e.ldz) && flat(e.res, e.ldr) && flat(e.bias, 0);
  if constexpr (!AMN && !BMN)
    if (o.K % 8 == 0 && (o.M == 1 || (o.M <= 16 && (long long)o.M * o.N <= kGemvDots && 2ll * o.M * o.N * o.K <= kGemvBytes)))
      return launch_gemv<T>(o, e, l);
  if constexpr (!AMN)
    if (streams(o.M, o.N, o.K)) return launch_stream<BMN>(o, e, l);
  const Split split = split_of(o.M, o.N, o.K);
  constexpr bool kHalfType = std::is_same<T, __half>::value;
  const double more = (e.act > PSR_ACT_RELU ? 3200.0 : 0.0) + (e.z ? 2600.0 : 0.0) + (e.res ? 3200.0 : 0.0) + (e.bias ? 1000.0 : 0.0);
  return launch_pair<AMN, BMN, kHalfType>(o, e, wide_tiles<AMN, BMN>(o, more, split, l.n_sm / 2), split, l);
}

template <class T>
static int backward(const psr_linear_shape* sh, const Sizes& s, const void* dy, const void* z, const void* x,
                    const void* w, void* dx, void* dw, void* db, uint8_t* ws, Launch& l) {
  const bool act = sh->act != PSR_ACT_NONE;
  void* dz = act ? ws + s.dz : nullptr;
  int rc = PSR_OK;
  if (sh->M > 0 && (db || (act && (dx || dw)))) {
    T* out = dx || dw ? static_cast<T*>(dz) : nullptr;
    float* partial = db ? reinterpret_cast<float*>(ws + s.partial) : nullptr;
    auto flat = [&](const void* p, long long ld) { return !p || (aligned_to(p, 16) && (sh->M == 1 || ld % 8 == 0)); };
    const bool vec = sh->N % 8 == 0 && flat(dy, s.ldy) && flat(z, s.ldz);
    const int wide = 32 * (vec ? 8 : 1);  // columns of a block
    const long long blocks = (sh->N + wide - 1) / wide * (long long)s.chunks;  // the chunks of the same columns follow one another
    if (blocks >= (1ll << 31)) return PSR_ERR_UNSUPPORTED;
    const unsigned grid = (unsigned)blocks;
    const T *dy_t = static_cast<const T*>(dy), *z_t = static_cast<const T*>(z);
    if (vec) dz_kernel<T, 8><<<grid, 256, 0, l.st>>>(dy_t, s.ldy, z_t, s.ldz, out, s.lddz, partial, sh->M, sh->N, sh->act, l.clear);
    else dz_kernel<T, 1><<<grid, 256, 0, l.st>>>(dy_t, s.ldy, z_t, s.ldz, out, s.lddz, partial, sh->M, sh->N, sh->act, l.clear);
    l.clear = nullptr;
    if ((rc = launch_status()) != PSR_OK) return rc;
  }
  if (db) {
    db_kernel<T><<<(unsigned)((sh->N + 31) / 32), 256, 0, l.st>>>(reinterpret_cast<float*>(ws + s.partial), s.chunks, sh->N,
                                                                 static_cast<T*>(db));
    if ((rc = launch_status()) != PSR_OK) return rc;
  }
  const void* g = act ? dz : dy;
  long long ldg = act ? s.lddz : s.ldy, ldw = s.ldw, ldx = s.ldx;
  if (sh->M > 0) {
    if ((dx || dw) && (rc = align(g, ldg, s.dy, sh->M, sh->N, ws, l)) != PSR_OK) return rc;
    if (dx && (rc = align(w, ldw, s.w, sh->N, sh->K, ws, l)) != PSR_OK) return rc;
    if (dw && (rc = align(x, ldx, s.x, sh->M, sh->K, ws, l)) != PSR_OK) return rc;
  }
  Epilogue e = {};
  e.half = sh->type == PSR_F16;
  e.ldy = sh->K;
  if (dx) {
    e.y = dx;
    if ((rc = product<T, false, true>({g, ldg, w, ldw, sh->M, sh->K, sh->N}, e, l)) != PSR_OK) return rc;
  }
  if (dw) {
    e.y = dw;
    if (sh->M == 0) {
      if (cudaMemsetAsync(dw, 0, (size_t)sh->N * sh->K * 2, l.st) != cudaSuccess) return PSR_ERR_CUDA;
    } else {
      rc = product<T, true, true>({g, ldg, x, ldx, sh->N, sh->K, sh->M}, e, l);
    }
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
  if (sizes(sh, backward != 0, s) != PSR_OK) return 0;
  return s.total;
}

int psr_linear(const psr_linear_shape* sh, const void* x, const void* w, const void* bias, const void* residual,
               void* y, void* z, void* workspace, size_t ws_bytes, int timeout_ms, void* stream) {
  if (!sh || !x || !w || !y || !workspace) return PSR_ERR_ARG;
  if (!aligned_to(workspace, 256)) return PSR_ERR_ARG;
  for (const void* ptr : {x, w, bias, residual, (const void*)y, (const void*)z})
    if (!aligned_to(ptr, 2)) return PSR_ERR_ARG;
  Sizes s;
  int rc = sizes(sh, false, s);
  if (rc != PSR_OK) return rc;
  if (ws_bytes < s.total || !placed(x, s.x) || !placed(w, s.w)) return PSR_ERR_ARG;
  Launch l;
  if ((rc = launch_of(workspace, s, timeout_ms, stream, l)) != PSR_OK) return rc;
  Epilogue e = {};
  e.bias = bias; e.res = residual; e.y = y; e.z = z;
  e.ldr = s.ldr; e.ldy = s.ldy; e.ldz = s.ldz;
  e.act = sh->act;
  e.half = sh->type == PSR_F16;
  if ((rc = align(x, s.ldx, s.x, sh->M, sh->K, workspace, l)) != PSR_OK) return rc;
  if (sh->M > 0 && (rc = align(w, s.ldw, s.w, sh->N, sh->K, workspace, l)) != PSR_OK) return rc;
  const Operands o = {x, s.ldx, w, s.ldw, sh->M, sh->N, sh->K};
  rc = sh->type == PSR_BF16 ? product<__nv_bfloat16, false, false>(o, e, l) : product<__half, false, false>(o, e, l);
  return rc != PSR_OK ? rc : clear_rest(l);
}

int psr_linear_bwd(const psr_linear_shape* sh, const void* dy, const void* z, const void* x, const void* w, void* dx,
                   void* dw, void* db, void* workspace, size_t ws_bytes, int timeout_ms, void* stream) {
  if (!sh || !dy || !x || !w || !workspace || (sh->act != PSR_ACT_NONE && !z)) return PSR_ERR_ARG;
  if (!aligned_to(workspace, 256)) return PSR_ERR_ARG;
  for (const void* ptr : {dy, z, x, w, (const void*)dx, (const void*)dw, (const void*)db})
    if (!aligned_to(ptr, 2)) return PSR_ERR_ARG;
  Sizes s;
  int rc = sizes(sh, true, s);
  if (rc != PSR_OK) return rc;
  if (ws_bytes < s.total || !placed(x, s.x) || !placed(w, s.w)) return PSR_ERR_ARG;
  if (sh->act == PSR_ACT_NONE && !placed(dy, s.dy)) return PSR_ERR_ARG;
  Launch l;
  if ((rc = launch_of(workspace, s, timeout_ms, stream, l)) != PSR_OK) return rc;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  rc = sh->type == PSR_BF16 ? backward<__nv_bfloat16>(sh, s, dy, z, x, w, dx, dw, db, ws, l)
                            : backward<__half>(sh, s, dy, z, x, w, dx, dw, db, ws, l);
  return rc != PSR_OK ? rc : clear_rest(l);
}

}  // extern "C"
