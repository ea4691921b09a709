// Rotary positions of Q and K on sm_103a: each pair of columns of a row turned by its position's angle.
//
// The angle of pair i at position p is p * f_i.  In fp32 that product has lost every digit of its
// fraction of a turn once p reaches millions, so the frequencies are held as turns per position in 64-bit
// fixed point: one 64-bit integer product is the angle modulo a turn, exactly, for positive and negative
// positions alike, and its top 32 bits (2^-32 of a turn) go to sincospi.
#include <cmath>

#include "psr_host.h"

namespace psr {
namespace rotary {

struct Operand {
  const void* in;
  void* out;
  psr_strides si, so;
};

struct Params {
  Operand q, k;
  const uint64_t* table;
  const int64_t* positions;
  long long positions_b, offset;
  int B, Hq, Hkv, S, d, rot;
  int half;  // rows of a half-chunk of load-balanced shards (S / (2P)), 0: rows are in order
  int P;
  int chunk;  // heads that a thread goes through
  float amplitude, sign;
};

// Global position of row s: load-balanced shard r holds half-chunks r and 2P-1-r.
__device__ __forceinline__ long long position(const Params& p, int b, int s) {
  if (p.positions) return p.positions[b * p.positions_b + s];
  long long g = s;
  if (p.half) {
    const int c = s / p.half, r = c / 2, i = s - c * p.half;
    g = (long long)((c & 1) ? 2 * p.P - 1 - r : r) * p.half + i;
  }
  return p.offset + g;
}

// cos and sin (times the amplitude, sin signed) of a pair at a position
__device__ __forceinline__ void turn(const Params& p, long long pos, uint64_t freq, float& c, float& s) {
  const uint64_t t = (uint64_t)pos * freq;
  sincospif((float)(int32_t)(t >> 32) * 4.656612873077393e-10f, &s, &c);  // half turns: 2^-31 of the top word
  c *= p.amplitude;
  s *= p.sign * p.amplitude;
}

// Memory bound: every element is read and written once.  A thread takes V pairs of a row (two vectors of V elements, 16 bytes
// each where the layout allows it) or V copied columns, computes their cosines and sines once, and goes through the heads
// of its chunk with kAhead of them in flight.  Q (32 heads) and K (8) of 32768 rows, d = 128, bf16: 106 us, 6.3 TB/s; with
// four heads in flight the registers leave two blocks to an SM and it takes 158 us, with 8-byte vectors 182.
constexpr int kAhead = 2;

template <class T, bool INTER, int V>
__global__ void __launch_bounds__(256, 4) rotary_kernel(const __grid_constant__ Params p) {
  struct alignas(sizeof(T) * V) Vec { T e[V]; };
  const int pairs = p.rot / 2 / V, units = pairs + (p.d - p.rot) / V;
  const long long i = blockIdx.x * 256ll + threadIdx.x, rows = (long long)p.B * p.S;
  const long long r = i / units;
  if (r >= rows) return;
  const int u = (int)(i - r * units), b = (int)(r / p.S), s = (int)(r - (long long)b * p.S);
  const int h0 = blockIdx.y * p.chunk, h1 = min(h0 + p.chunk, p.Hq + p.Hkv);
  const bool turned = u < pairs;
  const int c1 = !turned ? p.rot + (u - pairs) * V : INTER ? 2 * V * u : V * u;
  const int c2 = INTER ? c1 + V : c1 + p.rot / 2;
  float cs[V], sn[V];
  if (turned) {
    const long long pos = position(p, b, s);
#pragma unroll
    for (int e = 0; e < V; ++e) turn(p, pos, p.table[u * V + e], cs[e], sn[e]);
  }
  auto at = [&](int h, bool out) -> T* {
    const bool q = h < p.Hq;
    const Operand& o = q ? p.q : p.k;
    const psr_strides& st = out ? o.so : o.si;
    return static_cast<T*>(const_cast<void*>(out ? o.out : o.in)) + b * st.b + (q ? h : h - p.Hq) * st.h + s * st.s;
  };
  for (int h = h0; h < h1; h += kAhead) {
    Vec x1[kAhead], x2[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (h + a >= h1) break;
      const T* x = at(h + a, false);
      x1[a] = *reinterpret_cast<const Vec*>(x + c1);
      if (turned) x2[a] = *reinterpret_cast<const Vec*>(x + c2);
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (h + a >= h1) break;
      T* y = at(h + a, true);
      if (!turned) {
        *reinterpret_cast<Vec*>(y + c1) = x1[a];
        continue;
      }
      Vec y1, y2;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        // pair e: element e of either vector, or elements 2e and 2e + 1 of the two taken as one
        const float f1 = to_f32(!INTER ? x1[a].e[e] : 2 * e < V ? x1[a].e[2 * e % V] : x2[a].e[2 * e % V]);
        const float f2 = to_f32(!INTER ? x2[a].e[e] : 2 * e + 1 < V ? x1[a].e[(2 * e + 1) % V] : x2[a].e[(2 * e + 1) % V]);
        const T g1 = from_f32<T>(f1 * cs[e] - f2 * sn[e]), g2 = from_f32<T>(f2 * cs[e] + f1 * sn[e]);
        if (!INTER) {
          y1.e[e] = g1;
          y2.e[e] = g2;
        } else {
          (2 * e < V ? y1 : y2).e[2 * e % V] = g1;
          (2 * e + 1 < V ? y1 : y2).e[(2 * e + 1) % V] = g2;
        }
      }
      *reinterpret_cast<Vec*>(y + c1) = y1;
      *reinterpret_cast<Vec*>(y + c2) = y2;
    }
  }
}

template <class T, bool INTER, int V>
static int launch_v(Params& p, int n_sm, cudaStream_t st) {
  const long long threads = (long long)p.B * p.S * (p.rot / 2 / V + (p.d - p.rot) / V), blocks = (threads + 255) / 256;
  const int H = p.Hq + p.Hkv;
  // a chunk of heads shares the cosines and sines; shorter ones where there are few rows
  p.chunk = 32;
  while (p.chunk > 1 && blocks * ((H + p.chunk - 1) / p.chunk) < 8 * n_sm) p.chunk /= 2;
  const int chunks = (H + p.chunk - 1) / p.chunk;
  if (blocks >= (1ll << 31) || chunks > 65535) return PSR_ERR_UNSUPPORTED;
  rotary_kernel<T, INTER, V><<<dim3((unsigned)blocks, (unsigned)chunks), 256, 0, st>>>(p);
  return launch_status();
}

template <class T, bool INTER>
static int launch_t(Params& p, int n_sm, cudaStream_t st) {
  // the longest vectors that every row, column group and pair of column groups starts on a boundary of
  auto fits = [&](int v) {
    auto even = [&](const Operand& o, int H) {
      for (const psr_strides* t : {&o.si, &o.so})
        if ((p.B > 1 && t->b % v) || (H > 1 && t->h % v) || (p.S > 1 && t->s % v)) return false;
      return aligned_to(o.in, v * sizeof(T)) && aligned_to(o.out, v * sizeof(T));
    };
    return (INTER ? p.rot % (2 * v) == 0 : p.rot / 2 % v == 0) && (p.d - p.rot) % v == 0 && even(p.q, p.Hq) &&
           (p.Hkv == 0 || even(p.k, p.Hkv));
  };
  constexpr int kMost = 16 / sizeof(T);
  if (fits(kMost)) return launch_v<T, INTER, kMost>(p, n_sm, st);
  if (kMost > 4 && fits(4)) return launch_v<T, INTER, kMost < 4 ? kMost : 4>(p, n_sm, st);
  if (fits(2)) return launch_v<T, INTER, 2>(p, n_sm, st);
  return launch_v<T, INTER, 1>(p, n_sm, st);
}

template <class T>
static int launch(Params& p, bool inter, int n_sm, cudaStream_t st) {
  return inter ? launch_t<T, true>(p, n_sm, st) : launch_t<T, false>(p, n_sm, st);
}

}  // namespace rotary
}  // namespace psr

using namespace psr;
using namespace psr::rotary;

extern "C" {

int psr_rotary_table(int rot, double base, int scaling, double factor, double original_length, double beta_fast,
                     double beta_slow, uint64_t* table) {
  if (!table || rot < 2 || rot > 1024 || rot % 2 != 0 || !(base > 1.0) || !std::isfinite(base)) return PSR_ERR_ARG;
  if (scaling < PSR_ROTARY_PLAIN || scaling > PSR_ROTARY_BY_PARTS) return PSR_ERR_ARG;
  if (scaling != PSR_ROTARY_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return PSR_ERR_ARG;
  double low = 0, high = 0;
  const double two_pi = 6.283185307179586476925;
  if (scaling == PSR_ROTARY_BY_PARTS) {
    if (!(original_length >= 1.0) || !std::isfinite(original_length) || !(beta_slow > 0.0) ||
        !(beta_fast > beta_slow) || !std::isfinite(beta_fast))
      return PSR_ERR_ARG;
    // the pair index (as a real number) that makes `turns` turns over the original length
    auto pair_of = [&](double turns) {
      return rot * std::log(original_length / (turns * two_pi)) / (2.0 * std::log(base));
    };
    low = std::floor(pair_of(beta_fast));
    if (low < 0) low = 0;
    high = std::ceil(pair_of(beta_slow));
    if (high > rot - 1) high = rot - 1;
  }
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (scaling == PSR_ROTARY_LINEAR) f /= factor;
    if (scaling == PSR_ROTARY_BY_PARTS) {
      const double span = high - low > 0.001 ? high - low : 0.001;
      double ramp = (i - low) / span;
      ramp = ramp < 0 ? 0 : ramp > 1 ? 1 : ramp;
      f = f * (1.0 - ramp) + f / factor * ramp;
    }
    table[i] = (uint64_t)(f / two_pi * 18446744073709551616.0);  // f <= 1 radian: below 2^62
  }
  return PSR_OK;
}

int psr_rotary(const psr_rotary_shape* sh, const void* q, const psr_strides* qs, void* q_out, const psr_strides* qos,
               const void* k, const psr_strides* ks, void* k_out, const psr_strides* kos, const uint64_t* table,
               const int64_t* positions, long long positions_b, void* stream) {
  if (!sh || !q || !qs || !q_out || !qos || !table) return PSR_ERR_ARG;
  if (sh->B < 0 || sh->S < 0 || sh->Hq < 1 || sh->Hkv < 0 || sh->P < 1) return PSR_ERR_ARG;
  if (sh->Hkv > 0 && (!k || !ks || !k_out || !kos)) return PSR_ERR_ARG;
  if (sh->d < 1 || sh->d > 1024 || sh->rot < 2 || sh->rot > sh->d || sh->rot % 2 != 0) return PSR_ERR_ARG;
  if (sh->type < PSR_BF16 || sh->type > PSR_F32 || sh->causal < 0 || sh->causal > PSR_CAUSAL_BALANCED) return PSR_ERR_ARG;
  if (sh->S % sh->P != 0) return PSR_ERR_UNSUPPORTED;
  const bool balanced = sh->causal == PSR_CAUSAL_BALANCED && !positions;
  if (balanced && (sh->S / sh->P) % 2 != 0) return PSR_ERR_UNSUPPORTED;
  const size_t es = sh->type == PSR_F32 ? 4 : 2;
  if (!aligned_to(q, es) || !aligned_to(q_out, es) || !aligned_to(table, 8) || !aligned_to(positions, 8)) return PSR_ERR_ARG;
  if (sh->Hkv > 0 && (!aligned_to(k, es) || !aligned_to(k_out, es))) return PSR_ERR_ARG;
  int n_sm = 0;
  const int rc = check_device(&n_sm);
  if (rc != PSR_OK) return rc;
  if (sh->B == 0 || sh->S == 0) return PSR_OK;

  Params p = {};
  p.q = {q, q_out, *qs, *qos};
  if (sh->Hkv > 0) p.k = {k, k_out, *ks, *kos};
  p.table = table;
  p.positions = positions;
  p.positions_b = positions_b;
  p.offset = sh->offset;
  p.B = sh->B; p.Hq = sh->Hq; p.Hkv = sh->Hkv; p.S = sh->S; p.d = sh->d; p.rot = sh->rot;
  p.P = sh->P;
  p.half = balanced ? sh->S / sh->P / 2 : 0;
  p.amplitude = sh->amplitude;
  p.sign = sh->inverse ? -1.0f : 1.0f;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (sh->type) {
    case PSR_BF16: return launch<__nv_bfloat16>(p, sh->interleaved != 0, n_sm, st);
    case PSR_F16: return launch<__half>(p, sh->interleaved != 0, n_sm, st);
    default: return launch<float>(p, sh->interleaved != 0, n_sm, st);
  }
}

}  // extern "C"
