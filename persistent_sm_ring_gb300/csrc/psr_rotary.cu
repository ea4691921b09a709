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

template <class T, bool INTER>
__global__ void rotary_kernel(const Params p) {
  const int units = p.rot / 2 + (p.d - p.rot);  // pairs, then copied columns
  const int H = p.Hq + p.Hkv;
  const long long n = (long long)p.B * p.S * H * units;
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
    const int u = (int)(i % units);
    long long r = i / units;
    const int h = (int)(r % H);
    r /= H;
    const int s = (int)(r % p.S), b = (int)(r / p.S);
    const Operand& o = h < p.Hq ? p.q : p.k;
    const int hh = h < p.Hq ? h : h - p.Hq;
    const T* x = static_cast<const T*>(o.in) + b * o.si.b + hh * o.si.h + s * o.si.s;
    T* y = static_cast<T*>(o.out) + b * o.so.b + hh * o.so.h + s * o.so.s;
    if (u >= p.rot / 2) {
      const int c = p.rot / 2 + u;
      y[c] = x[c];
      continue;
    }
    const int c1 = INTER ? 2 * u : u, c2 = INTER ? 2 * u + 1 : u + p.rot / 2;
    float cs, sn;
    turn(p, position(p, b, s), p.table[u], cs, sn);
    const float x1 = to_f32(x[c1]), x2 = to_f32(x[c2]);
    y[c1] = from_f32<T>(x1 * cs - x2 * sn);
    y[c2] = from_f32<T>(x2 * cs + x1 * sn);
  }
}

template <class T>
static int launch(const Params& p, bool inter, int n_sm, cudaStream_t st) {
  const long long n = (long long)p.B * p.S * (p.Hq + p.Hkv) * (p.rot / 2 + (p.d - p.rot));
  long long blocks = (n + 255) / 256;
  if (blocks > n_sm * 64) blocks = n_sm * 64;
  if (inter) rotary_kernel<T, true><<<(unsigned)blocks, 256, 0, st>>>(p);
  else rotary_kernel<T, false><<<(unsigned)blocks, 256, 0, st>>>(p);
  return launch_status();
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
