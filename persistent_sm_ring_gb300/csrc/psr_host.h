// Shared by the layer operators (rotary positions, linear, 4-bit cache): host-side checks, element types, bounded waits
// and launches that follow one another.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/psr.h"
#include "psr_control.cuh"

namespace psr {

// The current device is an sm_103 one; its SM count.
inline int check_device(int* n_sm) {
  int dev = 0, major = 0, minor = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return PSR_ERR_CUDA;
  }
  if (major != 10 || minor != 3) return PSR_ERR_UNSUPPORTED;
  if (n_sm) *n_sm = sms;
  return PSR_OK;
}

inline bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Status of the launch just made.
inline int launch_status() { return cudaGetLastError() == cudaSuccess ? PSR_OK : PSR_ERR_CUDA; }

template <class T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }

template <class T>
__device__ __forceinline__ T from_f32(float v);  // round to nearest even
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }

// Bounded wait on a barrier: false after the timeout, or once another wait of the CTA has given up.  The control block's
// abort word is not consulted: it is cleared by the launch itself (clear_ctrl), while other CTAs already run.
// The clock is first read after 32 polls, most waits being shorter.
template <bool CL = false, class KP, class SC>
__device__ __forceinline__ bool wait_own(uint64_t* bar, uint32_t parity, const KP& p, SC* sc, uint32_t site) {
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (CL ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
    if (it % 32 == 0) {
      if (sc->abort) return false;
      const uint64_t now = globaltimer_ns();
      if (it == 32) {
        t0 = now;
      } else if (now - t0 > p.timeout_ns) {
        raise_error(p, site);
        sc->abort = 1;
        return false;
      }
    }
  }
}

// Wait for at most 100 ms, at the end of a kernel.
__device__ __forceinline__ void wait_last(uint64_t* bar, uint32_t parity) {
  uint64_t t0 = 0;
  for (uint32_t it = 1; !mbar_try_wait(bar, parity); ++it) {
    if (it % 32) continue;
    const uint64_t now = globaltimer_ns();
    if (it == 32) t0 = now;
    else if (now - t0 > 100000000ull) return;
  }
}

// The first kernel of a call clears the control block (a memset before it would cost a launch).  A wait of the same call
// can give up only a timeout later.
__device__ __forceinline__ void clear_ctrl(Ctrl* ctrl) {
  if (ctrl && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < sizeof(Ctrl) / 4)
    reinterpret_cast<uint32_t*>(ctrl)[threadIdx.x] = 0;
}

// Programmatic launches: let the next kernel's launch begin / wait for the whole previous kernel and its writes.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launch a kernel whose launch may begin while the previous one ends (it calls wait_previous before it reads).
template <class Kern, class P>
inline int launch_after(Kern kern, dim3 grid, int threads, const P& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) {
    cudaGetLastError();
    return PSR_ERR_CUDA;
  }
  return PSR_OK;
}

}  // namespace psr
