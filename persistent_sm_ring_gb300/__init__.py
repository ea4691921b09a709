"""persistent_sm_ring_gb300: Ring Attention forward on one GB300 (sm_103a).

Thin Python binding over the C ABI of ``libpsr.so`` (declared in
``include/psr.h``).  It only marshals arguments: every step of the ring
(staging, readiness flags, the tcgen05 FlashAttention pass, the LSE-exact
merge, the on-GPU partition controller) runs in the library's CUDA kernel.
The layer around the ring (rotary positions, linear with its gradients, a
4-bit KV cache with its attention) is bound at the end of the file.
PyTorch supplies device memory and streams.  There is no fallback: if the
library is missing or the device is not an sm_103 GPU, calls raise.
"""
from __future__ import annotations

import ctypes
import os
import threading

from .build import LIB, LIB_PAIRS, LIB_TRACE, build as _build

__all__ = ["build", "load", "Shape", "AgShape", "RsShape", "Partition", "Stats", "ring_attn_fwd", "ring_attn_fwd_host",
           "workspace_bytes", "ag_gemm", "ag_gemm_workspace_bytes", "gemm_rs", "gemm_rs_workspace_bytes",
           "ring_attn_bwd", "ring_attn_bwd_workspace_bytes",
           "rotary_table", "rotary", "rotary_bwd", "linear", "linear_bwd", "linear_workspace_bytes",
           "kv4_cache", "kv4_append", "kv4_read", "kv4_attn", "kv4_attn_workspace_bytes",
           "get_stats", "get_trajectory", "controller_target", "num_ctas", "status_string", "PsrError",
           "STATIC", "ADAPTIVE", "FAULT_NONE", "FAULT_DROP_FIRST_FLAG", "FAULT_SLOW_STAGING", "CAUSAL",
           "CAUSAL_BALANCED"]

OK, ERR_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT = 0, 1, 2, 3, 4
STATIC, ADAPTIVE = 0, 1
FAULT_NONE, FAULT_DROP_FIRST_FLAG, FAULT_SLOW_STAGING = 0, 1, 2
CAUSAL, CAUSAL_BALANCED = 1, 2

EXPORTED = ("psr_workspace_bytes", "psr_ring_attn_fwd", "psr_ring_attn_fwd_host", "psr_get_stats",
            "psr_get_trajectory", "psr_controller_target", "psr_status_string", "psr_num_ctas",
            "psr_ring_attn_fwd_noalloc", "psr_noalloc_get_stats", "psr_ag_gemm_workspace_bytes", "psr_ag_gemm", "psr_gemm_rs_workspace_bytes",
            "psr_gemm_rs", "psr_ring_attn_bwd_workspace_bytes", "psr_ring_attn_bwd",
            "psr_rotary_table", "psr_rotary", "psr_linear_workspace_bytes", "psr_linear", "psr_linear_bwd",
            "psr_kv4_cache_bytes", "psr_kv4_append", "psr_kv4_read", "psr_kv4_attn_workspace_bytes", "psr_kv4_attn")

BF16, F16, F32 = 0, 1, 2
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
ROTARY_SCALINGS = {"plain": 0, "linear": 1, "by_parts": 2}


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("S", ctypes.c_int),
                ("P", ctypes.c_int), ("d", ctypes.c_int), ("causal", ctypes.c_int), ("scale", ctypes.c_float)]


class AgShape(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int), ("K", ctypes.c_int), ("Ns", ctypes.c_int), ("P", ctypes.c_int)]


class RsShape(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int), ("N", ctypes.c_int), ("Ks", ctypes.c_int), ("P", ctypes.c_int)]


class Strides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_longlong), ("h", ctypes.c_longlong), ("s", ctypes.c_longlong)]


class RotaryShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("S", ctypes.c_int),
                ("P", ctypes.c_int), ("d", ctypes.c_int), ("causal", ctypes.c_int), ("rot", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("inverse", ctypes.c_int), ("type", ctypes.c_int),
                ("amplitude", ctypes.c_float), ("offset", ctypes.c_longlong)]


class LinearShape(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int), ("N", ctypes.c_int), ("K", ctypes.c_int), ("act", ctypes.c_int),
                ("type", ctypes.c_int), ("ldx", ctypes.c_longlong), ("ldw", ctypes.c_longlong),
                ("ldr", ctypes.c_longlong), ("ldy", ctypes.c_longlong), ("ldz", ctypes.c_longlong), ("odd", ctypes.c_int)]


class Kv4Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("S", ctypes.c_int),
                ("d", ctypes.c_int), ("page", ctypes.c_int), ("n_pages", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("type", ctypes.c_int), ("scale", ctypes.c_float)]


class Partition(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int), ("n_staging", ctypes.c_int), ("n_min", ctypes.c_int),
                ("n_max", ctypes.c_int), ("fault", ctypes.c_int), ("timeout_ms", ctypes.c_int)]


class Stats(ctypes.Structure):
    _fields_ = [("status", ctypes.c_int), ("error_site", ctypes.c_int), ("n_cta", ctypes.c_int),
                ("n_s_initial", ctypes.c_int), ("n_s_final", ctypes.c_int), ("n_s_min", ctypes.c_int),
                ("n_s_max", ctypes.c_int), ("traj_len", ctypes.c_int),
                ("staging_cycles", ctypes.c_ulonglong), ("compute_cycles", ctypes.c_ulonglong),
                ("staging_tasks", ctypes.c_ulonglong), ("compute_items", ctypes.c_ulonglong),
                ("compute_tiles", ctypes.c_ulonglong), ("staging_bytes", ctypes.c_ulonglong),
                ("role_switches", ctypes.c_ulonglong), ("idle_polls", ctypes.c_ulonglong),
                ("trace_softmax_wait", ctypes.c_ulonglong), ("trace_softmax_busy", ctypes.c_ulonglong),
                ("trace_mma_issue", ctypes.c_ulonglong), ("trace_mma_wait_kv", ctypes.c_ulonglong),
                ("trace_producer_wait_empty", ctypes.c_ulonglong), ("trace_producer_wait_flag", ctypes.c_ulonglong)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class PsrError(RuntimeError):
    def __init__(self, status, where=""):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


_lib = None
_lock = threading.Lock()


def build(force: bool = False, trace: bool = False, variant: str = "") -> str:
    """Compile libpsr.so in-tree for sm_103a, or a variant: "trace" (trace=True; cycle-tracing
    libpsr_trace.so) or "pairs" (libpsr_pairs.so, CTA-pair compute units for d = 128)."""
    return _build(force=force, trace=trace, variant=variant)


def load(trace: bool = False, variant: str = "") -> ctypes.CDLL:
    """Load libpsr.so (or the variant built by build(variant=...)); raises if it has not been built
    (no fallback path exists).

    One library per process: the first call decides which."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = LIB_TRACE if (trace or variant == "trace") else (LIB_PAIRS if variant == "pairs" else LIB)
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: run persistent_sm_ring_gb300.build() (nvcc, sm_103a) first")
        lib = ctypes.CDLL(path)
        vp, sz = ctypes.c_void_p, ctypes.c_size_t
        P_shape, P_part = ctypes.POINTER(Shape), ctypes.POINTER(Partition)
        lib.psr_workspace_bytes.argtypes = [P_shape]
        lib.psr_workspace_bytes.restype = sz
        lib.psr_ring_attn_fwd.argtypes = [P_shape, vp, vp, vp, vp, vp, vp, sz, P_part, vp]
        lib.psr_ring_attn_fwd.restype = ctypes.c_int
        lib.psr_ring_attn_fwd_host.argtypes = [P_shape, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, P_part, vp]
        lib.psr_ring_attn_fwd_host.restype = ctypes.c_int
        lib.psr_get_stats.argtypes = [vp, ctypes.POINTER(Stats), vp]
        lib.psr_get_stats.restype = ctypes.c_int
        lib.psr_get_trajectory.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32), ctypes.c_int, vp]
        lib.psr_get_trajectory.restype = ctypes.c_int
        lib.psr_controller_target.argtypes = [ctypes.c_int, ctypes.c_double, ctypes.c_double, ctypes.c_double,
                                              ctypes.c_double, ctypes.c_int, ctypes.c_int]
        lib.psr_controller_target.restype = ctypes.c_int
        lib.psr_status_string.argtypes = [ctypes.c_int]
        lib.psr_status_string.restype = ctypes.c_char_p
        P_ag = ctypes.POINTER(AgShape)
        lib.psr_ag_gemm_workspace_bytes.argtypes = [P_ag]
        lib.psr_ag_gemm_workspace_bytes.restype = sz
        lib.psr_ag_gemm.argtypes = [P_ag, vp, vp, vp, vp, sz, P_part, vp]
        lib.psr_ag_gemm.restype = ctypes.c_int
        lib.psr_ring_attn_bwd_workspace_bytes.argtypes = [ctypes.POINTER(Shape)]
        lib.psr_ring_attn_bwd_workspace_bytes.restype = sz
        lib.psr_ring_attn_bwd.argtypes = [ctypes.POINTER(Shape), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz,
                                          ctypes.c_int, vp]
        lib.psr_ring_attn_bwd.restype = ctypes.c_int
        P_rs = ctypes.POINTER(RsShape)
        lib.psr_gemm_rs_workspace_bytes.argtypes = [P_rs]
        lib.psr_gemm_rs_workspace_bytes.restype = sz
        lib.psr_gemm_rs.argtypes = [P_rs, vp, vp, vp, vp, sz, P_part, vp]
        lib.psr_gemm_rs.restype = ctypes.c_int
        lib.psr_ring_attn_fwd_noalloc.argtypes = [P_shape, vp, vp, vp, vp, vp, P_part, vp]
        lib.psr_ring_attn_fwd_noalloc.restype = ctypes.c_int
        lib.psr_noalloc_get_stats.argtypes = [ctypes.POINTER(Stats), vp]
        lib.psr_noalloc_get_stats.restype = ctypes.c_int
        P_st, P_rot, P_lin, P_kv4 = map(ctypes.POINTER, (Strides, RotaryShape, LinearShape, Kv4Shape))
        dbl = ctypes.c_double
        lib.psr_rotary_table.argtypes = [ctypes.c_int, dbl, ctypes.c_int, dbl, dbl, dbl, dbl, vp]
        lib.psr_rotary.argtypes = [P_rot, vp, P_st, vp, P_st, vp, P_st, vp, P_st, vp, vp, ctypes.c_longlong, vp]
        lib.psr_linear_workspace_bytes.argtypes = [P_lin, ctypes.c_int]
        lib.psr_linear.argtypes = [P_lin, vp, vp, vp, vp, vp, vp, vp, sz, ctypes.c_int, vp]
        lib.psr_linear_bwd.argtypes = [P_lin, vp, vp, vp, vp, vp, vp, vp, vp, sz, ctypes.c_int, vp]
        lib.psr_kv4_cache_bytes.argtypes = [P_kv4]
        lib.psr_kv4_append.argtypes = [P_kv4, vp, P_st, vp, P_st, vp, vp, vp, vp, vp]
        lib.psr_kv4_read.argtypes = [P_kv4, vp, vp, vp, vp, vp, vp, vp]
        lib.psr_kv4_attn_workspace_bytes.argtypes = [P_kv4]
        lib.psr_kv4_attn.argtypes = [P_kv4, vp, P_st, vp, vp, vp, vp, P_st, vp, vp, sz, vp]
        for name in ("psr_rotary_table", "psr_rotary", "psr_linear", "psr_linear_bwd", "psr_kv4_append", "psr_kv4_read",
                     "psr_kv4_attn"):
            getattr(lib, name).restype = ctypes.c_int
        for name in ("psr_linear_workspace_bytes", "psr_kv4_cache_bytes", "psr_kv4_attn_workspace_bytes"):
            getattr(lib, name).restype = sz
        lib.psr_num_ctas.argtypes = []
        lib.psr_num_ctas.restype = ctypes.c_int
        _lib = lib
        return lib


def status_string(status: int) -> str:
    return load().psr_status_string(int(status)).decode()


def make_shape(B, Hq, Hkv, S, P, d, causal, scale=None) -> Shape:
    """causal: False/0, True/1 (CAUSAL), or 2 (CAUSAL_BALANCED: load-balanced shards)."""
    return Shape(int(B), int(Hq), int(Hkv), int(S), int(P), int(d), int(causal),
                 float(scale) if scale is not None else 0.0)


def make_partition(mode=ADAPTIVE, n_staging=0, n_min=0, n_max=0, fault=FAULT_NONE, timeout_ms=0) -> Partition:
    return Partition(int(mode), int(n_staging), int(n_min), int(n_max), int(fault), int(timeout_ms))


def workspace_bytes(shape: Shape) -> int:
    n = load().psr_workspace_bytes(ctypes.byref(shape))
    if n == 0:
        raise PsrError(ERR_UNSUPPORTED, "psr_workspace_bytes")
    return int(n)


def controller_target(n_cta, R_s, C_s, R_p, C_p, n_min=1, n_max=1 << 30) -> int:
    return int(load().psr_controller_target(int(n_cta), float(R_s), float(C_s), float(R_p), float(C_p), int(n_min),
                                            int(n_max)))


def num_ctas() -> int:
    n = load().psr_num_ctas()
    if n < 0:
        raise PsrError(-n, "psr_num_ctas")
    return n


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check_tensor(t, name, shape, dtype):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_host(t, name, shape, dtypes):
    import torch
    if not isinstance(t, torch.Tensor) or t.device.type != "cpu":
        raise ValueError(f"{name} must be a host (CPU) tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {dtypes}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _same_device(tensors, what):
    devs = {t.device for t in tensors}
    if len(devs) != 1:
        raise ValueError(f"{what}: all device tensors must be on one GPU, got {sorted(map(str, devs))}")


def ring_attn_fwd(q, k, v, *, P, causal, scale=None, partition=None, workspace=None, out=None, lse=None,
                  stream=None):
    """Ring Attention forward over P shards held on this GPU.

    q: [B, Hq, S, d] bf16; k, v: [B, Hkv, S, d] bf16 (CUDA, contiguous).
    Returns (o [B, Hq, S, d] bf16, lse [B, Hq, S] fp32, workspace).  The call is
    asynchronous on `stream`; use get_stats(workspace) to read the device
    status (timeouts) and the controller's statistics.
    """
    import torch
    lib = load()
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k, v must be 4-d [B, H, S, d]")
    B, Hq, S, d = q.shape
    Hkv = k.shape[1]
    _check_tensor(q, "q", (B, Hq, S, d), torch.bfloat16)
    _check_tensor(k, "k", (B, Hkv, S, d), torch.bfloat16)
    _check_tensor(v, "v", (B, Hkv, S, d), torch.bfloat16)
    shape = make_shape(B, Hq, Hkv, S, P, d, causal, scale)
    need = workspace_bytes(shape)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    elif not workspace.is_cuda or workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must be a CUDA tensor of at least {need} bytes")
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_tensor(out, "out", (B, Hq, S, d), torch.bfloat16)
    if lse is None:
        lse = torch.empty((B, Hq, S), dtype=torch.float32, device=q.device)
    else:
        _check_tensor(lse, "lse", (B, Hq, S), torch.float32)
    _same_device((q, k, v, out, lse, workspace), "ring_attn_fwd")
    part = partition if partition is not None else make_partition()
    rc = lib.psr_ring_attn_fwd(ctypes.byref(shape), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                               lse.data_ptr(), workspace.data_ptr(), need, ctypes.byref(part),
                               _stream_handle(stream))
    if rc != OK:
        raise PsrError(rc, "psr_ring_attn_fwd")
    return out, lse, workspace


def ring_attn_fwd_host(q_host, k_host, v_host, o_host, lse_host, dq, dk, dv, d_o, d_lse, *, P, causal, scale=None,
                       partition=None, workspace=None, stream=None):
    """Host-buffer variant: copies in, runs, copies out and synchronises (one C call; large shapes
    run in slices whose copies overlap the kernels).

    q_host, o_host: [B, Hq, S, d]; k_host, v_host: [B, Hkv, S, d] -- pinned host tensors holding
    bf16 values (dtype bfloat16, or int16 carrying the bf16 bit patterns); lse_host: [B, Hq, S]
    fp32, pinned.  dq, d_o: [B, Hq, S, d] and dk, dv: [B, Hkv, S, d] bf16, d_lse: [B, Hq, S] fp32 --
    the device buffers the copies land in (CUDA, contiguous, one GPU)."""
    import torch
    lib = load()
    if not isinstance(q_host, torch.Tensor) or q_host.dim() != 4 or not isinstance(k_host, torch.Tensor) \
            or k_host.dim() != 4:
        raise ValueError("q_host, k_host, v_host must be 4-d [B, H, S, d] tensors")
    B, Hq, S, d = q_host.shape
    Hkv = k_host.shape[1]
    bits = (torch.bfloat16, torch.int16)
    _check_host(q_host, "q_host", (B, Hq, S, d), bits)
    _check_host(k_host, "k_host", (B, Hkv, S, d), bits)
    _check_host(v_host, "v_host", (B, Hkv, S, d), bits)
    _check_host(o_host, "o_host", (B, Hq, S, d), bits)
    _check_host(lse_host, "lse_host", (B, Hq, S), (torch.float32,))
    _check_tensor(dq, "dq", (B, Hq, S, d), torch.bfloat16)
    _check_tensor(dk, "dk", (B, Hkv, S, d), torch.bfloat16)
    _check_tensor(dv, "dv", (B, Hkv, S, d), torch.bfloat16)
    _check_tensor(d_o, "d_o", (B, Hq, S, d), torch.bfloat16)
    _check_tensor(d_lse, "d_lse", (B, Hq, S), torch.float32)
    _same_device((dq, dk, dv, d_o, d_lse), "ring_attn_fwd_host")
    for t, name in ((q_host, "q_host"), (k_host, "k_host"), (v_host, "v_host"), (o_host, "o_host"),
                    (lse_host, "lse_host")):
        if not t.is_pinned():
            raise ValueError(f"{name} must be in pinned host memory (tensor.pin_memory()): the copies run "
                             f"asynchronously on the library's streams")
    shape = make_shape(B, Hq, Hkv, S, P, d, causal, scale)
    need = workspace_bytes(shape)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dq.device)
    elif not workspace.is_cuda or workspace.device != dq.device or workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must be a CUDA tensor on {dq.device} of at least {need} bytes")
    part = partition if partition is not None else make_partition()
    rc = lib.psr_ring_attn_fwd_host(ctypes.byref(shape), q_host.data_ptr(), k_host.data_ptr(), v_host.data_ptr(),
                                    o_host.data_ptr(), lse_host.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                    dv.data_ptr(), d_o.data_ptr(), d_lse.data_ptr(), workspace.data_ptr(), need,
                                    ctypes.byref(part), _stream_handle(stream))
    if rc != OK:
        raise PsrError(rc, "psr_ring_attn_fwd_host")
    return workspace


def ag_gemm_workspace_bytes(M, K, Ns, P) -> int:
    n = load().psr_ag_gemm_workspace_bytes(ctypes.byref(AgShape(int(M), int(K), int(Ns), int(P))))
    if n == 0:
        raise PsrError(ERR_UNSUPPORTED, "psr_ag_gemm_workspace_bytes")
    return int(n)


def ag_gemm(a, w, *, P, partition=None, workspace=None, out=None, stream=None):
    """AllGather + GEMM through the C ABI: a [M][K] bf16 (rank j's shard = rows j*M/P..),
    w [P][Ns][K] bf16 -> c [P][M][Ns] bf16, C_r = gather(A) @ W_r^T.  Returns (c, workspace)."""
    import torch
    lib = load()
    if a.dim() != 2 or w.dim() != 3:
        raise ValueError("ag_gemm: a must be [M, K] and w [P, Ns, K]")
    M, K = a.shape
    Ns = w.shape[1]
    shape = AgShape(int(M), int(K), int(Ns), int(P))
    need = ag_gemm_workspace_bytes(M, K, Ns, P)
    _check_tensor(a, "a", (M, K), torch.bfloat16)
    _check_tensor(w, "w", (P, Ns, K), torch.bfloat16)
    if out is None:
        out = torch.empty((P, M, Ns), dtype=torch.bfloat16, device=a.device)
    _check_tensor(out, "out", (P, M, Ns), torch.bfloat16)
    _same_device((a, w, out), "ag_gemm")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=a.device)
    elif not workspace.is_cuda or workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"ag_gemm: workspace must be a CUDA tensor of at least {need} bytes")
    part = partition if partition is not None else make_partition()
    rc = lib.psr_ag_gemm(ctypes.byref(shape), a.data_ptr(), w.data_ptr(), out.data_ptr(), workspace.data_ptr(),
                         workspace.numel() * workspace.element_size(), ctypes.byref(part), _stream_handle(stream))
    if rc != OK:
        raise PsrError(rc, "psr_ag_gemm")
    return out, workspace


def ring_attn_bwd_workspace_bytes(shape: Shape) -> int:
    n = load().psr_ring_attn_bwd_workspace_bytes(ctypes.byref(shape))
    if n == 0:
        raise PsrError(ERR_UNSUPPORTED, "psr_ring_attn_bwd_workspace_bytes")
    return int(n)


def ring_attn_bwd(q, k, v, o, lse, dout, *, P, causal, scale=None, workspace=None, dq=None, dk=None, dv=None,
                  timeout_ms=0, stream=None):
    """Ring Attention backward through the C ABI: q, o, dout [B][Hq][S][d], k, v [B][Hkv][S][d]
    (bf16), lse [B][Hq][S] fp32 (the forward's) -> (dq, dk, dv, workspace)."""
    import torch
    lib = load()
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("ring_attn_bwd: q, k, v must be 4-d [B, H, S, d]")
    B, Hq, S, d = q.shape
    Hkv = k.shape[1]
    shape = make_shape(B, Hq, Hkv, S, P, d, causal, scale)
    need = ring_attn_bwd_workspace_bytes(shape)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    for t, name in ((q, "q"), (o, "o"), (dout, "dout"), (dq, "dq")):
        _check_tensor(t, name, (B, Hq, S, d), torch.bfloat16)
    for t, name in ((k, "k"), (v, "v"), (dk, "dk"), (dv, "dv")):
        _check_tensor(t, name, (B, Hkv, S, d), torch.bfloat16)
    _check_tensor(lse, "lse", (B, Hq, S), torch.float32)
    _same_device((q, k, v, o, lse, dout, dq, dk, dv), "ring_attn_bwd")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    elif not workspace.is_cuda or workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"ring_attn_bwd: workspace must be a CUDA tensor of at least {need} bytes")
    rc = lib.psr_ring_attn_bwd(ctypes.byref(shape), q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                               lse.data_ptr(), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                               workspace.data_ptr(), workspace.numel() * workspace.element_size(), int(timeout_ms),
                               _stream_handle(stream))
    if rc != OK:
        raise PsrError(rc, "psr_ring_attn_bwd")
    return dq, dk, dv, workspace


def gemm_rs_workspace_bytes(M, N, Ks, P) -> int:
    n = load().psr_gemm_rs_workspace_bytes(ctypes.byref(RsShape(int(M), int(N), int(Ks), int(P))))
    if n == 0:
        raise PsrError(ERR_UNSUPPORTED, "psr_gemm_rs_workspace_bytes")
    return int(n)


def gemm_rs(a, w, *, partition=None, workspace=None, out=None, stream=None):
    """GEMM + ReduceScatter through the C ABI: a [P][M][Ks] bf16 (rank r's activations),
    w [P][N][Ks] bf16 (rank r's weights) -> out [M][N] bf16 = sum_r a[r] @ w[r]^T, rows
    q*M/P .. belonging to rank q.  Returns (out, workspace)."""
    import torch
    lib = load()
    if a.dim() != 3 or w.dim() != 3:
        raise ValueError("gemm_rs: a must be [P, M, Ks] and w [P, N, Ks]")
    P, M, Ks = a.shape
    N = w.shape[1]
    shape = RsShape(int(M), int(N), int(Ks), int(P))
    need = gemm_rs_workspace_bytes(M, N, Ks, P)
    _check_tensor(a, "a", (P, M, Ks), torch.bfloat16)
    _check_tensor(w, "w", (P, N, Ks), torch.bfloat16)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    _check_tensor(out, "out", (M, N), torch.bfloat16)
    _same_device((a, w, out), "gemm_rs")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=a.device)
    elif not workspace.is_cuda or workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"gemm_rs: workspace must be a CUDA tensor of at least {need} bytes")
    part = partition if partition is not None else make_partition()
    rc = lib.psr_gemm_rs(ctypes.byref(shape), a.data_ptr(), w.data_ptr(), out.data_ptr(), workspace.data_ptr(),
                         workspace.numel() * workspace.element_size(), ctypes.byref(part), _stream_handle(stream))
    if rc != OK:
        raise PsrError(rc, "psr_gemm_rs")
    return out, workspace


# ------------------------------------------------------------------------------------------------
# The attention layer around the ring: rotary positions, linear, 4-bit KV cache
# ------------------------------------------------------------------------------------------------
# These calls run on their tensors' device whatever the current one is.  Memory that a call makes
# (outputs and workspaces not passed in) belongs to the stream the call runs on.

class _Launch:
    """The device and stream of a call: makes the device current, and the stream while memory is made."""
    __slots__ = ("torch", "device", "stream", "handle", "other", "back")

    def __init__(self, device, stream, what):
        import torch
        self.torch, self.device, self.stream = torch, device, stream
        if stream is not None and stream.device != device:
            raise ValueError(f"{what}: the stream is on {stream.device}, the tensors on {device}")

    def __enter__(self):
        # the raw getters: torch.cuda.current_stream() alone takes longer than a small call's kernel
        raw, index = self.torch._C, self.device.index
        self.back = raw._cuda_getDevice()
        if self.back != index:
            self.torch.cuda.set_device(index)
        current = raw._cuda_getCurrentRawStream(index)
        self.handle = current if self.stream is None else self.stream.cuda_stream
        self.other = self.handle != current
        return self

    def __exit__(self, *exc):
        if self.back != self.device.index:
            self.torch.cuda.set_device(self.back)

    def empty(self, shape, dtype):
        if not self.other:
            return self.torch.empty(shape, dtype=dtype, device=self.device)
        with self.torch.cuda.stream(self.stream):
            return self.torch.empty(shape, dtype=dtype, device=self.device)


# What the checks of a call found, by the shapes, strides, types and devices of its tensors and its other arguments: the checks
# take longer than a small call's kernel, and the same call comes again for every layer and token.  Addresses are no part of
# it (but for their alignment); what depends on them is checked every time.
_plans = {}


def _meta(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.device)


def _plan(key, check):
    """The plan under a key, or what `check` returns for a new one.  key: a function (arguments that are no tensors, or
    cannot be looked up, are for the checks to refuse) that takes numbers by their values: they may come as tensors, too."""
    try:
        key = key()
        plan = _plans.get(key)
    except (AttributeError, TypeError):
        return check()
    if plan is None:
        plan = check()
        if len(_plans) >= 1024:
            _plans.clear()
        _plans[key] = plan
    return plan


_TYPES = {}  # torch.dtype -> type code


def _type_code(dtype, name, allowed):
    if not _TYPES:
        import torch
        _TYPES.update({torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32})
    code = _TYPES.get(dtype, F32 + 1)
    if code > allowed:
        raise ValueError(f"{name} must be bfloat16{', float16 or float32' if allowed == F32 else ' or float16'}, "
                         f"got {dtype}")
    return code


def _type_of(t, name, allowed):
    """The type code of a tensor."""
    return _type_code(t.dtype, name, allowed)


def _check_like(t, name, shape, dtype, device):
    """A CUDA tensor of this shape and type on this device, of any strides."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _check_flat(t, name, shape, dtype, device):
    _check_like(t, name, shape, dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_cuda(t, name, dims):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must be {dims}-d, got {tuple(t.shape)}")


def _heads_strides(t, name, written=False):
    """Strides of a [B, H, S, d] tensor whose last axis is contiguous; no element of a written one twice."""
    b, h, s, e = t.stride()
    B, H, S, d = t.shape
    if e != 1 and d > 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    if written and t.numel() > 0:
        reach = d  # elements spanned so far; every further axis must step over them
        for step, n in sorted(zip((b, h, s), (B, H, S))):
            if n > 1:
                if step < reach:
                    raise ValueError(f"{name}: elements overlap (strides {t.stride()})")
                reach = step * (n - 1) + reach
    return Strides(b, h, s)


def _span(t):
    """First byte and the byte past the last of a tensor's elements."""
    last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()


def _check_apart(out, x, what, same_ok, kinds="an output overlaps an input"):
    """`out` shares no memory with `x`, or is `x` itself where that is allowed.  Column ranges of the same rows are
    apart."""
    if out.numel() == 0 or x.numel() == 0:
        return
    if same_ok and out.data_ptr() == x.data_ptr() and out.stride() == x.stride():
        return
    (a, b), (c, d) = _span(out), _span(x)
    if a < d and c < b:
        ld, size = out.stride(0), out.element_size()
        if out.dim() == x.dim() == 2 and x.stride(0) == ld > 0 and size == x.element_size() and (a - c) % size == 0:
            right = (a - c) // size % ld  # out's first column, counted from x's
            if right >= x.shape[1] and ld - right >= out.shape[1]:
                return
        raise ValueError(f"{what}: {kinds}")


def _check_outputs(what, outs, inputs, workspace=None):
    """Outputs passed in, and the workspace, share no memory with the inputs or one another."""
    outs = [t for t in outs if t is not None]
    for i, out in enumerate(outs):
        for x in inputs:
            if x is not None:
                _check_apart(out, x, what, False)
        for other in outs[:i]:
            _check_apart(out, other, what, False, "the outputs overlap")
    if workspace is not None:
        first = workspace.data_ptr()  # contiguous, or refused later
        past = first + workspace.numel() * workspace.element_size()
        for x in (*inputs, *outs):
            if x is not None and x.numel() > 0:
                a, b = _span(x)
                if a < past and first < b:
                    raise ValueError(f"{what}: the workspace overlaps a tensor")


def _check_other(out, x, what, kinds):
    """Of [B, H, S, d] tensors: `out` is not `x`, and shares nothing with it if both are contiguous (views of one buffer
    may lie between one another)."""
    if out.data_ptr() == x.data_ptr() or (out.is_contiguous() and x.is_contiguous()):
        _check_apart(out, x, what, False, kinds)


def rotary_table(rot, base=10000.0, *, scaling="plain", factor=1.0, original_length=0, beta_fast=32.0, beta_slow=1.0,
                 device="cuda"):
    """Frequencies of `rot` rotated columns for rotary(): [rot/2] int64 holding turns per position in 64-bit
    fixed point.  scaling: "plain", "linear" (all divided by `factor`) or "by_parts" (those that turn less than beta_slow
    times over `original_length` divided, those that turn more than beta_fast times kept, blended between)."""
    import torch
    if scaling not in ROTARY_SCALINGS:
        raise ValueError(f"rotary_table: scaling must be one of {sorted(ROTARY_SCALINGS)}, got {scaling!r}")
    host = torch.empty(max(0, int(rot)) // 2, dtype=torch.int64)
    rc = load().psr_rotary_table(int(rot), float(base), ROTARY_SCALINGS[scaling], float(factor), float(original_length),
                                 float(beta_fast), float(beta_slow), host.data_ptr() if rot > 0 else None)
    if rc != OK:
        raise PsrError(rc, "psr_rotary_table")
    return host.to(device)


def rotary(q, k, table, *, P=1, causal=CAUSAL, positions=None, offset=0, interleaved=False, amplitude=1.0, q_out=None,
           k_out=None, stream=None, inverse=False):
    """Rotary positions of q [B, Hq, S, d] and k [B, Hkv, S, d] (or None), bf16, fp16 or fp32, any strides with a
    contiguous last axis (views of a projection's output, say).  The first 2 * len(table) columns are turned, pairs
    (i, i + rot/2) or, interleaved, (2i, 2i + 1); the others are copied.

    positions: int64 [S] or [B, S]; None takes offset + the global position of each row in the ring's shard order
    (P, causal as for ring_attn_fwd).  Returns (q_out, k_out), contiguous unless passed in; an output may be its own
    input, and shares no element with the other input or output."""
    shape, qs, qos, ks, kos, pos_b, dev, q_shape, k_shape = _plan(
        lambda: (rotary, _meta(q), _meta(k), _meta(table), _meta(positions), int(P), int(causal), bool(interleaved),
                 float(amplitude), bool(inverse), _meta(q_out), _meta(k_out)),
        lambda: _rotary_plan(q, k, table, P, causal, positions, interleaved, amplitude, q_out, k_out, inverse))
    if offset:
        shape = RotaryShape.from_buffer_copy(shape)
        shape.offset = int(offset)
    if q_out is not None or k_out is not None:
        for x, out in ((q, q_out), (k, k_out)):
            if out is not None:
                _check_apart(out, x, "rotary", True)
        if k is not None:
            for out, x in ((q_out, k), (k_out, q)):
                if out is not None:
                    _check_other(out, x, "rotary", "an output overlaps the other input")
            if q_out is not None and k_out is not None:
                _check_other(q_out, k_out, "rotary", "the outputs overlap")
        for out in (q_out, k_out):
            if out is not None:
                _check_outputs("rotary", (out,), (table, positions))
    with _Launch(dev, stream, "rotary") as at:
        if q_out is None:
            q_out = at.empty(q_shape, q.dtype)
        if k is None:
            k_in = k_to = None
        else:
            if k_out is None:
                k_out = at.empty(k_shape, q.dtype)
            k_in, k_to = k.data_ptr(), k_out.data_ptr()
        if shape.B == 0 or shape.S == 0:  # no rows, no pointers
            return q_out, k_out
        rc = load().psr_rotary(shape, q.data_ptr(), qs, q_out.data_ptr(), qos, k_in, ks, k_to, kos, table.data_ptr(),
                               None if positions is None else positions.data_ptr(), pos_b, at.handle)
    if rc != OK:
        raise PsrError(rc, "psr_rotary")
    return q_out, k_out


def _rotary_plan(q, k, table, P, causal, positions, interleaved, amplitude, q_out, k_out, inverse):
    import torch
    _check_cuda(q, "q", 4)
    B, Hq, S, d = q.shape
    dev, dtype = q.device, q.dtype
    code = _type_of(q, "q", F32)
    Hkv = 0
    if k is not None:
        _check_cuda(k, "k", 4)
        Hkv = k.shape[1]
        _check_like(k, "k", (B, Hkv, S, d), dtype, dev)
    _check_flat(table, "table", (table.numel(),), torch.int64, dev)
    pos_b = 0
    if positions is not None:
        _check_like(positions, "positions", (B, S) if positions.dim() == 2 else (S,), torch.int64, dev)
        if S > 1 and positions.stride(-1) != 1:
            raise ValueError("positions: the last axis must be contiguous")
        pos_b = positions.stride(0) if positions.dim() == 2 else 0
    if k is None and k_out is not None:
        raise ValueError("k_out without k")
    for x, out, name in ((q, q_out, "q_out"), (k, k_out, "k_out")):
        if out is not None:
            _check_like(out, name, x.shape, dtype, dev)
    flat = lambda H: Strides(H * S * d, S * d, d)
    qs, qos = _heads_strides(q, "q"), flat(Hq) if q_out is None else _heads_strides(q_out, "q_out", True)
    ks = kos = None
    if k is not None:
        ks, kos = _heads_strides(k, "k"), flat(Hkv) if k_out is None else _heads_strides(k_out, "k_out", True)
    if (B == 0 or S == 0) and (int(P) < 1 or S % int(P)):
        raise PsrError(ERR_ARG if int(P) < 1 else ERR_UNSUPPORTED, "psr_rotary")
    shape = RotaryShape(B, Hq, Hkv, S, int(P), d, int(causal), 2 * table.numel(), int(bool(interleaved)), int(bool(inverse)),
                        code, float(amplitude), 0)
    return shape, qs, qos, ks, kos, pos_b, dev, (B, Hq, S, d), (B, Hkv, S, d)


def rotary_bwd(dq, dk, table, **kwargs):
    """The gradient of rotary(): dq, dk are those of its outputs, the arguments are the forward's.  Returns the
    gradients of its inputs (rows turned back; the same scaling by `amplitude`)."""
    return rotary(dq, dk, table, inverse=True, **kwargs)


def _linear_shape(x, w, activation, what):
    _check_cuda(x, "x", 2)
    _check_cuda(w, "w", 2)
    if activation not in ACTIVATIONS:
        raise ValueError(f"{what}: activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")
    code = _type_of(x, "x", F16)
    M, K = x.shape
    N = w.shape[0]
    _check_like(w, "w", (N, K), x.dtype, x.device)
    sh = LinearShape(M, N, K, ACTIVATIONS[activation], code, _row_stride(x, "x"), _row_stride(w, "w"), 0, 0, 0,
                     (1 if x.data_ptr() % 16 else 0) | (2 if w.data_ptr() % 16 else 0))
    return sh, M, N, K


def _row_stride(t, name):
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: rows must be contiguous")
    if rows <= 1:
        return 0
    if t.stride(0) < cols:
        raise ValueError(f"{name}: rows must not overlap (stride {t.stride(0)}, {cols} columns)")
    return t.stride(0)


def _workspace(at, workspace, need, what):
    if workspace is None:
        import torch
        return at.empty((need,), torch.uint8)
    if not workspace.is_cuda or workspace.device != at.device or not workspace.is_contiguous() \
            or workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"{what}: workspace must be a contiguous CUDA tensor on {at.device} of at least {need} bytes")
    return workspace


def _clear_status(at, workspace):
    """Of a call with nothing to do, which never reaches the library: its workspace reports success."""
    with at.torch.cuda.stream(at.stream):  # None: the current one
        workspace.flatten().view(at.torch.uint8)[:256].zero_()


def linear_workspace_bytes(M, N, K, *, activation="none", backward=False) -> int:
    """Bytes of workspace that linear() or linear_bwd() needs for contiguous tensors, or views whose row strides are
    multiples of 8 elements and that start on 16-byte boundaries."""
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")
    n = load().psr_linear_workspace_bytes(LinearShape(int(M), int(N), int(K), ACTIVATIONS[activation], BF16),
                                          int(bool(backward)))
    if n == 0:
        raise PsrError(ERR_ARG, "psr_linear_workspace_bytes")
    return int(n)


def linear(x, w, bias=None, residual=None, *, activation="none", save_z=False, out=None, z=None, workspace=None,
           timeout_ms=0, stream=None):
    """y = act(x w^T + bias) + residual: x [M, K], w [N, K], bias [N], residual [M, N], bf16 or fp16, fp32 sums;
    rows may be strided.  activation: "none", "relu", "gelu", "gelu_tanh" or "silu".

    Returns (y [M, N], z, workspace).  With save_z (or a tensor z) z = x w^T + bias is written too, for
    linear_bwd(); otherwise it is None.  `out` may be the residual."""
    sh, need, dev, shape = _plan(
        lambda: (linear, _meta(x), _meta(w), _meta(bias), _meta(residual), activation, _meta(out), _meta(z), x.data_ptr() % 16,
                 w.data_ptr() % 16),
        lambda: _linear_plan(x, w, bias, residual, activation, out, z))
    if out is not None:
        for t in (x, w, bias):
            if t is not None:
                _check_apart(out, t, "linear", False)
        if residual is not None:
            _check_apart(out, residual, "linear", True)
    if z is not None:
        for t in (x, w, bias, residual, out):
            if t is not None:
                _check_apart(z, t, "linear", False)
    if workspace is not None:
        _check_outputs("linear", (), (x, w, bias, residual, out, z), workspace)
    with _Launch(dev, stream, "linear") as at:
        if out is None:
            out = at.empty(shape, x.dtype)
        if z is None and save_z:
            z = at.empty(shape, x.dtype)
        workspace = _workspace(at, workspace, need, "linear")
        if shape[0] == 0:
            _clear_status(at, workspace)
            return out, z, workspace
        rc = load().psr_linear(sh, x.data_ptr(), w.data_ptr(), None if bias is None else bias.data_ptr(),
                               None if residual is None else residual.data_ptr(), out.data_ptr(),
                               None if z is None else z.data_ptr(), workspace.data_ptr(), need, int(timeout_ms), at.handle)
    if rc != OK:
        raise PsrError(rc, "psr_linear")
    return out, z, workspace


def _linear_plan(x, w, bias, residual, activation, out, z):
    sh, M, N, K = _linear_shape(x, w, activation, "linear")
    dev, dtype = x.device, x.dtype
    if bias is not None:
        _check_flat(bias, "bias", (N,), dtype, dev)
    if residual is not None:
        _check_like(residual, "residual", (M, N), dtype, dev)
        sh.ldr = _row_stride(residual, "residual")
    if out is not None:
        _check_like(out, "out", (M, N), dtype, dev)
        sh.ldy = _row_stride(out, "out")
    if z is not None:
        _check_like(z, "z", (M, N), dtype, dev)
        sh.ldz = _row_stride(z, "z")
    need = load().psr_linear_workspace_bytes(sh, 0)
    if need == 0:
        raise PsrError(ERR_ARG, "psr_linear")
    return sh, need, dev, (M, N)


def linear_bwd(dy, x, w, z=None, *, activation="none", need_dx=True, need_dw=True, need_db=True, dx=None, dw=None,
               db=None, workspace=None, timeout_ms=0, stream=None):
    """Gradients of linear(): dy [M, N] is that of y, z the forward's (needed unless activation is "none"); the
    residual's gradient is dy itself.  Returns (dx [M, K], dw [N, K], db [N], workspace), None for those not asked for;
    dx, dw, db may be passed in (contiguous)."""
    sh, need, dev, shapes = _plan(
        lambda: (linear_bwd, _meta(dy), _meta(x), _meta(w), _meta(z), activation, _meta(dx), _meta(dw), _meta(db),
                 x.data_ptr() % 16, w.data_ptr() % 16, dy.data_ptr() % 16),
        lambda: _linear_bwd_plan(dy, x, w, z, activation, dx, dw, db))
    _check_outputs("linear_bwd", (dx, dw, db), (dy, x, w, z), workspace)
    with _Launch(dev, stream, "linear_bwd") as at:
        if dx is None and need_dx:
            dx = at.empty(shapes[0], x.dtype)
        if dw is None and need_dw:
            dw = at.empty(shapes[1], x.dtype)
        if db is None and need_db:
            db = at.empty(shapes[2], x.dtype)
        workspace = _workspace(at, workspace, need, "linear_bwd")
        if shapes[0][0] == 0:  # sums over no rows
            _clear_status(at, workspace)
            with at.torch.cuda.stream(stream):  # None: the current one
                for t in (dw, db):
                    if t is not None:
                        t.zero_()
            return dx, dw, db, workspace
        rc = load().psr_linear_bwd(sh, dy.data_ptr(), z.data_ptr() if activation != "none" else None, x.data_ptr(),
                                   w.data_ptr(), *(None if t is None else t.data_ptr() for t in (dx, dw, db)),
                                   workspace.data_ptr(), need, int(timeout_ms), at.handle)
    if rc != OK:
        raise PsrError(rc, "psr_linear_bwd")
    return dx, dw, db, workspace


def _linear_bwd_plan(dy, x, w, z, activation, dx, dw, db):
    sh, M, N, K = _linear_shape(x, w, activation, "linear_bwd")
    dev, dtype = x.device, x.dtype
    _check_like(dy, "dy", (M, N), dtype, dev)
    sh.ldy = _row_stride(dy, "dy")
    if dy.data_ptr() % 16:
        sh.odd |= 4
    if activation != "none":
        if z is None:
            raise ValueError(f"linear_bwd: activation {activation!r} needs the forward's z")
        _check_like(z, "z", (M, N), dtype, dev)
        sh.ldz = _row_stride(z, "z")
    shapes = (M, K), (N, K), (N,)
    for t, name, shape in zip((dx, dw, db), ("dx", "dw", "db"), shapes):
        if t is not None:
            _check_flat(t, name, shape, dtype, dev)
    need = load().psr_linear_workspace_bytes(sh, 1)
    if need == 0:
        raise PsrError(ERR_ARG, "psr_linear_bwd")
    return sh, need, dev, shapes


def kv4_cache(n_pages, Hkv, d, page, device="cuda"):
    """An empty 4-bit KV cache, uint8 [n_pages, Hkv, page * (d + 8)] (a page is one contiguous piece); d 64 or 128,
    page 16, 32, 64, 128 or 256 tokens."""
    import torch
    need = load().psr_kv4_cache_bytes(Kv4Shape(0, int(Hkv), int(Hkv), 0, int(d), int(page), int(n_pages), 1, BF16, 0.0))
    if need == 0:
        raise PsrError(ERR_UNSUPPORTED, "psr_kv4_cache_bytes")
    return torch.zeros((int(n_pages), int(Hkv), int(page) * (int(d) + 8)), dtype=torch.uint8, device=device)


def _kv4_shape(cache, table, B, Hq, Hkv, S, d, page, code, scale, dev):
    import torch
    _check_cuda(cache, "cache", 3)
    _check_flat(cache, "cache", (cache.shape[0], int(Hkv), int(page) * (d + 8)), torch.uint8, dev)
    _check_cuda(table, "table", 2)
    _check_flat(table, "table", (B, table.shape[1]), torch.int32, dev)
    return Kv4Shape(B, Hq, int(Hkv), S, d, int(page), cache.shape[0], table.shape[1], code,
                    0.0 if scale is None else float(scale))


def _check_counts(B, dev, **named):
    import torch
    for name, t in named.items():
        if t is not None:
            _check_flat(t, name, (B,), torch.int32, dev)


def kv4_append(k, v, cache, table, start, *, page, count=None, stream=None):
    """Quantises k, v [B, Hkv, S, d] (bf16 or fp16, any strides with a contiguous last axis) into the cache: row i of
    sequence b, i < count[b] (default: all S), goes to position start[b] + i, which is on page table[b, position // page].

    table: int32 [B, max_pages]; start, count: int32 [B].  Rows whose position is outside the table or whose page is
    outside the cache are left out.  The places written must differ, and the cache shares no memory with the other tensors.
    Returns the cache."""
    sh, ks, vs, dev = _plan(lambda: (kv4_append, _meta(k), _meta(v), _meta(cache), _meta(table), _meta(start), _meta(count), int(page)),
                            lambda: _kv4_append_plan(k, v, cache, table, start, count, page))
    if sh.B == 0 or sh.S == 0:
        return cache
    with _Launch(dev, stream, "kv4_append") as at:
        rc = load().psr_kv4_append(sh, k.data_ptr(), ks, v.data_ptr(), vs, cache.data_ptr(), table.data_ptr(),
                                   start.data_ptr(), None if count is None else count.data_ptr(), at.handle)
    if rc != OK:
        raise PsrError(rc, "psr_kv4_append")
    return cache


def _kv4_append_plan(k, v, cache, table, start, count, page):
    _check_cuda(k, "k", 4)
    B, Hkv, S, d = k.shape
    dev = k.device
    code = _type_of(k, "k", F16)
    _check_like(v, "v", k.shape, k.dtype, dev)
    sh = _kv4_shape(cache, table, B, Hkv, Hkv, S, d, page, code, None, dev)
    _check_counts(B, dev, start=start, count=count)
    return sh, _heads_strides(k, "k"), _heads_strides(v, "v"), dev


def kv4_read(cache, table, start, *, S, Hkv, d, page, count=None, dtype=None, k=None, v=None, stream=None):
    """Positions start[b] .. start[b] + S - 1 of each sequence, read back as k, v [B, Hkv, S, d] (bf16 unless `dtype`
    says float16): zeros from row count[b] on, NaN where the table or the cache has no such place."""
    sh, shape, dtype, dev = _plan(
        lambda: (kv4_read, _meta(cache), _meta(table), _meta(start), _meta(count), int(S), int(Hkv), int(d), int(page), dtype,
                 _meta(k), _meta(v)),
        lambda: _kv4_read_plan(cache, table, start, count, S, Hkv, d, page, dtype, k, v))
    _check_outputs("kv4_read", (k, v), (cache, table, start, count))
    with _Launch(dev, stream, "kv4_read") as at:
        k = at.empty(shape, dtype) if k is None else k
        v = at.empty(shape, dtype) if v is None else v
        if k.numel() == 0:
            return k, v
        rc = load().psr_kv4_read(sh, cache.data_ptr(), table.data_ptr(), start.data_ptr(),
                                 None if count is None else count.data_ptr(), k.data_ptr(), v.data_ptr(), at.handle)
    if rc != OK:
        raise PsrError(rc, "psr_kv4_read")
    return k, v


def _kv4_read_plan(cache, table, start, count, S, Hkv, d, page, dtype, k, v):
    import torch
    _check_cuda(table, "table", 2)
    B, dev = table.shape[0], table.device
    dtype = dtype if dtype is not None else (k.dtype if k is not None else torch.bfloat16)
    shape = (B, int(Hkv), int(S), int(d))
    sh = _kv4_shape(cache, table, B, int(Hkv), Hkv, int(S), int(d), page, _type_code(dtype, "dtype", F16), None, dev)
    _check_counts(B, dev, start=start, count=count)
    for t, name in ((k, "k"), (v, "v")):
        if t is not None:
            _check_flat(t, name, shape, dtype, dev)
    return sh, shape, dtype, dev


def kv4_attn_workspace_bytes(B, Hq, Hkv, S, d, *, page, n_pages, max_pages) -> int:
    """Bytes of workspace that kv4_attn() needs on the current device."""
    n = load().psr_kv4_attn_workspace_bytes(Kv4Shape(int(B), int(Hq), int(Hkv), int(S), int(d), int(page), int(n_pages),
                                                     int(max_pages), BF16, 0.0))
    if n == 0:
        raise PsrError(ERR_UNSUPPORTED, "psr_kv4_attn_workspace_bytes")
    return int(n)


def kv4_attn(q, cache, table, lens, *, Hkv, page, scale=None, out=None, lse=None, workspace=None, stream=None):
    """Attention of the last S positions of each cached sequence over the sequence (S = 1: single tokens).

    q: [B, Hq, S, d] bf16 or fp16, any strides with a contiguous last axis; cache, table as in kv4_append; lens: int32
    [B], the positions cached, the S new ones included.  Query i of sequence b sees positions 0 .. lens[b] - S + i.
    scale: of the scores, finite; None, 0 or less: 1/sqrt(d).
    Returns (o [B, Hq, S, d], lse [B, Hq, S] fp32, workspace): o = 0 and lse = -inf for a query that sees nothing, NaN
    for a sequence whose length or pages are out of range."""
    sh, qs, os_, need, dev = _plan(
        lambda: (kv4_attn, _meta(q), _meta(cache), _meta(table), _meta(lens), int(Hkv), int(page),
                 None if scale is None else float(scale), _meta(out), _meta(lse)),
        lambda: _kv4_attn_plan(q, cache, table, lens, Hkv, page, scale, out, lse))
    _check_outputs("kv4_attn", (out, lse), (q, cache, table, lens), workspace)
    with _Launch(dev, stream, "kv4_attn") as at:
        if out is None:
            out = at.empty(q.shape, q.dtype)
        if lse is None:
            lse = at.empty(q.shape[:3], at.torch.float32)
        workspace = _workspace(at, workspace, need, "kv4_attn")
        if sh.B == 0 or sh.S == 0:
            _clear_status(at, workspace)
            return out, lse, workspace
        rc = load().psr_kv4_attn(sh, q.data_ptr(), qs, cache.data_ptr(), table.data_ptr(), lens.data_ptr(), out.data_ptr(), os_,
                                 lse.data_ptr(), workspace.data_ptr(), need, at.handle)
    if rc != OK:
        raise PsrError(rc, "psr_kv4_attn")
    return out, lse, workspace


def _kv4_attn_plan(q, cache, table, lens, Hkv, page, scale, out, lse):
    import torch
    _check_cuda(q, "q", 4)
    B, Hq, S, d = q.shape
    dev = q.device
    sh = _kv4_shape(cache, table, B, Hq, Hkv, S, d, page, _type_of(q, "q", F16), scale, dev)
    _check_counts(B, dev, lens=lens)
    qs, os_ = _heads_strides(q, "q"), Strides(Hq * S * d, S * d, d)
    if out is not None:
        _check_like(out, "out", (B, Hq, S, d), q.dtype, dev)
        os_ = _heads_strides(out, "out", True)
    if lse is not None:
        _check_flat(lse, "lse", (B, Hq, S), torch.float32, dev)
    need = load().psr_kv4_attn_workspace_bytes(sh)
    if need == 0:
        raise PsrError(ERR_UNSUPPORTED, "psr_kv4_attn")
    return sh, qs, os_, need, dev


def get_stats(workspace, stream=None) -> dict:
    st = Stats()
    rc = load().psr_get_stats(ctypes.c_void_p(workspace.data_ptr()), ctypes.byref(st), _stream_handle(stream))
    if rc not in (OK, ERR_TIMEOUT):
        raise PsrError(rc, "psr_get_stats")
    return st.as_dict()


def get_trajectory(workspace, max_entries=4096, stream=None):
    buf = (ctypes.c_uint32 * (2 * max_entries))()
    n = load().psr_get_trajectory(ctypes.c_void_p(workspace.data_ptr()), buf, max_entries, _stream_handle(stream))
    if n < 0:
        raise PsrError(-n, "psr_get_trajectory")
    return [(int(buf[2 * i]), int(buf[2 * i + 1])) for i in range(n)]
