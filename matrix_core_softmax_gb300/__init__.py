"""Python binding of libfsa.so, the GB300 Fused-Softmax MX attention library.

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in ``include/fsa.h``.  PyTorch supplies
device memory and streams.  There is no fallback: if the library cannot be
loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libfsa.so")

FSA_MXFP8, FSA_MXFP6, FSA_MXFP4, FSA_MXFP4_EFQ = 0, 1, 2, 3
FORMATS = {"mxfp8": FSA_MXFP8, "mxfp6": FSA_MXFP6, "mxfp4": FSA_MXFP4, "mxfp4_efq": FSA_MXFP4_EFQ}
ELEM_E4M3, ELEM_E2M3, ELEM_E2M1 = 0, 1, 2
DEBUG_SKIP_KV_ARRIVE, DEBUG_LOSE_ONE_WAIT = 0x1, 0x2

STATUS = {0: "FSA_OK", 1: "FSA_ERR_INVALID_ARGUMENT", 2: "FSA_ERR_UNSUPPORTED",
          3: "FSA_ERR_CUDA", 4: "FSA_ERR_OUT_OF_MEMORY", 5: "FSA_ERR_TIMEOUT"}

# every symbol include/fsa.h declares
EXPORTS = ("fsa_quantize_mx", "fsa_attention_fwd", "fsa_attention_fwd_ex",
           "fsa_attention_prepare", "fsa_attention_run", "fsa_attention_workspace_size", "fsa_bf16_attention_fwd", "fsa_get_device_error",
           "fsa_status_string", "fsa_release_workspace", "fsa_attention_fwd_noalloc",
           "fsa_cross_attention_fwd", "fsa_cross_attention_workspace_size",
           "fsa_cross_attention_prepare", "fsa_cross_attention_run",
           "fsa_attention_fwd_host", "fsa_cross_attention_fwd_host", "fsa_mma_rate_probe",
           "fsa_kv4_page_bytes", "fsa_kv4_append", "fsa_kv4_read", "fsa_kv4_attention_fwd",
           "fsa_kv4_attention_workspace_size", "fsa_varlen_attention_fwd", "fsa_kv4_attention_fwd_ex",
           "fsa_varlen_attention_fwd_ex", "fsa_mx_pack", "fsa_mx_unpack", "fsa_rms_norm_mx", "fsa_mx_linear",
           "fsa_rms_norm_mx_ex")


class FsaError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)}")
        self.status = status


class Options(ctypes.Structure):
    _fields_ = [
        ("sm_scale", ctypes.c_float),
        ("rollback_bits", ctypes.c_void_p),
        ("rollback_count", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_uint64),
        ("wait_timeout_ms", ctypes.c_int),
        ("debug_flags", ctypes.c_int),
        ("efq_tau", ctypes.c_float),
        ("efq_h", ctypes.c_float),
        ("host_inputs_ready", ctypes.c_int),
        ("gate_mode", ctypes.c_int),
    ]

GATE_MODES = {"fp32": 0, "shortcut": 1}


_lock = threading.Lock()
_lib = None


def load(path: str | None = None):
    """Load libfsa.so (built by ``matrix_core_softmax_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            p = path or LIB_PATH
            if not os.path.exists(p):
                raise OSError(f"libfsa.so not built ({p}); run matrix_core_softmax_gb300/build.py")
            lib = ctypes.CDLL(p)
            V, I, I64, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
            lib.fsa_quantize_mx.argtypes = [V, I64, I64, I64, I, I, V, V, V]
            lib.fsa_quantize_mx.restype = I
            lib.fsa_attention_fwd.argtypes = [V, V, V, V, I, I, I, I, I, F, V]
            lib.fsa_attention_fwd.restype = I
            lib.fsa_attention_fwd_ex.argtypes = [V, V, V, V, I, I, I, I, I, F,
                                                 ctypes.POINTER(Options), V]
            lib.fsa_attention_fwd_ex.restype = I
            lib.fsa_attention_prepare.argtypes = [V, V, V, I, I, I, I, I, V, ctypes.c_uint64, V]
            lib.fsa_attention_prepare.restype = I
            lib.fsa_attention_run.argtypes = [V, ctypes.c_uint64, V, I, I, I, I, I, F,
                                              ctypes.POINTER(Options), V]
            lib.fsa_attention_run.restype = I
            lib.fsa_attention_workspace_size.argtypes = [I, I, I, I, I]
            lib.fsa_attention_workspace_size.restype = ctypes.c_uint64
            lib.fsa_cross_attention_fwd.argtypes = [V, V, V, V, I, I, I, I, I, I, F,
                                                    ctypes.POINTER(Options), V]
            lib.fsa_cross_attention_fwd.restype = I
            lib.fsa_cross_attention_workspace_size.argtypes = [I, I, I, I, I, I]
            lib.fsa_cross_attention_workspace_size.restype = ctypes.c_uint64
            lib.fsa_cross_attention_prepare.argtypes = [V, V, V, I, I, I, I, I, I, V,
                                                        ctypes.c_uint64, V]
            lib.fsa_cross_attention_prepare.restype = I
            lib.fsa_cross_attention_run.argtypes = [V, ctypes.c_uint64, V, I, I, I, I, I, I, F,
                                                    ctypes.POINTER(Options), V]
            lib.fsa_cross_attention_run.restype = I
            lib.fsa_attention_fwd_host.argtypes = [V, V, V, V, I, I, I, I, I, F,
                                                   ctypes.POINTER(Options), V]
            lib.fsa_attention_fwd_host.restype = I
            lib.fsa_cross_attention_fwd_host.argtypes = [V, V, V, V, I, I, I, I, I, I, F,
                                                         ctypes.POINTER(Options), V]
            lib.fsa_cross_attention_fwd_host.restype = I
            lib.fsa_attention_fwd_noalloc.argtypes = [V, V, V, V, I, I, I, I, I, F, V]
            lib.fsa_attention_fwd_noalloc.restype = I
            lib.fsa_bf16_attention_fwd.argtypes = [V, V, V, V, I, I, I, I, V]
            lib.fsa_bf16_attention_fwd.restype = I
            lib.fsa_mma_rate_probe.argtypes = [I, I, I, ctypes.POINTER(ctypes.c_double), V]
            lib.fsa_mma_rate_probe.restype = I
            lib.fsa_kv4_page_bytes.argtypes = [I, I, I]
            lib.fsa_kv4_page_bytes.restype = ctypes.c_uint64
            lib.fsa_kv4_append.argtypes = [V, V, I64, I64, V, I64, I, I, V, I64, I, V]
            lib.fsa_kv4_append.restype = I
            lib.fsa_kv4_read.argtypes = [V, I64, I, V, I64, I, I, V, V, I64, I64, V]
            lib.fsa_kv4_read.restype = I
            lib.fsa_kv4_attention_workspace_size.argtypes = [I, I, I, I, I, I, I]
            lib.fsa_kv4_attention_workspace_size.restype = ctypes.c_uint64
            lib.fsa_kv4_attention_fwd.argtypes = [V, I64, V, V, V, V, V, I, I, I, I, I, I64, I, I, F, V,
                                                  ctypes.c_uint64, V]
            lib.fsa_kv4_attention_fwd.restype = I
            lib.fsa_varlen_attention_fwd.argtypes = [V, V, V, I64, I64, I64, V, V, V, V, I, I, I, I, I, I, I, F, V]
            lib.fsa_varlen_attention_fwd.restype = I
            lib.fsa_kv4_attention_fwd_ex.argtypes = [V, I64, V, V, V, V, V, I, I, I, I, I, I64, I, I,
                                                     ctypes.POINTER(Options), V]
            lib.fsa_kv4_attention_fwd_ex.restype = I
            lib.fsa_varlen_attention_fwd_ex.argtypes = [V, V, V, I64, I64, I64, V, V, V, V, I, I, I, I, I, I, I,
                                                        ctypes.POINTER(Options), V]
            lib.fsa_varlen_attention_fwd_ex.restype = I
            lib.fsa_mx_pack.argtypes = [V, I64, I64, I64, I, V, V, V]
            lib.fsa_mx_pack.restype = I
            lib.fsa_mx_unpack.argtypes = [V, V, I64, I64, I, V, I64, V]
            lib.fsa_mx_unpack.restype = I
            lib.fsa_rms_norm_mx.argtypes = [V, I64, V, I64, V, F, I64, I64, I, V, I64, V, V, V]
            lib.fsa_rms_norm_mx.restype = I
            lib.fsa_rms_norm_mx_ex.argtypes = [V, I64, V, I64, V, F, I64, I64, I, V, I64, V, V, ctypes.POINTER(Options), V]
            lib.fsa_rms_norm_mx_ex.restype = I
            lib.fsa_mx_linear.argtypes = [V, V, I, V, V, I, I64, I64, I64, V, I64, ctypes.POINTER(Options), V]
            lib.fsa_mx_linear.restype = I
            lib.fsa_get_device_error.argtypes = [V]
            lib.fsa_get_device_error.restype = I
            lib.fsa_status_string.argtypes = [I]
            lib.fsa_status_string.restype = ctypes.c_char_p
            lib.fsa_release_workspace.argtypes = []
            lib.fsa_release_workspace.restype = None
            _lib = lib
    return _lib


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(status: int, what: str):
    if status != 0:
        raise FsaError(status, what)


def _bhsd(t: torch.Tensor, name: str):
    if t.dtype != torch.bfloat16 or not t.is_cuda or t.dim() != 4 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA bf16 tensor [B, H, S, D]")


def quantize_mx(x: torch.Tensor, block_axis: int, elem: int, stream=None):
    """MX-quantize x [batch, rows, cols] (bf16, CUDA).  Returns (codes, scales)
    in the layouts documented for fsa_quantize_mx."""
    if x.dtype != torch.bfloat16 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous CUDA bf16 tensor")
    x3 = x if x.dim() == 3 else x.reshape(1, *x.shape[-2:])
    b, r, c = x3.shape
    if block_axis == 1:
        codes = torch.empty((b, r, c), dtype=torch.uint8, device=x.device)
        scales = torch.empty((b, r, (c + 31) // 32), dtype=torch.uint8, device=x.device)
    else:
        codes = torch.empty((b, c, r), dtype=torch.uint8, device=x.device)
        scales = torch.empty((b, c, (r + 31) // 32), dtype=torch.uint8, device=x.device)
    _check(load().fsa_quantize_mx(_ptr(x3), b, r, c, block_axis, elem, _ptr(codes), _ptr(scales),
                                  _stream(stream)), "fsa_quantize_mx")
    return codes, scales


def workspace_size(B: int, H: int, S: int, D: int, fmt: str = "mxfp8") -> int:
    return int(load().fsa_attention_workspace_size(B, H, S, D, FORMATS[fmt]))


def attention_fwd(q, k, v, fmt: str = "mxfp8", threshold: float = 8.0, *, out=None,
                  sm_scale: float = 0.0, rollback_bits=None, rollback_count=None,
                  workspace=None, wait_timeout_ms: int = 0, efq_tau: float = 0.0, efq_h: float = 0.0, debug_flags: int = 0, gate: str = "fp32", stream=None):
    """Fused-Softmax MX attention forward (fsa_attention_fwd_ex).

    q, k, v: contiguous CUDA bf16 [B, H, S, D].  rollback_bits: optional uint8
    CUDA tensor [B*H*S, ceil(S/128)]; rollback_count: optional int64 CUDA
    tensor [1] to which the number of gate firings is added."""
    for n, t in (("q", q), ("k", k), ("v", v)):
        _bhsd(t, n)
    B, H, S, D = q.shape
    o = torch.empty_like(q) if out is None else out
    opt = Options()
    opt.sm_scale = sm_scale
    opt.rollback_bits = None if rollback_bits is None else rollback_bits.data_ptr()
    opt.rollback_count = None if rollback_count is None else rollback_count.data_ptr()
    if workspace is not None:
        opt.workspace = workspace.data_ptr()
        opt.workspace_bytes = workspace.numel() * workspace.element_size()
    opt.efq_tau, opt.efq_h = efq_tau, efq_h
    opt.gate_mode = GATE_MODES[gate]
    opt.wait_timeout_ms = wait_timeout_ms
    opt.debug_flags = debug_flags
    _check(load().fsa_attention_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, H, S, D,
                                       FORMATS[fmt], float(threshold), ctypes.byref(opt),
                                       _stream(stream)), "fsa_attention_fwd_ex")
    return o


def cross_attention_fwd(q, k, v, fmt: str = "mxfp8", threshold: float = 8.0, *, out=None,
                        sm_scale: float = 0.0, rollback_bits=None, rollback_count=None,
                        workspace=None, wait_timeout_ms: int = 0, efq_tau: float = 0.0, efq_h: float = 0.0, gate: str = "fp32", stream=None):
    """fsa_cross_attention_fwd: q contiguous CUDA bf16 [B, H, Sq, D], k and v
    [B, H, Sk, D]; returns o [B, H, Sq, D].  rollback_bits: optional uint8
    CUDA tensor [B*H*Sq, ceil(Sk/128)]."""
    for n, t in (("q", q), ("k", k), ("v", v)):
        _bhsd(t, n)
    B, H, Sq, D = q.shape
    Sk = k.shape[2]
    if k.shape != (B, H, Sk, D) or v.shape != k.shape:
        raise ValueError("k and v must be [B, H, Sk, D] with q's B, H and D")
    o = torch.empty_like(q) if out is None else out
    opt = Options()
    opt.sm_scale = sm_scale
    opt.rollback_bits = None if rollback_bits is None else rollback_bits.data_ptr()
    opt.rollback_count = None if rollback_count is None else rollback_count.data_ptr()
    if workspace is not None:
        opt.workspace = workspace.data_ptr()
        opt.workspace_bytes = workspace.numel() * workspace.element_size()
    opt.efq_tau, opt.efq_h = efq_tau, efq_h
    opt.gate_mode = GATE_MODES[gate]
    opt.wait_timeout_ms = wait_timeout_ms
    _check(load().fsa_cross_attention_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, H, Sq, Sk, D,
                                          FORMATS[fmt], float(threshold), ctypes.byref(opt),
                                          _stream(stream)), "fsa_cross_attention_fwd")
    return o


def _host_bhsd(t, name):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or t.is_cuda or t.dim() != 4 \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous host (CPU) bf16 tensor [B, H, S, D]")


def cross_attention_fwd_host(q, k, v, fmt: str = "mxfp8", threshold: float = 8.0, *, out=None,
                             sm_scale: float = 0.0, rollback_bits=None, rollback_count=None,
                             efq_tau: float = 0.0, efq_h: float = 0.0, host_inputs_ready: bool = False,
                             gate: str = "fp32", stream=None):
    """fsa_cross_attention_fwd_host: q, k, v contiguous HOST bf16 tensors
    ([B, H, Sq, D] and [B, H, Sk, D]; pinned memory lets the copies overlap
    the computation); returns the host output o [B, H, Sq, D] (or fills
    `out`).  Asynchronous on `stream`: synchronise it before reading o.
    rollback_bits / rollback_count, when given, are CUDA tensors.
    host_inputs_ready: q, k, v are final now (no earlier work on `stream`
    writes them), so their copy-in need not wait for that work."""
    for n, t in (("q", q), ("k", k), ("v", v)):
        _host_bhsd(t, n)
    B, H, Sq, D = q.shape
    Sk = k.shape[2]
    if k.shape != (B, H, Sk, D) or v.shape != k.shape:
        raise ValueError("k and v must be [B, H, Sk, D] with q's B, H and D")
    o = torch.empty(q.shape, dtype=torch.bfloat16, pin_memory=q.is_pinned()) if out is None else out
    _host_bhsd(o, "out")
    if o.shape != q.shape:
        raise ValueError("out must have q's shape")
    opt = Options()
    opt.sm_scale = sm_scale
    opt.rollback_bits = None if rollback_bits is None else rollback_bits.data_ptr()
    opt.rollback_count = None if rollback_count is None else rollback_count.data_ptr()
    opt.efq_tau, opt.efq_h = efq_tau, efq_h
    opt.gate_mode = GATE_MODES[gate]
    opt.host_inputs_ready = int(bool(host_inputs_ready))
    _check(load().fsa_cross_attention_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, H, Sq, Sk, D,
                                               FORMATS[fmt], float(threshold), ctypes.byref(opt),
                                               _stream(stream)), "fsa_cross_attention_fwd_host")
    return o


def attention_fwd_host(q, k, v, fmt: str = "mxfp8", threshold: float = 8.0, *, out=None,
                       sm_scale: float = 0.0, rollback_bits=None, rollback_count=None,
                       efq_tau: float = 0.0, efq_h: float = 0.0, host_inputs_ready: bool = False,
                       gate: str = "fp32", stream=None):
    """fsa_attention_fwd_host: self-attention on contiguous HOST bf16 tensors
    [B, H, S, D]; see cross_attention_fwd_host."""
    for n, t in (("q", q), ("k", k), ("v", v)):
        _host_bhsd(t, n)
    B, H, S, D = q.shape
    if k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k and v must have one shape [B, H, S, D]")
    o = torch.empty(q.shape, dtype=torch.bfloat16, pin_memory=q.is_pinned()) if out is None else out
    _host_bhsd(o, "out")
    if o.shape != q.shape:
        raise ValueError("out must have q's shape")
    opt = Options()
    opt.sm_scale = sm_scale
    opt.rollback_bits = None if rollback_bits is None else rollback_bits.data_ptr()
    opt.rollback_count = None if rollback_count is None else rollback_count.data_ptr()
    opt.efq_tau, opt.efq_h = efq_tau, efq_h
    opt.gate_mode = GATE_MODES[gate]
    opt.host_inputs_ready = int(bool(host_inputs_ready))
    _check(load().fsa_attention_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, H, S, D,
                                         FORMATS[fmt], float(threshold), ctypes.byref(opt),
                                         _stream(stream)), "fsa_attention_fwd_host")
    return o


def cross_workspace_size(B: int, H: int, Sq: int, Sk: int, D: int, fmt: str = "mxfp8") -> int:
    return int(load().fsa_cross_attention_workspace_size(B, H, Sq, Sk, D, FORMATS[fmt]))


def new_cross_workspace(B: int, H: int, Sq: int, Sk: int, D: int, fmt: str = "mxfp8", device="cuda"):
    """A device workspace tensor sized for cross_attention_prepare / _run."""
    return torch.empty(cross_workspace_size(B, H, Sq, Sk, D, fmt), dtype=torch.uint8, device=device)


def cross_attention_prepare(q, k, v, workspace, fmt: str = "mxfp8", stream=None):
    """First half of cross_attention_fwd: MX-quantize q, k, v into `workspace`."""
    for n, t in (("q", q), ("k", k), ("v", v)):
        _bhsd(t, n)
    B, H, Sq, D = q.shape
    Sk = k.shape[2]
    _check(load().fsa_cross_attention_prepare(_ptr(q), _ptr(k), _ptr(v), B, H, Sq, Sk, D,
                                              FORMATS[fmt], _ptr(workspace), workspace.numel(),
                                              _stream(stream)), "fsa_cross_attention_prepare")


def cross_attention_run(workspace, out, Sk: int, fmt: str = "mxfp8", threshold: float = 8.0, *,
                        sm_scale: float = 0.0, rollback_bits=None, rollback_count=None,
                        wait_timeout_ms: int = 0, efq_tau: float = 0.0, efq_h: float = 0.0, gate: str = "fp32", stream=None):
    """Second half of cross_attention_fwd: `out` [B, H, Sq, D] fixes B, H, Sq and D;
    Sk is the key length given to cross_attention_prepare."""
    _bhsd(out, "out")
    B, H, Sq, D = out.shape
    opt = Options()
    opt.sm_scale = sm_scale
    opt.rollback_bits = None if rollback_bits is None else rollback_bits.data_ptr()
    opt.rollback_count = None if rollback_count is None else rollback_count.data_ptr()
    opt.efq_tau, opt.efq_h = efq_tau, efq_h
    opt.gate_mode = GATE_MODES[gate]
    opt.wait_timeout_ms = wait_timeout_ms
    _check(load().fsa_cross_attention_run(_ptr(workspace), workspace.numel(), _ptr(out), B, H, Sq,
                                          Sk, D, FORMATS[fmt], float(threshold), ctypes.byref(opt),
                                          _stream(stream)), "fsa_cross_attention_run")
    return out


def new_workspace(B: int, H: int, S: int, D: int, fmt: str = "mxfp8", device="cuda"):
    """A device workspace tensor sized for attention_prepare / attention_run."""
    return torch.empty(workspace_size(B, H, S, D, fmt), dtype=torch.uint8, device=device)


def attention_prepare(q, k, v, workspace, fmt: str = "mxfp8", stream=None):
    """First half of attention_fwd: MX-quantize q, k, v into `workspace`."""
    for n, t in (("q", q), ("k", k), ("v", v)):
        _bhsd(t, n)
    B, H, S, D = q.shape
    _check(load().fsa_attention_prepare(_ptr(q), _ptr(k), _ptr(v), B, H, S, D, FORMATS[fmt],
                                        _ptr(workspace), workspace.numel(), _stream(stream)),
           "fsa_attention_prepare")


def attention_run(workspace, out, fmt: str = "mxfp8", threshold: float = 8.0, *,
                  sm_scale: float = 0.0, rollback_bits=None, rollback_count=None,
                  wait_timeout_ms: int = 0, efq_tau: float = 0.0, efq_h: float = 0.0, gate: str = "fp32", stream=None):
    """Second half of attention_fwd: the fused kernel on a prepared workspace;
    `out` is the bf16 [B, H, S, D] output and fixes the shape."""
    _bhsd(out, "out")
    B, H, S, D = out.shape
    opt = Options()
    opt.sm_scale = sm_scale
    opt.rollback_bits = None if rollback_bits is None else rollback_bits.data_ptr()
    opt.rollback_count = None if rollback_count is None else rollback_count.data_ptr()
    opt.efq_tau, opt.efq_h = efq_tau, efq_h
    opt.gate_mode = GATE_MODES[gate]
    opt.wait_timeout_ms = wait_timeout_ms
    _check(load().fsa_attention_run(_ptr(workspace), workspace.numel(), _ptr(out), B, H, S, D,
                                    FORMATS[fmt], float(threshold), ctypes.byref(opt),
                                    _stream(stream)), "fsa_attention_run")
    return out


def attention_fwd_noalloc(q, k, v, fmt: str = "mxfp8", threshold: float = 8.0, *, out=None,
                          stream=None):
    """fsa_attention_fwd_noalloc: the fused attention with the library's fixed
    64 MiB scratch array instead of an allocated workspace (see include/fsa.h)."""
    for n, t in (("q", q), ("k", k), ("v", v)):
        _bhsd(t, n)
    B, H, S, D = q.shape
    o = torch.empty_like(q) if out is None else out
    _check(load().fsa_attention_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, H, S, D,
                                            FORMATS[fmt], float(threshold), _stream(stream)),
           "fsa_attention_fwd_noalloc")
    return o


def bf16_attention_fwd(q, k, v, *, out=None, stream=None):
    """Conventional BF16 flash attention (fsa_bf16_attention_fwd)."""
    for n, t in (("q", q), ("k", k), ("v", v)):
        _bhsd(t, n)
    B, H, S, D = q.shape
    o = torch.empty_like(q) if out is None else out
    _check(load().fsa_bf16_attention_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, H, S, D,
                                         _stream(stream)), "fsa_bf16_attention_fwd")
    return o


# ---- four-bit key/value cache and packed sequences --------------------------


# These calls are short (a decoding step makes several per layer), so the checks
# look at each property of a tensor once, and the current device and stream are
# read directly.

_raw_stream = torch._C._cuda_getCurrentRawStream
_device = torch._C._cuda_getDevice
_bf16, _f32, _i32, _i64, _u8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8


def _on(t, stream):
    """Makes `stream` (by default the current one of t's device) and its device
    current: what the call allocates then belongs to that stream."""
    s = torch.cuda.current_stream(t.device) if stream is None else stream
    if s.device != t.device:
        raise ValueError("stream and tensors are on different devices")
    return torch.cuda.stream(s)


def _heads(t: torch.Tensor, name: str, shape, dev: int):
    """A CUDA bf16 tensor [..., heads, D] of the given shape whose heads are
    contiguous; returns its strides."""
    st = t.stride()
    if t.dtype is not _bf16 or t.shape != shape or t.get_device() != dev:
        raise ValueError(f"{name} must be a bf16 tensor {list(shape)} on cuda:{dev}")
    if st[-1] != 1 or (st[-2] != shape[-1] and shape[-2] > 1):
        raise ValueError(f"the heads of {name} must be contiguous")
    return st


def _plain(t: torch.Tensor, name: str, dtype, shape, dev: int):
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on cuda:{dev}")
    return t


def kv4_new_cache(num_pages: int, page_size: int, n_kv_heads: int, D: int, device="cuda") -> torch.Tensor:
    """An empty four-bit key/value cache: uint8 [num_pages, n_kv_heads,
    page_size / 32, 34 * D] (layout: include/fsa.h), all zero."""
    if num_pages < 1 or not load().fsa_kv4_page_bytes(n_kv_heads, page_size, D):
        raise ValueError("a cache needs pages of a positive multiple of 32 tokens (at most 65536), "
                         "1 to 65535 heads and D 64 or 128")
    return torch.zeros((num_pages, n_kv_heads, page_size // 32, 34 * D), dtype=torch.uint8, device=device)


def _kv4(cache: torch.Tensor):
    """(pages, heads, page_size, D) of a cache tensor."""
    if cache.dtype is not _u8 or cache.get_device() < 0 or cache.dim() != 4 or not cache.is_contiguous():
        raise ValueError("cache must be a contiguous CUDA uint8 tensor [pages, heads, page_size / 32, 34 * D]")
    pages, heads, groups, last = cache.shape
    if last != 4352 and last != 2176:
        raise ValueError("the last dimension of a cache is 34 * D with D 64 or 128")
    return pages, heads, 32 * groups, last // 34


def kv4_append(cache, k, v, slots, stream=None):
    """fsa_kv4_append: quantizes k and v, CUDA bf16 [T, n_kv_heads, D] (heads
    contiguous, any token stride), into the cache at `slots`, int64 [T] =
    page * page_size + token; a negative slot skips its token."""
    pages, H, page_size, D = _kv4(cache)
    dev = cache.get_device()
    if stream is not None or dev != _device():
        with _on(cache, stream):
            return kv4_append(cache, k, v, slots)
    T = slots.numel()
    shape = (T, H, D)
    _plain(slots, "slots", _i64, (T,), dev)
    ks, vs = _heads(k, "k", shape, dev)[0], _heads(v, "v", shape, dev)[0]
    if T < 2:  # (a lone token's stride is arbitrary)
        ks = vs = H * D
    _check(load().fsa_kv4_append(k.data_ptr(), v.data_ptr(), ks, vs, slots.data_ptr(), T, H, D, cache.data_ptr(), pages,
                                 page_size, _raw_stream(dev)), "fsa_kv4_append")


def kv4_read(cache, slots, *, out_k=None, out_v=None, stream=None):
    """fsa_kv4_read: (k, v), the values that the cache holds at `slots` (int64
    [T]) as bf16 [T, n_kv_heads, D]; a negative slot reads as zeros.  out_k,
    out_v: written instead of new tensors (heads contiguous, tokens that do not
    overlap)."""
    pages, H, page_size, D = _kv4(cache)
    dev = cache.get_device()
    if stream is not None or dev != _device():
        with _on(cache, stream):
            return kv4_read(cache, slots, out_k=out_k, out_v=out_v)
    T = slots.numel()
    shape = (T, H, D)
    _plain(slots, "slots", _i64, (T,), dev)
    ks = vs = H * D
    if out_k is None:
        out_k = torch.empty(shape, dtype=_bf16, device=cache.device)
    else:
        st = _heads(out_k, "out_k", shape, dev)
        ks = st[0] if T > 1 else ks
    if out_v is None:
        out_v = torch.empty(shape, dtype=_bf16, device=cache.device)
    else:
        st = _heads(out_v, "out_v", shape, dev)
        vs = st[0] if T > 1 else vs
    _check(load().fsa_kv4_read(cache.data_ptr(), pages, page_size, slots.data_ptr(), T, H, D, out_k.data_ptr(),
                               out_v.data_ptr(), ks, vs, _raw_stream(dev)), "fsa_kv4_read")
    return out_k, out_v


@functools.lru_cache(maxsize=1024)
def kv4_attention_workspace_size(B: int, Sq: int, n_heads: int, n_kv_heads: int, D: int, page_size: int,
                                 max_pages: int) -> int:
    """Bytes of workspace of kv4_attention_fwd (fsa_kv4_attention_workspace_size)."""
    return int(load().fsa_kv4_attention_workspace_size(B, Sq, n_heads, n_kv_heads, D, page_size, max_pages))


def kv4_attention_fwd(q, cache, page_table, seq_lens, *, out=None, return_lse: bool = False, lse=None,
                      sm_scale: float = 0.0, workspace=None, wait_timeout_ms: int = 0, debug_flags: int = 0, stream=None):
    """fsa_kv4_attention_fwd: attention of q, CUDA bf16 [B, Sq, n_heads, D] (the
    last Sq tokens of each sequence, already in the cache; heads contiguous, all
    tokens at one distance), over the four-bit cache.  page_table int32 [B,
    max_pages], seq_lens int32 [B] (keys of each sequence, its query tokens
    included).  Returns o [B, Sq, n_heads, D], with return_lse also the
    log-sum-exps, float32 [B, Sq, n_heads] (written into `lse` if given).
    workspace: uint8 tensor of kv4_attention_workspace_size bytes for callers
    that keep one; calls that may overlap need their own.  wait_timeout_ms: limit
    of the kernels' bounded waits (0: 2000)."""
    pages, Hkv, page_size, D = _kv4(cache)
    dev = cache.get_device()
    if stream is not None or dev != _device():
        with _on(cache, stream):
            return kv4_attention_fwd(q, cache, page_table, seq_lens, out=out, return_lse=return_lse, lse=lse,
                                     sm_scale=sm_scale, workspace=workspace, wait_timeout_ms=wait_timeout_ms,
                                     debug_flags=debug_flags)
    if q.dim() != 4 or page_table.dim() != 2:
        raise ValueError("q must be [B, Sq, n_heads, D] and page_table [B, max_pages]")
    shape = q.shape
    B, Sq, Hq, Dq = shape
    if Hkv == 0 or Dq != D or Hq % Hkv or Sq * Hq == 0:
        raise ValueError(f"q must be [B, Sq, n_heads, {D}] with a query token and a multiple of {Hkv} heads")
    st = _heads(q, "q", shape, dev)
    q_stride = st[1] if Sq > 1 else st[0] if B > 1 else Hq * D
    if B > 1 and st[0] != Sq * q_stride:
        raise ValueError("the tokens of q must lie at one distance")
    max_pages = page_table.shape[1]
    _plain(page_table, "page_table", _i32, (B, max_pages), dev)
    _plain(seq_lens, "seq_lens", _i32, (B,), dev)
    o = torch.empty(shape, dtype=_bf16, device=cache.device) if out is None else _plain(out, "out", _bf16, shape, dev)
    if lse is not None:
        _plain(lse, "lse", _f32, (B, Sq, Hq), dev)
    elif return_lse:
        lse = torch.empty((B, Sq, Hq), dtype=_f32, device=cache.device)
    if B == 0:
        return (o, lse) if return_lse else o
    ws, ws_bytes = None, kv4_attention_workspace_size(B, Sq, Hq, Hkv, D, page_size, max_pages)
    if workspace is not None:
        if not workspace.is_contiguous() or workspace.get_device() != dev:
            raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
        ws, ws_bytes = workspace, workspace.numel() * workspace.element_size()
    elif ws_bytes:
        ws = torch.empty(ws_bytes, dtype=_u8, device=cache.device)
    args = (q.data_ptr(), q_stride, cache.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(), o.data_ptr(),
            None if lse is None else lse.data_ptr(), B, Sq, Hq, Hkv, D, pages, page_size, max_pages)
    if wait_timeout_ms or debug_flags:
        opt = Options(sm_scale=sm_scale, workspace=None if ws is None else ws.data_ptr(), workspace_bytes=ws_bytes,
                      wait_timeout_ms=wait_timeout_ms, debug_flags=debug_flags)
        _check(load().fsa_kv4_attention_fwd_ex(*args, ctypes.byref(opt), _raw_stream(dev)), "fsa_kv4_attention_fwd_ex")
    else:
        _check(load().fsa_kv4_attention_fwd(*args, sm_scale, None if ws is None else ws.data_ptr(), ws_bytes,
                                            _raw_stream(dev)), "fsa_kv4_attention_fwd")
    return (o, lse) if return_lse else o


def varlen_attention_fwd(q, k, v, cu_seqlens_q, cu_seqlens_k=None, *, causal: bool = True, out=None,
                         return_lse: bool = False, lse=None, sm_scale: float = 0.0, wait_timeout_ms: int = 0,
                         debug_flags: int = 0, stream=None):
    """fsa_varlen_attention_fwd: BF16 attention over packed sequences.  q CUDA
    bf16 [Tq, n_heads, D], k and v [Tk, n_kv_heads, D] (heads contiguous, any
    token stride that keeps tokens apart); cu_seqlens_q and cu_seqlens_k (by
    default the same) int32 [B + 1].  Returns o [Tq, n_heads, D], with
    return_lse also the log-sum-exps, float32 [Tq, n_heads].  Rows outside every
    sequence are not written (a new output leaves them undefined).
    wait_timeout_ms: limit of the kernel's bounded waits (0: 2000)."""
    dev = q.get_device()
    if dev < 0:
        raise ValueError("q must be a CUDA tensor")
    if stream is not None or dev != _device():
        with _on(q, stream):
            return varlen_attention_fwd(q, k, v, cu_seqlens_q, cu_seqlens_k, causal=causal, out=out,
                                        return_lse=return_lse, lse=lse, sm_scale=sm_scale,
                                        wait_timeout_ms=wait_timeout_ms, debug_flags=debug_flags)
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q must be [Tq, n_heads, D], k and v [Tk, n_kv_heads, D]")
    cu_k = cu_seqlens_q if cu_seqlens_k is None else cu_seqlens_k
    qshape, kshape = q.shape, k.shape
    Tq, Hq, D = qshape
    Tk, Hkv, Dk = kshape
    if D != Dk or Hkv == 0 or Hq == 0 or Hq % Hkv:
        raise ValueError("k and v must be [Tk, n_kv_heads, D] with q's D and a head count that divides q's")
    qs, ks, vs = _heads(q, "q", qshape, dev)[0], _heads(k, "k", kshape, dev)[0], _heads(v, "v", kshape, dev)[0]
    if Tq < 2:  # (a lone token's stride is arbitrary)
        qs = Hq * D
    if Tk < 2:
        ks = vs = Hkv * D
    nb = cu_seqlens_q.numel()
    if nb < 2:
        raise ValueError("cu_seqlens_q must have B + 1 >= 2 entries")
    _plain(cu_seqlens_q, "cu_seqlens_q", _i32, (nb,), dev)
    if cu_seqlens_k is not None:
        _plain(cu_k, "cu_seqlens_k", _i32, (nb,), dev)
    o = torch.empty(qshape, dtype=_bf16, device=q.device) if out is None else _plain(out, "out", _bf16, qshape, dev)
    if lse is not None:
        _plain(lse, "lse", _f32, (Tq, Hq), dev)
    elif return_lse:
        lse = torch.empty((Tq, Hq), dtype=_f32, device=q.device)
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs, cu_seqlens_q.data_ptr(), cu_k.data_ptr(), o.data_ptr(),
            None if lse is None else lse.data_ptr(), nb - 1, Tq, Tk, Hq, Hkv, D, 1 if causal else 0)
    if wait_timeout_ms or debug_flags:
        opt = Options(sm_scale=sm_scale, wait_timeout_ms=wait_timeout_ms, debug_flags=debug_flags)
        _check(load().fsa_varlen_attention_fwd_ex(*args, ctypes.byref(opt), _raw_stream(dev)),
               "fsa_varlen_attention_fwd_ex")
    else:
        _check(load().fsa_varlen_attention_fwd(*args, sm_scale, _raw_stream(dev)), "fsa_varlen_attention_fwd")
    return (o, lse) if return_lse else o


# ---- products of matrices in MX formats --------------------------------------


def _empty_dispatched(size, stride, dtype) -> torch.Tensor:
    return torch.empty_strided(size, stride, dtype=dtype, device="cuda")


# New tensors on the current device, past torch's dispatcher where this torch has such a
# function (of two calls that pack a token and read it back, 11.8 us of host time with it,
# 19.6 with torch.empty and a storage for the operand).
try:
    _empty_cuda = torch._C._dynamo.guards._empty_strided_cuda
except AttributeError:
    _empty_cuda = _empty_dispatched

# element and bytes of 128 codes of a row
_OPERANDS = {"mxfp4": (ELEM_E2M1, 64), "mxfp8": (ELEM_E4M3, 128)}


def _operand_format(fmt: str):
    try:
        return _OPERANDS[fmt]
    except KeyError:
        raise ValueError(f"an operand's format is mxfp4 or mxfp8, not {fmt!r}") from None


class MxOperand:
    """A matrix [rows, cols] in an MX format as an operand of mx_linear (layout:
    include/fsa.h): codes uint8 [rows, ceil(cols / 128) * 64 ("mxfp4") or * 128
    ("mxfp8")], scales uint8 [ceil(rows / 128), ceil(cols / 128), 512].

    MxOperand(codes, scales, cols, fmt) is one of given tensors; mx_new_operand, mx_pack
    and rms_norm_mx make one of a single tensor of bytes, of which codes and scales are
    views that are made when they are asked for.

    The tensors that mx_pack, mx_unpack, rms_norm_mx and mx_linear make do not pass
    torch's dispatcher: dispatch modes and the deterministic fill of empty tensors do not
    see them (what a call does not write of them are scale bytes of rows behind the last)."""
    __slots__ = ("rows", "cols", "fmt", "elem", "_dev", "_bytes", "_codes", "_scales")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, cols: int, fmt: str):
        elem, width = _operand_format(fmt)
        atoms, shape = (cols + 127) >> 7, codes.shape
        rows = shape[0] if shape else 0
        if cols < 1 or shape != (rows, atoms * width) or scales.shape != ((rows + 127) >> 7, atoms, 512):
            raise ValueError(f"codes {list(shape)} and scales {list(scales.shape)} are not those of {cols} columns in {fmt}")
        if codes.dtype is not _u8 or scales.dtype is not _u8 or codes.get_device() != scales.get_device():
            raise ValueError("codes and scales must be uint8 tensors on one device")
        if not codes.is_contiguous() or not scales.is_contiguous():
            raise ValueError("codes and scales must be contiguous")
        self.rows, self.cols, self.fmt, self.elem = rows, cols, fmt, elem
        self._dev, self._bytes, self._codes, self._scales = codes.get_device(), None, codes, scales

    @classmethod
    def _new(cls, rows: int, cols: int, fmt: str, dev: int, device=None):
        """An operand with arbitrary contents on the current CUDA device dev, or on `device`."""
        elem, width = _operand_format(fmt)
        if rows < 0 or cols < 1:
            raise ValueError("an operand has at least one column")
        self = cls.__new__(cls)
        atoms = (cols + 127) >> 7
        size = atoms * (rows * width + ((rows + 127) >> 7) * 512)
        if device is None:
            data = _empty_cuda((size,), (1,), _u8)
        else:
            data = torch.empty(size, dtype=_u8, device=device)
            dev = data.get_device()
        self.rows, self.cols, self.fmt, self.elem = rows, cols, fmt, elem
        self._dev, self._bytes, self._codes, self._scales = dev, data, None, None
        return self

    def _pointers(self):
        if self._bytes is None:
            return self._codes.data_ptr(), self._scales.data_ptr()
        at = self._bytes.data_ptr()
        return at, at + self.rows * ((self.cols + 127) >> 7) * _OPERANDS[self.fmt][1]

    def _split(self):
        atoms, width = (self.cols + 127) >> 7, _OPERANDS[self.fmt][1]
        size = self.rows * atoms * width
        self._codes = self._bytes[:size].view(self.rows, atoms * width)
        self._scales = self._bytes[size:].view((self.rows + 127) >> 7, atoms, 512)

    @property
    def codes(self) -> torch.Tensor:
        if self._codes is None:
            self._split()
        return self._codes

    @property
    def scales(self) -> torch.Tensor:
        if self._scales is None:
            self._split()
        return self._scales

    @property
    def device(self) -> torch.device:
        return (self._codes if self._bytes is None else self._bytes).device

    def __reduce__(self):  # copies and files hold the two tensors
        return MxOperand, (self.codes, self.scales, self.cols, self.fmt)

    def __repr__(self):
        return f"MxOperand(rows={self.rows}, cols={self.cols}, fmt={self.fmt!r}, device={str(self.device)!r})"


def mx_new_operand(rows: int, cols: int, fmt: str, device="cuda") -> MxOperand:
    """An operand whose contents are arbitrary, for mx_pack and rms_norm_mx to fill."""
    return MxOperand._new(rows, cols, fmt, -1, device)


def _rows(t: torch.Tensor, name: str, shape, dev: int) -> int:
    """A CUDA bf16 tensor [rows, cols] of the given shape whose rows are contiguous;
    returns their distance."""
    if t.dtype is not _bf16 or t.shape != shape or t.get_device() != dev:
        raise ValueError(f"{name} must be a bf16 tensor {list(shape)} on cuda:{dev}")
    step, one = t.stride()
    if one != 1 and shape[1] > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return step if shape[0] > 1 else shape[1]  # (a lone row's stride is arbitrary)


def _new_rows(rows: int, cols: int) -> torch.Tensor:
    """bf16 [rows, cols] with arbitrary contents on the current device."""
    return _empty_cuda((rows, cols), (cols, 1), _bf16)


def _filled(out, shape, fmt: str, dev: int) -> MxOperand:
    """The operand that a call fills, new or given."""
    if out is None:
        return MxOperand._new(*shape, fmt, dev)
    if (out.rows, out.cols) != tuple(shape) or out.fmt != fmt or out._dev != dev:
        raise ValueError(f"out must be an operand of {list(shape)} in {fmt} on cuda:{dev}")
    return out


def mx_pack(x, fmt: str = "mxfp4", *, out=None, stream=None) -> MxOperand:
    """fsa_mx_pack: x, CUDA bf16 [rows, cols] (contiguous rows at any distance),
    quantized into an operand of mx_linear (`out`, or a new one)."""
    dev, shape = x.get_device(), x.shape
    if dev < 0 or len(shape) != 2:
        raise ValueError("x must be a CUDA tensor [rows, cols]")
    if stream is not None or dev != _device():
        with _on(x, stream):
            return mx_pack(x, fmt, out=out)
    step = _rows(x, "x", shape, dev)
    op = _filled(out, shape, fmt, dev)
    _check(load().fsa_mx_pack(x.data_ptr(), step, *shape, op.elem, *op._pointers(), _raw_stream(dev)), "fsa_mx_pack")
    return op


def mx_unpack(op: MxOperand, *, out=None, stream=None):
    """fsa_mx_unpack: an operand's values as bf16 [rows, cols]."""
    dev = op._dev
    if dev < 0:
        raise ValueError("op must be an operand on a CUDA device")
    if stream is not None or dev != _device():
        with _on(op, stream):
            return mx_unpack(op, out=out)
    rows, cols = op.rows, op.cols
    if out is None:
        out, step = _new_rows(rows, cols), cols
    else:
        step = _rows(out, "out", (rows, cols), dev)
    _check(load().fsa_mx_unpack(*op._pointers(), rows, cols, op.elem, out.data_ptr(), step, _raw_stream(dev)), "fsa_mx_unpack")
    return out


def rms_norm_mx(x, gain, *, residual=None, eps: float = 1e-6, fmt: str = "mxfp8", out=None, out_sum=None,
                wait_timeout_ms: int = 0, debug_flags: int = 0, stream=None):
    """fsa_rms_norm_mx: the root-mean-square norm of x, CUDA bf16 [rows, cols]
    (contiguous rows at any distance), times gain, bf16 [cols], as an operand of
    mx_linear.  With a residual, bf16 like x, the norm is that of h = x + residual
    (rounded to bf16), and (operand, h) is returned; out_sum, written instead of a new
    tensor, may be x or residual itself.  wait_timeout_ms: limit of the kernel's bounded
    waits (0: 2000)."""
    dev, shape = x.get_device(), x.shape
    if dev < 0 or len(shape) != 2:
        raise ValueError("x must be a CUDA tensor [rows, cols]")
    if stream is not None or dev != _device():
        with _on(x, stream):
            return rms_norm_mx(x, gain, residual=residual, eps=eps, fmt=fmt, out=out, out_sum=out_sum,
                               wait_timeout_ms=wait_timeout_ms, debug_flags=debug_flags)
    step, res, res_step, total, total_step = _rows(x, "x", shape, dev), None, 0, None, 0
    _plain(gain, "gain", _bf16, shape[1:], dev)
    if residual is not None:
        res_step, res = _rows(residual, "residual", shape, dev), residual.data_ptr()
        if out_sum is None:
            out_sum, total_step = _new_rows(*shape), shape[1]
        else:
            total_step = _rows(out_sum, "out_sum", shape, dev)
        total = out_sum.data_ptr()
    elif out_sum is not None:
        raise ValueError("there is no sum without a residual")
    op = _filled(out, shape, fmt, dev)
    opt = None
    if wait_timeout_ms or debug_flags:
        opt = ctypes.byref(Options(wait_timeout_ms=wait_timeout_ms, debug_flags=debug_flags))
    _check(load().fsa_rms_norm_mx_ex(x.data_ptr(), step, res, res_step, gain.data_ptr(), eps, *shape, op.elem, total, total_step,
                                     *op._pointers(), opt, _raw_stream(dev)), "fsa_rms_norm_mx")
    return op if residual is None else (op, out_sum)


def mx_linear(x: MxOperand, w: MxOperand, *, out=None, wait_timeout_ms: int = 0, debug_flags: int = 0, stream=None):
    """fsa_mx_linear: y = x w^T of two operands, activations [T, K] and a weight [N,
    K], as bf16 [T, N].  Formats of x and w: mxfp4 and mxfp4, mxfp8 and mxfp4, mxfp8
    and mxfp8.  out: written instead of a new tensor (contiguous rows at any distance
    that keeps them apart).  wait_timeout_ms: limit of the kernel's bounded waits (0:
    2000)."""
    dev = x._dev
    if dev < 0 or w._dev != dev:
        raise ValueError("x and w must be operands on one CUDA device")
    if stream is not None or dev != _device():
        with _on(x, stream):
            return mx_linear(x, w, out=out, wait_timeout_ms=wait_timeout_ms, debug_flags=debug_flags)
    T, N, K = x.rows, w.rows, x.cols
    if w.cols != K:
        raise ValueError(f"x has {K} columns and w {w.cols}")
    if out is None:
        out, step = _new_rows(T, N), N
    else:
        step = _rows(out, "out", (T, N), dev)
    opt = None
    if wait_timeout_ms or debug_flags:
        opt = ctypes.byref(Options(wait_timeout_ms=wait_timeout_ms, debug_flags=debug_flags))
    _check(load().fsa_mx_linear(*x._pointers(), x.elem, *w._pointers(), w.elem, T, N, K, out.data_ptr(), step, opt,
                                _raw_stream(dev)), "fsa_mx_linear")
    return out


# kinds of fsa_mma_rate_probe
PROBE_KINDS = {"mxf8f6f4_e4m3": 0, "mxf8f6f4_e2m3": 1, "mxf4_e2m1": 2, "attention_tile_e4m3": 3,
               "f16_bf16": 4}


def mma_rate_probe(kind: str, ctas: int, iters: int, stream=None) -> float:
    """fsa_mma_rate_probe: launches the tensor-core rate probe on the stream
    (the caller times it) and returns the launch's floating-point operations."""
    fl = ctypes.c_double(0.0)
    _check(load().fsa_mma_rate_probe(PROBE_KINDS[kind], int(ctas), int(iters), ctypes.byref(fl),
                                     _stream(stream)), "fsa_mma_rate_probe")
    return fl.value


def get_device_error(stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device error status."""
    return int(load().fsa_get_device_error(_stream(stream)))


def status_string(s: int) -> str:
    return load().fsa_status_string(int(s)).decode()


def release_workspace():
    load().fsa_release_workspace()
