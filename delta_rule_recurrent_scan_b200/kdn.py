"""Thin ctypes binding over libkdn.so (the C ABI declared in include/kdn.h).

Argument marshalling only: it checks torch tensors (device, dtype,
contiguity), allocates outputs and default initial states, and passes raw
pointers plus the current CUDA stream to the library.  The read-out o defaults
to fp32: rounding it to bf16 alone costs up to 2^-8 of its magnitude, more than
the 3e-3 the scan is held to; pass out_dtype=torch.bfloat16 to halve its bytes.  Every step of the scan
runs in the library's kernels.  There is no fallback: if the library is
missing or the tensors are not on a CUDA device, the call raises.

Every scan takes ``segments`` (kdn_dims.segments): 0 lets the library cut each
head's sequence into several segments scanned by separate CTAs when there are
too few heads to fill the GPU, 1 forces one serial pass per head, P >= 2 asks
for P segments (P must divide L).  Results agree up to rounding.
"""

from __future__ import annotations

import contextlib
import ctypes
import os
import re
from dataclasses import dataclass

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB_PATH = os.path.join(PKG, "lib", "libkdn.so")
HEADER = os.path.join(ROOT, "include", "kdn.h")

KDN_OK, KDN_ERR_INVALID_ARG, KDN_ERR_UNSUPPORTED, KDN_ERR_CUDA, KDN_ERR_NUMERIC, KDN_ERR_TIMEOUT = range(6)
KDN_ERR_CAPACITY = 6
KDN_F32, KDN_BF16 = 0, 1
VARIANTS = {"delta": 0, "kalman_diag": 1, "kalman_full": 2, "kalman_iso": 3}
_DTYPES = {torch.float32: KDN_F32, torch.bfloat16: KDN_BF16}


class KdnError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


class Dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("L", ctypes.c_int), ("dk", ctypes.c_int),
                ("dv", ctypes.c_int), ("chunk", ctypes.c_int), ("in_dtype", ctypes.c_int),
                ("out_dtype", ctypes.c_int), ("segments", ctypes.c_int)]


class PagesC(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("rows", ctypes.c_int),
                ("max_pages", ctypes.c_int), ("table", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("refs", ctypes.c_void_p)]


_lib = None


def exported_names() -> list[str]:
    """The entry points include/kdn.h declares."""
    with open(HEADER) as f:
        return re.findall(r"^KDN_EXPORT\s+[\w\s\*]+?\b(kdn_\w+)\s*\(", f.read(), flags=re.M)


def lib() -> ctypes.CDLL:
    """Open libkdn.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise FileNotFoundError(f"{LIB_PATH} is missing: build it with python -m delta_rule_recurrent_scan_b200.build")
    L = ctypes.CDLL(LIB_PATH)
    vp, sz, i, f = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
    dims = ctypes.POINTER(Dims)
    L.kdn_scan_delta.argtypes = [dims, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.kdn_scan_kalman_full.argtypes = [dims, vp, vp, vp, vp, vp, vp, f, vp, vp, vp, vp, vp, sz, vp]
    L.kdn_scan_kalman_diag.argtypes = [dims, vp, vp, vp, vp, vp, vp, f, vp, vp, vp, vp, vp, sz, vp]
    L.kdn_scan_kalman_iso.argtypes = [dims, vp, vp, vp, vp, vp, vp, f, vp, vp, vp, vp, vp, sz, vp]
    L.kdn_hola_cache_read.argtypes = [dims, vp, vp, vp, vp, vp, vp, vp, i, vp, vp, vp, sz, vp]
    L.kdn_decode_step.argtypes = [i, i, i, i, i, i, i, vp, vp, vp, vp, vp, vp, f, vp, vp, vp, vp, vp]
    L.kdn_scan_kalman_full_noalloc.argtypes = [dims, vp, vp, vp, vp, vp, vp, f, vp, vp, vp, vp, vp]
    L.kdn_scan_kalman_full_noalloc.restype = ctypes.c_int
    L.kdn_workspace_bytes.argtypes = [i, dims]
    L.kdn_workspace_bytes.restype = sz
    L.kdn_read_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_int), vp]
    L.kdn_scan_delta_backward.argtypes = [dims] + [vp] * 16 + [sz, vp]
    L.kdn_scan_delta_backward.restype = ctypes.c_int
    L.kdn_hola_workspace_bytes.argtypes = [dims]
    L.kdn_hola_workspace_bytes.restype = sz
    L.kdn_scan_kalman_iso_backward.argtypes = [dims, vp, vp, vp, vp, vp, vp, f] + [vp] * 14 + [vp, sz, vp]
    L.kdn_scan_kalman_iso_backward.restype = ctypes.c_int
    L.kdn_scan_kalman_diag_backward.argtypes = [dims, vp, vp, vp, vp, vp, vp, f] + [vp] * 14 + [vp, sz, vp]
    L.kdn_scan_kalman_diag_backward.restype = ctypes.c_int
    L.kdn_scan_kalman_full_backward.argtypes = [dims, vp, vp, vp, vp, vp, vp, f] + [vp] * 14 + [vp, sz, vp]
    L.kdn_scan_kalman_full_backward.restype = ctypes.c_int
    L.kdn_backward_workspace_bytes.argtypes = [i, dims]
    L.kdn_backward_workspace_bytes.restype = sz
    L.kdn_selftest_wait_timeout.argtypes = [vp, ctypes.c_longlong, vp]
    L.kdn_selftest_wait_timeout.restype = ctypes.c_int
    L.kdn_status_string.argtypes = [i]
    L.kdn_status_string.restype = ctypes.c_char_p
    L.kdn_last_error.argtypes = []
    L.kdn_last_error.restype = ctypes.c_char_p
    L.kdn_api_version.restype = ctypes.c_int
    L.kdn_plan.argtypes = [i, dims, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_char_p),
                           ctypes.POINTER(ctypes.c_char_p)]
    L.kdn_plan.restype = ctypes.c_int
    pages = ctypes.POINTER(PagesC)
    L.kdn_window_attn.argtypes = [dims, i, vp, vp, vp, vp, i, i, i, f, vp, vp, vp, sz, vp]
    L.kdn_window_attn_backward.argtypes = [dims, i, vp, vp, vp, vp, i, i, i, f] + [vp] * 7 + [sz, vp]
    L.kdn_window_workspace_bytes.argtypes = [dims, i, i, i, i]
    L.kdn_pages_reserve.argtypes = [pages, i, vp, vp, i, vp, sz, vp]
    L.kdn_pages_fork.argtypes = [pages, i, vp, vp, vp, vp, sz, vp]
    L.kdn_pages_free.argtypes = [pages, i, vp, vp, sz, vp]
    L.kdn_pages_compact.argtypes = [pages, vp, vp, sz, vp]
    L.kdn_pages_workspace_bytes.argtypes = [pages]
    L.kdn_pages_copy.argtypes = [i, vp, i, i, i, i, i, i, vp, vp, vp]
    L.kdn_pages_write.argtypes = [pages, i, vp, vp, i, i, i, i, i, vp, vp, vp, vp, vp]
    L.kdn_pages_write_reserved.argtypes = [pages, i, vp, vp, i, i, i, i, i, vp, vp, vp, vp, vp, sz, vp]
    L.kdn_paged_attn_step.argtypes = [pages, i, vp, i, i, i, i, i, i, vp, vp, vp, i, i, f, vp, vp, vp, sz, vp]
    L.kdn_paged_step_workspace_bytes.argtypes = [pages] + [i] * 8
    for name in ("kdn_window_workspace_bytes", "kdn_pages_workspace_bytes", "kdn_paged_step_workspace_bytes"):
        getattr(L, name).restype = sz
    for name in ("kdn_scan_delta", "kdn_scan_kalman_full", "kdn_scan_kalman_diag", "kdn_decode_step",
                 "kdn_read_device_status"):
        getattr(L, name).restype = ctypes.c_int
    _lib = L
    return L


def _check(status: int, what: str):
    if status != KDN_OK:
        msg = lib().kdn_last_error().decode()
        raise KdnError(status, f"{what}: {lib().kdn_status_string(status).decode()}: {msg}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t: torch.Tensor, name: str, shape, dtype=None, device=None):
    if isinstance(t, torch.Tensor) and t.is_cuda and t.shape == shape and (dtype is None or t.dtype == dtype) and \
            (device is None or t.device == device) and t.is_contiguous():
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (got {t.device})")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def workspace_bytes(variant: str, B: int, H: int, L: int, dk: int, dv: int, chunk: int = 0,
                    in_dtype=torch.bfloat16, out_dtype=None, segments: int = 0) -> int:
    d = Dims(B, H, L, dk, dv, chunk, _DTYPES[in_dtype], _DTYPES[out_dtype or torch.float32], segments)
    return int(lib().kdn_workspace_bytes(VARIANTS[variant], ctypes.byref(d)))


def plan(variant: str, B: int, H: int, L: int, dk: int, dv: int, chunk: int = 0, in_dtype=torch.bfloat16,
         out_dtype=None, segments: int = 0) -> dict:
    """The library's own account of the kernels a scan with these sizes runs."""
    d = Dims(B, H, L, dk, dv, chunk, _DTYPES[in_dtype], _DTYPES[out_dtype or torch.float32], segments)
    n, name, arith = ctypes.c_int(0), ctypes.c_char_p(), ctypes.c_char_p()
    _check(lib().kdn_plan(VARIANTS[variant], ctypes.byref(d), ctypes.byref(n), ctypes.byref(name),
                          ctypes.byref(arith)), "kdn_plan")
    return {"launches": n.value, "kernel": name.value.decode(), "arith": arith.value.decode()}


def _scan_common(q, k, v, o, m, S, chunk, out_dtype, segments=0):
    if q.dim() != 4:
        raise ValueError("q must be [B, H, L, d_k]")
    B, H, L, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    if q.dtype not in _DTYPES:
        raise ValueError(f"unsupported input dtype {q.dtype}")
    _need(q, "q", (B, H, L, dk), q.dtype)
    _need(k, "k", (B, H, L, dk), q.dtype, dev)
    _need(v, "v", (B, H, L, dv), q.dtype, dev)
    out_dtype = out_dtype or torch.float32
    if o is None:
        o = torch.empty(B, H, L, dv, dtype=out_dtype, device=dev)
    _need(o, "o", (B, H, L, dv), out_dtype, dev)
    if m is None:
        m = torch.empty(B, H, L, dtype=torch.float32, device=dev)
    _need(m, "m", (B, H, L), torch.float32, dev)
    if S is None:
        S = torch.zeros(B, H, dk, dv, dtype=torch.float32, device=dev)
    _need(S, "S", (B, H, dk, dv), torch.float32, dev)
    dims = Dims(B, H, L, dk, dv, chunk, _DTYPES[q.dtype], _DTYPES[out_dtype], segments)
    return dims, o, m, S


def _workspace(variant, dims, workspace, dev):
    need = int(lib().kdn_workspace_bytes(VARIANTS[variant], ctypes.byref(dims)))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    if workspace.device.type != "cuda" or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 CUDA tensor")
    return workspace


def scan_delta(q, k, v, beta, a=None, S=None, o=None, m=None, workspace=None, chunk=0, out_dtype=None, segments=0,
               stream=None):
    """Gated delta rule scan.  Returns (o, m, S); S is updated in place when given."""
    dims, o, m, S = _scan_common(q, k, v, o, m, S, chunk, out_dtype, segments)
    tok = tuple(q.shape[:3])
    _need(beta, "beta", tok, torch.float32, q.device)
    if a is not None:
        _need(a, "a", tok, torch.float32, q.device)
    workspace = _workspace("delta", dims, workspace, q.device)
    st = lib().kdn_scan_delta(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(a), _ptr(S), _ptr(o),
                              _ptr(m), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "kdn_scan_delta")
    return o, m, S


def scan_delta_backward(q, k, v, beta, dO, a=None, S0=None, dm=None, dS_L=None, workspace=None, stream=None,
                        want_da=True):
    """Gradients of the gated delta rule scan for upstream dO (and dm, dS_L).  Returns a dict with dq, dk,
    dv, dbeta, da (None if not wanted) and dS0, all fp32."""
    if q.dim() != 4:
        raise ValueError("q must be [B, H, L, d_k]")
    B, H, L, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    if q.dtype not in _DTYPES:
        raise ValueError(f"unsupported input dtype {q.dtype}")
    _need(q, "q", (B, H, L, dk), q.dtype)
    _need(k, "k", (B, H, L, dk), q.dtype, dev)
    _need(v, "v", (B, H, L, dv), q.dtype, dev)
    tok = (B, H, L)
    _need(beta, "beta", tok, torch.float32, dev)
    _need(dO, "dO", (B, H, L, dv), torch.float32, dev)
    for name, t, shape in (("a", a, tok), ("dm", dm, tok), ("S0", S0, (B, H, dk, dv)), ("dS_L", dS_L, (B, H, dk, dv))):
        if t is not None:
            _need(t, name, shape, torch.float32, dev)
    out = {"dq": torch.empty(B, H, L, dk, device=dev), "dk": torch.empty(B, H, L, dk, device=dev),
           "dv": torch.empty(B, H, L, dv, device=dev), "dbeta": torch.empty(B, H, L, device=dev),
           "da": torch.empty(B, H, L, device=dev) if want_da else None,
           "dS0": torch.empty(B, H, dk, dv, device=dev)}
    dims = Dims(B, H, L, dk, dv, 0, _DTYPES[q.dtype], KDN_F32, 0)
    need = int(lib().kdn_backward_workspace_bytes(VARIANTS["delta"], ctypes.byref(dims)))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    st = lib().kdn_scan_delta_backward(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(a), _ptr(S0),
                                       _ptr(dO), _ptr(dm), _ptr(dS_L), _ptr(out["dq"]), _ptr(out["dk"]),
                                       _ptr(out["dv"]), _ptr(out["dbeta"]), _ptr(out["da"]), _ptr(out["dS0"]),
                                       _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "kdn_scan_delta_backward")
    return out


def scan_kalman_diag_backward(q, k, v, r, dO, a=None, qn=None, S0=None, p0=None, dm=None, dS_L=None, dp_L=None,
                              workspace=None, stream=None, want_da=True):
    """Gradients of the diagonal Kalman scan for upstream dO (and dm, dS_L, dp_L).  Returns a dict with dq, dk,
    dv, dr, da (None if not wanted), dqn (per token), dS0 and dp0, all fp32."""
    return _kalman_backward("kalman_diag", q, k, v, r, dO, a, qn, S0, p0, dm, dS_L, dp_L, workspace, stream, want_da)


def scan_kalman_iso_backward(q, k, v, r, dO, a=None, qn=None, S0=None, c0=None, dm=None, dS_L=None, dc_L=None,
                             workspace=None, stream=None, want_da=True):
    """Gradients of the isotropic Kalman scan for upstream dO (and dm, dS_L, dc_L).  Returns a dict with dq, dk,
    dv, dr, da (None if not wanted), dqn (per token), dS0 and dc0, all fp32."""
    return _kalman_backward("kalman_iso", q, k, v, r, dO, a, qn, S0, c0, dm, dS_L, dc_L, workspace, stream, want_da)


def scan_kalman_full_backward(q, k, v, r, dO, a=None, qn=None, S0=None, P0=None, dm=None, dS_L=None, dP_L=None,
                              workspace=None, stream=None, want_da=True):
    """Gradients of the full-covariance Kalman scan for upstream dO (and dm, dS_L, dP_L).  Returns a dict with dq,
    dk, dv, dr, da (None if not wanted), dqn (per token), dS0 and dP0 (the gradient for a symmetric P0), all fp32."""
    return _kalman_backward("kalman_full", q, k, v, r, dO, a, qn, S0, P0, dm, dS_L, dP_L, workspace, stream, want_da)


def _kalman_backward(variant, q, k, v, r, dO, a, qn, S0, u0, dm, dS_L, du_L, workspace, stream, want_da):
    """The uncertainty-side backward shared by the isotropic (u = c, one per head), diagonal (u = p, one per
    coordinate) and full (u = P, d_k x d_k per head) variants."""
    if q.dim() != 4:
        raise ValueError("q must be [B, H, L, d_k]")
    B, H, L, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    if q.dtype not in _DTYPES:
        raise ValueError(f"unsupported input dtype {q.dtype}")
    _need(q, "q", (B, H, L, dk), q.dtype)
    _need(k, "k", (B, H, L, dk), q.dtype, dev)
    _need(v, "v", (B, H, L, dv), q.dtype, dev)
    tok = (B, H, L)
    _need(r, "r", tok, torch.float32, dev)
    _need(dO, "dO", (B, H, L, dv), torch.float32, dev)
    ushape = {"kalman_iso": (B, H), "kalman_diag": (B, H, dk), "kalman_full": (B, H, dk, dk)}[variant]
    uname = {"kalman_iso": "c", "kalman_diag": "p", "kalman_full": "P"}[variant]
    for name, t, shape in (("a", a, tok), ("dm", dm, tok), ("S0", S0, (B, H, dk, dv)), ("dS_L", dS_L, (B, H, dk, dv)),
                           (uname + "0", u0, ushape), ("d" + uname + "_L", du_L, ushape)):
        if t is not None:
            _need(t, name, shape, torch.float32, dev)
    qn_t, qn_s = _qn_args(qn, tok, dev)
    out = {"dq": torch.empty(B, H, L, dk, device=dev), "dk": torch.empty(B, H, L, dk, device=dev),
           "dv": torch.empty(B, H, L, dv, device=dev), "dr": torch.empty(B, H, L, device=dev),
           "da": torch.empty(B, H, L, device=dev) if want_da else None, "dqn": torch.empty(B, H, L, device=dev),
           "dS0": torch.empty(B, H, dk, dv, device=dev), "d" + uname + "0": torch.empty(*ushape, device=dev)}
    dims = Dims(B, H, L, dk, dv, 0, _DTYPES[q.dtype], KDN_F32, 0)
    need = int(lib().kdn_backward_workspace_bytes(VARIANTS[variant], ctypes.byref(dims)))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    fn = {"kalman_iso": lib().kdn_scan_kalman_iso_backward, "kalman_diag": lib().kdn_scan_kalman_diag_backward,
          "kalman_full": lib().kdn_scan_kalman_full_backward}[variant]
    st = fn(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(r), _ptr(a), _ptr(qn_t), qn_s, _ptr(S0), _ptr(u0),
            _ptr(dO), _ptr(dm), _ptr(dS_L), _ptr(du_L), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]),
            _ptr(out["dr"]), _ptr(out["da"]), _ptr(out["dqn"]), _ptr(out["dS0"]), _ptr(out["d" + uname + "0"]),
            _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "kdn_scan_" + variant + "_backward")
    return out


def _qn_args(qn, tok, dev):
    if qn is None:
        return None, 0.0
    if isinstance(qn, (int, float)):
        return None, float(qn)
    _need(qn, "qn", tok, torch.float32, dev)
    return qn, 0.0


def scan_kalman_full(q, k, v, r, a=None, qn=None, S=None, P=None, o=None, m=None, workspace=None, chunk=0,
                     out_dtype=None, segments=0, stream=None):
    """Full-covariance Kalman scan.  Returns (o, m, S, P); S and P are updated in place when given."""
    dims, o, m, S = _scan_common(q, k, v, o, m, S, chunk, out_dtype, segments)
    B, H, L, dk = q.shape
    tok = (B, H, L)
    _need(r, "r", tok, torch.float32, q.device)
    if a is not None:
        _need(a, "a", tok, torch.float32, q.device)
    qn_t, qn_s = _qn_args(qn, tok, q.device)
    if P is None:
        P = torch.eye(dk, dtype=torch.float32, device=q.device).repeat(B, H, 1, 1)
    _need(P, "P", (B, H, dk, dk), torch.float32, q.device)
    workspace = _workspace("kalman_full", dims, workspace, q.device)
    st = lib().kdn_scan_kalman_full(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(r), _ptr(qn_t), qn_s,
                                    _ptr(S), _ptr(P), _ptr(o), _ptr(m), _ptr(workspace), workspace.numel(),
                                    _stream(stream))
    _check(st, "kdn_scan_kalman_full")
    return o, m, S, P


def scan_kalman_full_noalloc(q, k, v, r, a=None, qn=None, S=None, P=None, o=None, m=None, chunk=0,
                             out_dtype=None, segments=0, stream=None):
    """Full-Kalman scan without a workspace, for callers that cannot allocate one: the library uses a static
    device array (B*H*L*d_k <= 4,194,304; overlapping calls race on it).  Returns (o, m, S, P)."""
    dims, o, m, S = _scan_common(q, k, v, o, m, S, chunk, out_dtype, segments)
    B, H, L, dk = q.shape
    tok = (B, H, L)
    _need(r, "r", tok, torch.float32, q.device)
    if a is not None:
        _need(a, "a", tok, torch.float32, q.device)
    qn_t, qn_s = _qn_args(qn, tok, q.device)
    if P is None:
        P = torch.eye(dk, dtype=torch.float32, device=q.device).repeat(B, H, 1, 1)
    _need(P, "P", (B, H, dk, dk), torch.float32, q.device)
    st = lib().kdn_scan_kalman_full_noalloc(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(r),
                                            _ptr(qn_t), qn_s, _ptr(S), _ptr(P), _ptr(o), _ptr(m), _stream(stream))
    _check(st, "kdn_scan_kalman_full_noalloc")
    return o, m, S, P


def scan_kalman_diag(q, k, v, r, a=None, qn=None, S=None, p=None, o=None, m=None, workspace=None, chunk=0,
                     out_dtype=None, segments=0, stream=None):
    """Diagonal-covariance Kalman scan.  Returns (o, m, S, p); S and p are updated in place when given."""
    dims, o, m, S = _scan_common(q, k, v, o, m, S, chunk, out_dtype, segments)
    B, H, L, dk = q.shape
    tok = (B, H, L)
    _need(r, "r", tok, torch.float32, q.device)
    if a is not None:
        _need(a, "a", tok, torch.float32, q.device)
    qn_t, qn_s = _qn_args(qn, tok, q.device)
    if p is None:
        p = torch.ones(B, H, dk, dtype=torch.float32, device=q.device)
    _need(p, "p", (B, H, dk), torch.float32, q.device)
    workspace = _workspace("kalman_diag", dims, workspace, q.device)
    st = lib().kdn_scan_kalman_diag(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(r), _ptr(qn_t), qn_s,
                                    _ptr(S), _ptr(p), _ptr(o), _ptr(m), _ptr(workspace), workspace.numel(),
                                    _stream(stream))
    _check(st, "kdn_scan_kalman_diag")
    return o, m, S, p


def scan_kalman_iso(q, k, v, r, a=None, qn=None, S=None, c=None, o=None, m=None, workspace=None, chunk=0,
                    out_dtype=None, segments=0, stream=None):
    """Isotropic-covariance Kalman scan (one uncertainty scalar per head).  Returns (o, m, S, c); S and c
    are updated in place when given."""
    dims, o, m, S = _scan_common(q, k, v, o, m, S, chunk, out_dtype, segments)
    B, H, L, dk = q.shape
    tok = (B, H, L)
    _need(r, "r", tok, torch.float32, q.device)
    if a is not None:
        _need(a, "a", tok, torch.float32, q.device)
    qn_t, qn_s = _qn_args(qn, tok, q.device)
    if c is None:
        c = torch.ones(B, H, dtype=torch.float32, device=q.device)
    _need(c, "c", (B, H), torch.float32, q.device)
    workspace = _workspace("kalman_iso", dims, workspace, q.device)
    st = lib().kdn_scan_kalman_iso(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(r), _ptr(qn_t), qn_s,
                                   _ptr(S), _ptr(c), _ptr(o), _ptr(m), _ptr(workspace), workspace.numel(),
                                   _stream(stream))
    _check(st, "kdn_scan_kalman_iso")
    return o, m, S, c


def hola_cache_read(q, k, v, m, gamma_q, gamma_k, sink, w=64, block=64, o=None, cache=None, workspace=None,
                    stream=None):
    """Surprise-cache read: q, k [B,H,L,d_k], v [B,H,L,d_v] (bf16 or fp32), m [B,H,L], gamma_q/gamma_k [d_k],
    sink [H].  Returns (o_cache [B,H,L,d_v] fp32, cache [B,H,w] int32 token indices, ascending, -1 empty)."""
    if q.dim() != 4:
        raise ValueError("q must be [B, H, L, d_k]")
    B, H, L, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    _need(q, "q", (B, H, L, dk), q.dtype)
    _need(k, "k", (B, H, L, dk), q.dtype, dev)
    _need(v, "v", (B, H, L, dv), q.dtype, dev)
    _need(m, "m", (B, H, L), torch.float32, dev)
    _need(gamma_q, "gamma_q", (dk,), torch.float32, dev)
    _need(gamma_k, "gamma_k", (dk,), torch.float32, dev)
    _need(sink, "sink", (H,), torch.float32, dev)
    if o is None:
        o = torch.empty(B, H, L, dv, dtype=torch.float32, device=dev)
    _need(o, "o", (B, H, L, dv), torch.float32, dev)
    if cache is None:
        cache = torch.empty(B, H, w, dtype=torch.int32, device=dev)
    _need(cache, "cache", (B, H, w), torch.int32, dev)
    dims = Dims(B, H, L, dk, dv, block, _DTYPES[q.dtype], KDN_F32)
    if workspace is None:
        need = int(lib().kdn_hola_workspace_bytes(ctypes.byref(dims)))
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    st = lib().kdn_hola_cache_read(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(m), _ptr(gamma_q),
                                   _ptr(gamma_k), _ptr(sink), int(w), _ptr(o), _ptr(cache), _ptr(workspace),
                                   workspace.numel(), _stream(stream))
    _check(st, "kdn_hola_cache_read")
    return o, cache


def decode_step(variant, q, k, v, S, beta=None, a=None, r=None, qn=0.0, p=None, o=None, m=None, out_dtype=None,
                stream=None):
    """One token per head against a resident state.  q, k [B,H,d_k], v [B,H,d_v]; S (and p: the diagonal
    variances [B,H,d_k], or for "kalman_iso" the uncertainty scalar [B,H]) updated in place.  Returns (o, m)."""
    if q.dim() != 3:
        raise ValueError("q must be [B, H, d_k]")
    B, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    _need(q, "q", (B, H, dk), q.dtype)
    _need(k, "k", (B, H, dk), q.dtype, dev)
    _need(v, "v", (B, H, dv), q.dtype, dev)
    _need(S, "S", (B, H, dk, dv), torch.float32, dev)
    out_dtype = out_dtype or torch.float32
    if o is None:
        o = torch.empty(B, H, dv, dtype=out_dtype, device=dev)
    _need(o, "o", (B, H, dv), out_dtype, dev)
    if m is None:
        m = torch.empty(B, H, dtype=torch.float32, device=dev)
    _need(m, "m", (B, H), torch.float32, dev)
    for name, t in (("beta", beta), ("a", a), ("r", r)):
        if t is not None:
            _need(t, name, (B, H), torch.float32, dev)
    if p is not None:  # diagonal: p [B,H,d_k]; isotropic: the uncertainty scalar c [B,H]
        _need(p, "p", (B, H) if variant == "kalman_iso" else (B, H, dk), torch.float32, dev)
    st = lib().kdn_decode_step(VARIANTS[variant], B, H, dk, dv, _DTYPES[q.dtype], _DTYPES[out_dtype], _ptr(q), _ptr(k),
                               _ptr(v), _ptr(beta), _ptr(a), _ptr(r), float(qn), _ptr(S), _ptr(p), _ptr(o), _ptr(m),
                               _stream(stream))
    _check(st, "kdn_decode_step")
    return o, m


def read_device_status(workspace: torch.Tensor | None, stream=None) -> int:
    """Synchronise the stream and return the device status of a scan's workspace (a KDN_* code).
    ``workspace=None`` reads the status word of the no-alloc full-Kalman scan on the current device."""
    out = ctypes.c_int(-1)
    st = lib().kdn_read_device_status(_ptr(workspace), ctypes.byref(out), _stream(stream))
    _check(st, "kdn_read_device_status")
    return out.value


def selftest_wait_timeout(workspace: torch.Tensor | None, wait_cycles: int = 100_000, stream=None) -> None:
    """Run the bounded-wait failure path once on purpose (a wait on an mbarrier nothing arrives at, with
    nothing in flight): afterwards ``read_device_status(workspace)`` reports KDN_ERR_TIMEOUT."""
    st = lib().kdn_selftest_wait_timeout(_ptr(workspace), int(wait_cycles), _stream(stream))
    _check(st, "kdn_selftest_wait_timeout")


# ---------------------------------------------------------------------------------- windowed attention

_SAME = contextlib.nullcontext()


def _on(stream):
    """Allocations of a call belong to the stream it runs on."""
    return _SAME if stream is None else torch.cuda.stream(stream)


# the current stream's handle without building a Stream object, where torch offers it (2 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(stream, dev):
    if stream is None:
        return torch.cuda.current_stream(dev).cuda_stream if _raw_stream is None else _raw_stream(dev.index)
    if stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
    return stream.cuda_stream


def _int32(x, name):
    if not -2**31 <= x < 2**31:
        raise ValueError(f"{name} = {x} does not fit 32 bits")
    return x


def _at(t):
    return None if t is None else t.data_ptr()


def _scratch(workspace, need, dev):
    if workspace is None:
        return torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    if workspace.device != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {dev}")
    return workspace


def _window_args(q, k, v, lens, scale, window, n_sink):
    _int32(window, "window"), _int32(n_sink, "n_sink")
    try:
        B, H, L, dk = q.shape
        _, Hkv, _, dv = v.shape
    except ValueError:
        raise ValueError("q must be [B, H, L, d_k], k [B, kv_heads, L, d_k] and v [B, kv_heads, L, d_v]") from None
    dtype, dev = q.dtype, q.device
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported input dtype {dtype}")
    _need(q, "q", (B, H, L, dk), dtype)
    _need(k, "k", (B, Hkv, L, dk), dtype, dev)
    _need(v, "v", (B, Hkv, L, dv), dtype, dev)
    if lens is not None:
        _need(lens, "lens", (B,), torch.int32, dev)
    return B, H, Hkv, L, dk, dv, dev, dk ** -0.5 if scale is None else float(scale)


def window_workspace_bytes(B, H, Hkv, L, dk, dv, window, n_sink=0, in_dtype=torch.bfloat16, out_dtype=None, backward=False):
    d = Dims(B, H, L, dk, dv, 0, _DTYPES[in_dtype], _DTYPES[out_dtype or in_dtype], 0)
    return int(lib().kdn_window_workspace_bytes(ctypes.byref(d), Hkv, window, n_sink, int(backward)))


def window_attn(q, k, v, window, n_sink=0, lens=None, scale=None, o=None, lse=None, workspace=None, out_dtype=None,
                stream=None):
    """Causal softmax attention in which token t sees the tokens j <= t with j > t - window or j < n_sink.

    q [B,H,L,d_k], k [B,kv_heads,L,d_k], v [B,kv_heads,L,d_v] (bf16 or fp32); query head h reads k/v head
    h // (H / kv_heads).  lens [B] int32 (or None): tokens of each sequence; rows behind them are left as they were
    in the given o and lse, and are zero in those allocated here.  scale defaults to 1 / sqrt(d_k), out_dtype to q's.
    Returns (o [B,H,L,d_v], lse [B,H,L] fp32)."""
    B, H, Hkv, L, dk, dv, dev, scale = _window_args(q, k, v, lens, scale, window, n_sink)
    out_dtype = out_dtype or (q.dtype if o is None else o.dtype)
    if out_dtype not in _DTYPES:
        raise ValueError(f"unsupported output dtype {out_dtype}")
    dims = Dims(B, H, L, dk, dv, 0, _DTYPES[q.dtype], _DTYPES[out_dtype], 0)
    if o is not None:
        _need(o, "o", (B, H, L, dv), out_dtype, dev)
    if lse is not None:
        _need(lse, "lse", (B, H, L), torch.float32, dev)
    fresh = o is None and lse is None
    if o is None or lse is None:
        # rows behind the sequences: the kernels zero them where both arrays are new, a fill does where one is
        new = torch.empty if lens is None or fresh else torch.zeros
        with _on(stream):
            if o is None:
                o = torch.empty_like(q) if new is torch.empty and dv == dk and out_dtype == q.dtype else \
                    new((B, H, L, dv), dtype=out_dtype, device=dev)
            if lse is None:
                lse = new((B, H, L), dtype=torch.float32, device=dev)
    if workspace is not None:
        _scratch(workspace, 256, dev)
    st = lib().kdn_window_attn(dims, Hkv, q.data_ptr(), k.data_ptr(), v.data_ptr(), _at(lens), fresh, window, n_sink, scale,
                               o.data_ptr(), lse.data_ptr(), _at(workspace),
                               0 if workspace is None else workspace.numel(), _stream_of(stream, dev))
    if st:
        _check(st, "kdn_window_attn")
    return o, lse


def window_attn_backward(q, k, v, o, lse, dO, window, n_sink=0, lens=None, scale=None, dq=None, dk=None, dv=None,
                         workspace=None, stream=None):
    """Gradients of window_attn for upstream dO (of o's type), from its inputs and its o and lse.  Returns a dict with
    dq, dk, dv in q's type (dk and dv summed over the heads that share them); rows behind a sequence's last token are
    left as they were in given tensors, and are zero in those allocated here."""
    B, H, Hkv, L, d_k, d_v, dev, scale = _window_args(q, k, v, lens, scale, window, n_sink)
    dtype = q.dtype
    if o.dtype not in _DTYPES:
        raise ValueError(f"unsupported output dtype {o.dtype}")
    _need(o, "o", (B, H, L, d_v), o.dtype, dev)
    _need(lse, "lse", (B, H, L), torch.float32, dev)
    _need(dO, "dO", (B, H, L, d_v), o.dtype, dev)
    dims = Dims(B, H, L, d_k, d_v, 0, _DTYPES[dtype], _DTYPES[o.dtype], 0)
    fresh = dq is None and dk is None and dv is None
    new = torch.empty_like if lens is None or fresh else torch.zeros_like
    with _on(stream):
        dq = new(q) if dq is None else _need(dq, "dq", (B, H, L, d_k), dtype, dev)
        dk = new(k) if dk is None else _need(dk, "dk", (B, Hkv, L, d_k), dtype, dev)
        dv = new(v) if dv is None else _need(dv, "dv", (B, Hkv, L, d_v), dtype, dev)
        if workspace is None:
            workspace = _scratch(None, lib().kdn_window_workspace_bytes(dims, Hkv, window, n_sink, 1), dev)
        else:
            _scratch(workspace, 256, dev)
    st = lib().kdn_window_attn_backward(dims, Hkv, q.data_ptr(), k.data_ptr(), v.data_ptr(), _at(lens), fresh, window, n_sink,
                                        scale, o.data_ptr(), lse.data_ptr(), dO.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                        dv.data_ptr(), workspace.data_ptr(), workspace.numel(), _stream_of(stream, dev))
    if st:
        _check(st, "kdn_window_attn_backward")
    return {"dq": dq, "dk": dk, "dv": dv}


# ---------------------------------------------------------------------------------- paged key-value cache

@dataclass
class Pages:
    """The books of a paged cache (kdn_pages): table [rows, max_pages], lens [rows] and refs [num_pages], int32.  One
    set serves every layer; a layer's pages are k_pages [num_pages, kv_heads, page_size, d_k] and v_pages.
    ``workspace`` (allocated with the books; one given here is set to zero) has the status of the last book-keeping call,
    read_device_status(pages.workspace), and which rows' last reservation was refused."""
    table: torch.Tensor
    lens: torch.Tensor
    refs: torch.Tensor
    page_size: int
    workspace: torch.Tensor | None = None

    def __post_init__(self):
        self._own = self._home = None
        self._fresh = True  # no call has come since the workspace was set to zero, on the stream _home
        if self.workspace is not None:
            if self.workspace.is_cuda:
                self.workspace.zero_()
                self._home = _stream_of(None, self.workspace.device)
        elif self.table.is_cuda:
            self._allocate(self._c())

    def _allocate(self, c):
        dev = self.table.device
        self.workspace = torch.zeros(max(256, lib().kdn_pages_workspace_bytes(c)), dtype=torch.uint8, device=dev)
        self._own, self._home, self._fresh = (c.num_pages, c.rows), _stream_of(None, dev), True

    def _visit(self, stream, dev):
        """A call on another stream than the workspace's own: the first one follows the zeros, and the memory stays the
        workspace's until the call has ended.  (A capture begins behind all work.)"""
        stream = torch.cuda.current_stream(dev) if stream is None else stream
        with torch.cuda.stream(stream):
            if self._fresh and self._home is not None and not torch.cuda.is_current_stream_capturing():
                home = torch.cuda.ExternalStream(self._home, device=dev) if self._home else torch.cuda.default_stream(dev)
                stream.wait_stream(home)
        if self.workspace.is_cuda:
            self.workspace.record_stream(stream)

    def _c(self, dev=None):
        table, lens, refs = self.table, self.lens, self.refs
        try:
            rows, most = table.shape
        except ValueError:
            raise ValueError("table must be [rows, max_pages]") from None
        _need(table, "table", (rows, most), torch.int32, dev)
        dev = table.device
        _need(lens, "lens", (rows,), torch.int32, dev)
        _need(refs, "refs", (refs.numel(),), torch.int32, dev)
        return PagesC(refs.numel(), self.page_size, rows, most, table.data_ptr(), lens.data_ptr(), refs.data_ptr())


def make_pages(num_pages, page_size, rows, max_pages, device="cuda") -> Pages:
    """The books of an empty cache."""
    full = lambda shape, x: torch.full(shape, x, dtype=torch.int32, device=device)  # noqa: E731
    return Pages(full((rows, max_pages), -1), full((rows,), 0), full((num_pages,), 0), page_size)


def _list(t, name, dev):
    if not isinstance(t, torch.Tensor) or t.dim() != 1:
        raise ValueError(f"{name} must be a 1-D int32 tensor")
    return _need(t, name, t.shape, torch.int32, dev)


def _books(pages, stream):
    c = pages._c()
    dev = pages.table.device
    if pages._own not in (None, (c.num_pages, c.rows)):  # the books were exchanged for larger or smaller ones
        with _on(stream):
            pages._allocate(c)
    st = _stream_of(stream, dev)
    if st != pages._home:
        pages._visit(stream, dev)
    pages._fresh = False
    return c, dev, pages.workspace, st


def pages_reserve(pages, rows, counts, stream=None):
    """Adds tokens to the listed rows (int32 [n]), with the pages they need: ``counts`` each, or counts[i] (int32 [n]).
    Refused as a whole where there is no room: read_device_status(pages.workspace) says so (it waits for the stream), and
    pages_write passes over the rows until a reservation succeeds."""
    c, dev, ws, at = _books(pages, stream)
    _list(rows, "rows", dev)
    each = isinstance(counts, torch.Tensor)
    if each:
        _need(counts, "counts", rows.shape, torch.int32, dev)
    else:
        _int32(counts, "counts")
    st = lib().kdn_pages_reserve(c, rows.numel(), _at(rows), _at(counts) if each else None,
                                 0 if each else counts, _at(ws), ws.numel(), at)
    if st:
        _check(st, "kdn_pages_reserve")


def pages_fork(pages, src_rows, dst_rows, moves=None, stream=None):
    """Makes each empty row dst_rows[i] a copy of src_rows[i], sharing its full pages.  Returns moves [n, 2] int32, the
    part-filled pages that pages_copy has to copy (in every layer) before the rows are used."""
    c, dev, ws, at = _books(pages, stream)
    _list(src_rows, "src_rows", dev)
    _need(dst_rows, "dst_rows", src_rows.shape, torch.int32, dev)
    with _on(stream):
        if moves is None:
            moves = torch.empty(src_rows.numel(), 2, dtype=torch.int32, device=dev)
    _need(moves, "moves", (src_rows.numel(), 2), torch.int32, dev)
    st = lib().kdn_pages_fork(c, src_rows.numel(), _at(src_rows), _at(dst_rows), _at(moves), _at(ws),
                              ws.numel(), at)
    if st:
        _check(st, "kdn_pages_fork")
    return moves


def pages_free(pages, rows, stream=None):
    """Empties the listed rows; pages that no row names any more are free."""
    c, dev, ws, at = _books(pages, stream)
    _list(rows, "rows", dev)
    st = lib().kdn_pages_free(c, rows.numel(), _at(rows), _at(ws), ws.numel(), at)
    if st:
        _check(st, "kdn_pages_free")


def pages_compact(pages, moves=None, stream=None):
    """Moves the pages in use to the lowest page numbers.  Returns moves [num_pages // 2, 2] int32 for pages_copy (in
    every layer), ending in pairs of -1."""
    c, dev, ws, at = _books(pages, stream)
    with _on(stream):
        if moves is None:
            moves = torch.empty(c.num_pages // 2, 2, dtype=torch.int32, device=dev)
    _need(moves, "moves", (c.num_pages // 2, 2), torch.int32, dev)
    st = lib().kdn_pages_compact(c, _at(moves), _at(ws), ws.numel(), at)
    if st:
        _check(st, "kdn_pages_compact")
    return moves


def _pool(k_pages, v_pages, dev=None):
    try:
        num, Hkv, page, dk = k_pages.shape
        _, _, _, dv = v_pages.shape
    except ValueError:
        raise ValueError("k_pages must be [num_pages, kv_heads, page_size, d_k] and v_pages "
                         "[num_pages, kv_heads, page_size, d_v]") from None
    if k_pages.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {k_pages.dtype} of k_pages")
    _need(k_pages, "k_pages", (num, Hkv, page, dk), k_pages.dtype, dev)
    _need(v_pages, "v_pages", (num, Hkv, page, dv), k_pages.dtype, k_pages.device)
    return num, Hkv, page, dk, dv


def pages_copy(moves, k_pages, v_pages, stream=None):
    """Copies page moves[i, 0] to page moves[i, 1] for every pair (pairs with a number out of range are skipped)."""
    num, Hkv, page, dk, dv = _pool(k_pages, v_pages)
    dev = k_pages.device
    _need(moves, "moves", (moves.shape[0], 2), torch.int32, dev)
    st = lib().kdn_pages_copy(moves.shape[0], _at(moves), num, page, Hkv, dk, dv, _DTYPES[k_pages.dtype], _at(k_pages),
                              _at(v_pages), _stream_of(stream, dev))
    if st:
        _check(st, "kdn_pages_copy")


def pages_write(pages, rows, k_new, v_new, k_pages, v_pages, counts=None, stream=None):
    """Writes the newest tokens of the listed rows (added by pages_reserve) into one layer's pages: k_new
    [n, kv_heads, tokens, d_k] and v_new; of entry i the first counts[i] (or all) are the row's last counts[i].  Rows whose
    last reservation was refused are left as they are."""
    dev = pages.table.device
    num, Hkv, page, dk, dv = _pool(k_pages, v_pages, dev)
    c, _, ws, at = _books(pages, stream)
    if num != c.num_pages or page != pages.page_size:
        raise ValueError(f"k_pages holds {num} pages of {page} tokens, the books {c.num_pages} of {pages.page_size}")
    _list(rows, "rows", dev)
    n = rows.numel()
    if k_new.dim() != 4:
        raise ValueError("k_new must be [n, kv_heads, tokens, d_k]")
    T = k_new.shape[2]
    _need(k_new, "k_new", (n, Hkv, T, dk), k_pages.dtype, dev)
    _need(v_new, "v_new", (n, Hkv, T, dv), k_pages.dtype, dev)
    if counts is not None:
        _need(counts, "counts", (n,), torch.int32, dev)
    st = lib().kdn_pages_write_reserved(c, n, _at(rows), _at(counts), T, Hkv, dk, dv, _DTYPES[k_pages.dtype], _at(k_new),
                                        _at(v_new), _at(k_pages), _at(v_pages), _at(ws), ws.numel(), at)
    if st:
        _check(st, "kdn_pages_write_reserved")


def paged_attn_step(q, k_pages, v_pages, table, lens, rows=None, window=0, n_sink=0, scale=None, o=None, lse=None,
                    workspace=None, out_dtype=None, stream=None):
    """One new token per sequence against its paged cache, which already holds it (pages_write): q [n,H,d_k], sequence i
    being row rows[i] (int32 [n]; None: i) of table [rows, max_pages] and lens [rows].  window = 0 sees the whole
    cache; otherwise visibility is window_attn's.  Returns (o [n,H,d_v], lse [n,H] fp32); an empty row gives 0 and
    -inf, a broken table entry NaN."""
    num, Hkv, page, dk, dv = _pool(k_pages, v_pages)
    dev = k_pages.device
    _int32(window, "window"), _int32(n_sink, "n_sink")
    if q.dim() != 3:
        raise ValueError("q must be [n, H, d_k]")
    n, H = q.shape[:2]
    _need(q, "q", (n, H, dk), k_pages.dtype, dev)
    if table.dim() != 2:
        raise ValueError("table must be [rows, max_pages]")
    _need(table, "table", tuple(table.shape), torch.int32, dev)
    _need(lens, "lens", (table.shape[0],), torch.int32, dev)
    if rows is not None:
        _need(rows, "rows", (n,), torch.int32, dev)
    out_dtype = out_dtype or (q.dtype if o is None else o.dtype)
    if out_dtype not in _DTYPES:
        raise ValueError(f"unsupported output dtype {out_dtype}")
    if o is not None:
        _need(o, "o", (n, H, dv), out_dtype, dev)
    if lse is not None:
        _need(lse, "lse", (n, H), torch.float32, dev)
    c = PagesC(num, page, table.shape[0], table.shape[1], table.data_ptr(), lens.data_ptr(), None)
    with _on(stream):
        if o is None:
            o = torch.empty_like(q) if dv == dk and out_dtype == q.dtype else \
                torch.empty((n, H, dv), dtype=out_dtype, device=dev)
        if lse is None:
            lse = torch.empty((n, H), dtype=torch.float32, device=dev)
        need = lib().kdn_paged_step_workspace_bytes(c, n, H, Hkv, dk, dv, _DTYPES[q.dtype], window, n_sink)
        if workspace is not None or need > 256:
            workspace = _scratch(workspace, need, dev)
    scale = float(dk ** -0.5 if scale is None else scale)
    st = lib().kdn_paged_attn_step(c, n, _at(rows), H, Hkv, dk, dv, _DTYPES[q.dtype], _DTYPES[out_dtype],
                                   _at(q), _at(k_pages), _at(v_pages), window, n_sink, scale, _at(o), _at(lse),
                                   _at(workspace), 0 if workspace is None else workspace.numel(), _stream_of(stream, dev))
    if st:
        _check(st, "kdn_paged_attn_step")
    return o, lse
