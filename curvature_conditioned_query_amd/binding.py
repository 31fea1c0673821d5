"""ctypes binding of ``libccq.so`` (the C ABI in ``include/ccq.h``).

Argument marshalling only: torch tensors are checked for device, dtype and
contiguity and handed to the library as raw device pointers together with the
caller's current HIP stream.  No step of the method runs here, and there is no
fallback: if the library is missing, every call raises.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional

CCQ_RULE_GLA = 0
CCQ_RULE_GDN = 1
CCQ_DTYPE_F32 = 0
CCQ_DTYPE_BF16 = 1

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None

# Every symbol include/ccq.h declares (kept in one place for the export test).
EXPORTED_SYMBOLS = (
    "ccq_fwd_chunked",
    "ccq_fwd_chunked_noalloc",
    "ccq_fwd_workspace_bytes",
    "ccq_decode_step",
    "ccq_key_subspace",
    "ccq_step_backward",
    "ccq_bwd_chunked",
    "ccq_bwd_workspace_bytes",
    "ccq_chunk_carry_bytes",
    "ccq_qk_norm_rope",
    "ccq_qk_norm_rope_backward",
    "ccq_qk_backward_workspace_bytes",
    "ccq_scan",
    "ccq_scan_workspace_bytes",
    "ccq_scan_backward",
    "ccq_scan_backward_workspace_bytes",
    "ccq_beam_select",
    "ccq_beam_select_workspace_bytes",
    "ccq_beam_reorder",
    "ccq_status_string",
    "ccq_abi_version",
)


class CcqError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: status {status} ({_status_string(status)})")


class FwdParams(ctypes.Structure):
    """Mirror of ``ccq_fwd_params``."""

    _fields_ = [
        ("rule", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("T", ctypes.c_int32),
        ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32),
        ("chunk", ctypes.c_int32), ("segments", ctypes.c_int32),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("log_alpha", ctypes.c_void_p), ("beta", ctypes.c_void_p),
        ("w_lambda", ctypes.c_void_p), ("b_lambda", ctypes.c_void_p),
        ("S0", ctypes.c_void_p), ("C0", ctypes.c_void_p), ("ksum0", ctypes.c_void_p),
        ("n0", ctypes.c_void_p),
        ("o", ctypes.c_void_p),
        ("S_out", ctypes.c_void_p), ("C_out", ctypes.c_void_p), ("ksum_out", ctypes.c_void_p),
        ("n_out", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("phase_events", ctypes.c_void_p),
        ("flags", ctypes.c_int32),
        ("chunk_carry", ctypes.c_void_p),
    ]


class BwdParams(ctypes.Structure):
    """Mirror of ``ccq_bwd_params``."""

    _fields_ = [
        ("rule", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("T", ctypes.c_int32),
        ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32), ("chunk", ctypes.c_int32),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("log_alpha", ctypes.c_void_p),
        ("w_lambda", ctypes.c_void_p), ("b_lambda", ctypes.c_void_p),
        ("S0", ctypes.c_void_p), ("C0", ctypes.c_void_p), ("ksum0", ctypes.c_void_p), ("n0", ctypes.c_void_p),
        ("d_o", ctypes.c_void_p),
        ("dS_T", ctypes.c_void_p), ("dC_T", ctypes.c_void_p), ("dksum_T", ctypes.c_void_p),
        ("dq", ctypes.c_void_p), ("dk", ctypes.c_void_p), ("dv", ctypes.c_void_p), ("dlog_alpha", ctypes.c_void_p),
        ("dw_lambda", ctypes.c_void_p), ("db_lambda", ctypes.c_void_p),
        ("dS0", ctypes.c_void_p), ("dC0", ctypes.c_void_p), ("dksum0", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("phase_events", ctypes.c_void_p),
        ("flags", ctypes.c_int32),
        ("beta", ctypes.c_void_p), ("dbeta", ctypes.c_void_p),
        ("chunk_carry", ctypes.c_void_p),
    ]


class QkParams(ctypes.Structure):
    """Mirror of ``ccq_qk_params``."""

    _fields_ = [
        ("dtype", ctypes.c_int32), ("B", ctypes.c_int32), ("T", ctypes.c_int32),
        ("H_q", ctypes.c_int32), ("H_k", ctypes.c_int32), ("d", ctypes.c_int32),
        ("q_norm", ctypes.c_int32), ("k_norm", ctypes.c_int32), ("rot", ctypes.c_int32),
        ("interleaved", ctypes.c_int32), ("expand_keys", ctypes.c_int32), ("eps", ctypes.c_float),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
        ("q_stride_b", ctypes.c_int64), ("q_stride_t", ctypes.c_int64), ("q_stride_h", ctypes.c_int64),
        ("k_stride_b", ctypes.c_int64), ("k_stride_t", ctypes.c_int64), ("k_stride_h", ctypes.c_int64),
        ("positions", ctypes.c_void_p), ("position0", ctypes.c_int64), ("inv_freq", ctypes.c_void_p),
        ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
        ("q_out", ctypes.c_void_p), ("k_out", ctypes.c_void_p),
    ]


class QkBwdParams(ctypes.Structure):
    """Mirror of ``ccq_qk_bwd_params``."""

    _fields_ = [
        ("fwd", QkParams),
        ("dq_out", ctypes.c_void_p), ("dk_out", ctypes.c_void_p), ("dq", ctypes.c_void_p), ("dk", ctypes.c_void_p),
        ("dq_stride_b", ctypes.c_int64), ("dq_stride_t", ctypes.c_int64), ("dq_stride_h", ctypes.c_int64),
        ("dk_stride_b", ctypes.c_int64), ("dk_stride_t", ctypes.c_int64), ("dk_stride_h", ctypes.c_int64),
        ("dq_weight", ctypes.c_void_p), ("dk_weight", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


class ScanParams(ctypes.Structure):
    """Mirror of ``ccq_scan_params``."""

    _fields_ = [
        ("dtype", ctypes.c_int32), ("B", ctypes.c_int32), ("T", ctypes.c_int32), ("D", ctypes.c_int32),
        ("complement", ctypes.c_int32),
        ("x", ctypes.c_void_p), ("log_alpha", ctypes.c_void_p),
        ("x_stride_b", ctypes.c_int64), ("x_stride_t", ctypes.c_int64),
        ("la_stride_b", ctypes.c_int64), ("la_stride_t", ctypes.c_int64),
        ("lengths", ctypes.c_void_p), ("h0", ctypes.c_void_p), ("y", ctypes.c_void_p), ("h_out", ctypes.c_void_p),
        ("chunk_carry", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


class ScanBwdParams(ctypes.Structure):
    """Mirror of ``ccq_scan_bwd_params``."""

    _fields_ = [
        ("dtype", ctypes.c_int32), ("B", ctypes.c_int32), ("T", ctypes.c_int32), ("D", ctypes.c_int32),
        ("complement", ctypes.c_int32),
        ("x", ctypes.c_void_p), ("log_alpha", ctypes.c_void_p), ("dy", ctypes.c_void_p),
        ("x_stride_b", ctypes.c_int64), ("x_stride_t", ctypes.c_int64),
        ("la_stride_b", ctypes.c_int64), ("la_stride_t", ctypes.c_int64),
        ("dy_stride_b", ctypes.c_int64), ("dy_stride_t", ctypes.c_int64),
        ("lengths", ctypes.c_void_p), ("h0", ctypes.c_void_p), ("dh_out", ctypes.c_void_p),
        ("chunk_carry", ctypes.c_void_p), ("dx", ctypes.c_void_p), ("dlog_alpha", ctypes.c_void_p),
        ("dh0", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


class BeamParams(ctypes.Structure):
    """Mirror of ``ccq_beam_params``."""

    _fields_ = [
        ("dtype", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("V", ctypes.c_int32),
        ("M", ctypes.c_int32),
        ("logits", ctypes.c_void_p), ("logits_stride", ctypes.c_int64), ("scores", ctypes.c_void_p),
        ("finished", ctypes.c_void_p), ("pad_token", ctypes.c_int32), ("token", ctypes.c_void_p),
        ("parent", ctypes.c_void_p), ("score", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


def library_path() -> str:
    return os.environ.get("CCQ_LIBRARY", os.path.join(_HERE, "libccq.so"))


def load_library():
    """Load libccq.so (once).  Raises if it has not been built."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with `python -m curvature_conditioned_query_amd.build` "
            "(there is no fallback implementation)")
    lib = ctypes.CDLL(path)
    vp = ctypes.c_void_p
    i32 = ctypes.c_int32
    lib.ccq_fwd_chunked.argtypes = [ctypes.POINTER(FwdParams), vp]
    lib.ccq_fwd_chunked.restype = ctypes.c_int
    lib.ccq_fwd_chunked_noalloc.argtypes = [ctypes.POINTER(FwdParams), vp]
    lib.ccq_fwd_chunked_noalloc.restype = ctypes.c_int
    lib.ccq_fwd_workspace_bytes.argtypes = [ctypes.POINTER(FwdParams)]
    lib.ccq_fwd_workspace_bytes.restype = ctypes.c_size_t
    lib.ccq_decode_step.argtypes = [i32, i32, i32, i32, i32, i32] + [vp] * 12 + [i32, vp]
    lib.ccq_decode_step.restype = ctypes.c_int
    lib.ccq_key_subspace.argtypes = [i32] * 6 + [vp] * 10 + [i32, vp]
    lib.ccq_key_subspace.restype = ctypes.c_int
    lib.ccq_step_backward.argtypes = [i32] * 6 + [vp] * 22 + [i32, vp]
    lib.ccq_step_backward.restype = ctypes.c_int
    lib.ccq_bwd_chunked.argtypes = [ctypes.POINTER(BwdParams), vp]
    lib.ccq_bwd_chunked.restype = ctypes.c_int
    lib.ccq_bwd_workspace_bytes.argtypes = [ctypes.POINTER(BwdParams)]
    lib.ccq_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.ccq_chunk_carry_bytes.argtypes = [i32] * 5
    lib.ccq_chunk_carry_bytes.restype = ctypes.c_size_t
    for name, cls in (("ccq_qk_norm_rope", QkParams), ("ccq_qk_norm_rope_backward", QkBwdParams),
                      ("ccq_scan", ScanParams), ("ccq_scan_backward", ScanBwdParams),
                      ("ccq_beam_select", BeamParams)):
        getattr(lib, name).argtypes = [ctypes.POINTER(cls), vp]
        getattr(lib, name).restype = ctypes.c_int
    for name, cls in (("ccq_qk_backward_workspace_bytes", QkBwdParams), ("ccq_scan_workspace_bytes", ScanParams),
                      ("ccq_scan_backward_workspace_bytes", ScanBwdParams),
                      ("ccq_beam_select_workspace_bytes", BeamParams)):
        getattr(lib, name).argtypes = [ctypes.POINTER(cls)]
        getattr(lib, name).restype = ctypes.c_size_t
    lib.ccq_beam_reorder.argtypes = [i32, ctypes.POINTER(vp), ctypes.POINTER(ctypes.c_size_t), i32, i32, vp, vp]
    lib.ccq_beam_reorder.restype = ctypes.c_int
    lib.ccq_status_string.argtypes = [i32]
    lib.ccq_status_string.restype = ctypes.c_char_p
    lib.ccq_abi_version.argtypes = []
    lib.ccq_abi_version.restype = i32
    _LIB = lib
    return lib


def _status_string(status: int) -> str:
    try:
        return load_library().ccq_status_string(status).decode()
    except Exception:  # pragma: no cover - only used for messages
        return "?"


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return CCQ_DTYPE_F32
    if t.dtype == torch.bfloat16:
        return CCQ_DTYPE_BF16
    raise TypeError(f"unsupported tensor dtype {t.dtype}")


def _stream_handle(stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _check_dev(name, t, dtype=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _rule_code(rule) -> int:
    if rule in ("gla", CCQ_RULE_GLA):
        return CCQ_RULE_GLA
    if rule in ("gdn", CCQ_RULE_GDN):
        return CCQ_RULE_GDN
    raise ValueError(f"unknown rule {rule!r}")


FLAG_NORMALIZE_KEYS = 1  # CCQ_FLAG_NORMALIZE_KEYS
FLAG_PACKED_COV = 2  # CCQ_FLAG_PACKED_COV


def _flags(normalize_keys: bool, packed_cov: bool) -> int:
    return (FLAG_NORMALIZE_KEYS if normalize_keys else 0) | (FLAG_PACKED_COV if packed_cov else 0)


def _check_numel(name, t, n):
    if t is not None and t.numel() != n:
        raise ValueError(f"{name} must hold {n} elements, got {t.numel()}")


def cov_numel(d_k: int, packed_cov: bool) -> int:
    """Floats per head of the second-moment state: d_k^2, or d_k (d_k + 1) / 2 packed."""
    return d_k * (d_k + 1) // 2 if packed_cov else d_k * d_k


def make_fwd_params(rule, q, k, v, log_alpha, beta, w_lambda, b_lambda, o,
                    carry_in=None, carry_out=None, segments: int = 0, chunk: int = 64,
                    workspace=None, normalize_keys: bool = False, packed_cov: bool = False) -> FwdParams:
    """Fill a ccq_fwd_params from tensors (carry_in / carry_out: (S, C, ksum, n) or None; C is
    [B, H, d_k, d_k], or its packed upper triangle [B, H, d_k (d_k + 1) / 2] with packed_cov)."""
    import torch
    B, H, T, d_k = q.shape
    d_v = v.shape[-1]
    p = FwdParams()
    p.rule = _rule_code(rule)
    p.dtype = _dtype_code(q)
    p.B, p.H, p.T, p.d_k, p.d_v = B, H, T, d_k, d_v
    p.chunk = chunk
    p.segments = segments
    p.flags = _flags(normalize_keys, packed_cov)
    for name, t in (("q", q), ("k", k), ("v", v), ("log_alpha", log_alpha), ("beta", beta), ("o", o)):
        _check_dev(name, t, q.dtype)
    _check_dev("w_lambda", w_lambda, torch.float32)
    _check_dev("b_lambda", b_lambda, torch.float32)
    p.q, p.k, p.v, p.log_alpha, p.beta = (_ptr(x) for x in (q, k, v, log_alpha, beta))
    p.w_lambda, p.b_lambda, p.o = _ptr(w_lambda), _ptr(b_lambda), _ptr(o)
    if carry_in is not None:
        S0, C0, m0, n0 = carry_in
        for name, t, dt in (("S0", S0, torch.float32), ("C0", C0, torch.float32),
                            ("ksum0", m0, torch.float32), ("n0", n0, torch.int64)):
            _check_dev(name, t, dt)
        _check_numel("S0", S0, B * H * d_v * d_k)
        _check_numel("C0", C0, B * H * cov_numel(d_k, packed_cov))
        _check_numel("ksum0", m0, B * H * d_k)
        _check_numel("n0", n0, B * H)
        p.S0, p.C0, p.ksum0, p.n0 = _ptr(S0), _ptr(C0), _ptr(m0), _ptr(n0)
    if carry_out is not None:
        S1, C1, m1, n1 = carry_out
        for name, t, dt in (("S_out", S1, torch.float32), ("C_out", C1, torch.float32),
                            ("ksum_out", m1, torch.float32), ("n_out", n1, torch.int64)):
            _check_dev(name, t, dt)
        _check_numel("S_out", S1, B * H * d_v * d_k)
        _check_numel("C_out", C1, B * H * cov_numel(d_k, packed_cov))
        _check_numel("ksum_out", m1, B * H * d_k)
        _check_numel("n_out", n1, B * H)
        p.S_out, p.C_out, p.ksum_out, p.n_out = _ptr(S1), _ptr(C1), _ptr(m1), _ptr(n1)
    if workspace is not None:
        _check_dev("workspace", workspace)
        p.workspace = workspace.data_ptr()
        p.workspace_bytes = workspace.numel() * workspace.element_size()
    return p


def ccq_fwd_workspace_bytes(p: FwdParams) -> int:
    return int(load_library().ccq_fwd_workspace_bytes(ctypes.byref(p)))


def ccq_chunk_carry_bytes(dtype_code: int, B: int, H: int, T: int, d: int) -> int:
    """Bytes of the chunk-carry buffer (ccq_chunk_carry_bytes)."""
    return int(load_library().ccq_chunk_carry_bytes(dtype_code, B, H, T, d))


def new_chunk_carry(q):
    """A chunk-carry buffer (uint8 device tensor) for a prefill / backward of q's shape and dtype."""
    import torch
    B, H, T, d = q.shape
    n = ccq_chunk_carry_bytes(_dtype_code(q), B, H, T, d)
    if n == 0:
        raise ValueError("unsupported shape or dtype for chunk carries")
    return torch.empty(n, dtype=torch.uint8, device=q.device)


def ccq_fwd_chunked(rule, q, k, v, log_alpha, beta, w_lambda, b_lambda, o=None,
                    carry_in=None, carry_out=None, segments: int = 0, chunk: int = 64,
                    workspace=None, stream=None, phase_events=None, normalize_keys: bool = False,
                    packed_cov: bool = False, chunk_carry=None):
    """Chunked CCQ prefill through the C ABI.  Allocates o (and the workspace if not
    given) with torch; returns o.  ``phase_events``: optional ctypes array of 4 hipEvent_t
    handles recorded around the kernels of the pass.  ``normalize_keys``: the kernels scale
    every key to unit L2 norm first (CCQ_FLAG_NORMALIZE_KEYS).  ``packed_cov``: the carry's
    C is the packed upper triangle (CCQ_FLAG_PACKED_COV).  ``chunk_carry``: optional buffer
    (``new_chunk_carry``) that receives the carry at every chunk start, for ccq_bwd_chunked."""
    import torch
    lib = load_library()
    if o is None:
        o = torch.empty(q.shape[:-1] + (v.shape[-1],), dtype=q.dtype, device=q.device)
    p = make_fwd_params(rule, q, k, v, log_alpha, beta, w_lambda, b_lambda, o,
                        carry_in, carry_out, segments, chunk, workspace, normalize_keys, packed_cov)
    if workspace is None:
        nbytes = int(lib.ccq_fwd_workspace_bytes(ctypes.byref(p)))
        if nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
            p.workspace = workspace.data_ptr()
            p.workspace_bytes = nbytes
    if phase_events is not None:
        p.phase_events = ctypes.cast(phase_events, ctypes.c_void_p)
    if chunk_carry is not None:
        _check_chunk_carry(chunk_carry, q)
        p.chunk_carry = chunk_carry.data_ptr()
    st = lib.ccq_fwd_chunked(ctypes.byref(p), _stream_handle(stream))
    if st != 0:
        raise CcqError(st, "ccq_fwd_chunked")
    return o


def _check_chunk_carry(buf, q):
    _check_dev("chunk_carry", buf)
    B, H, T, d = q.shape
    need = ccq_chunk_carry_bytes(_dtype_code(q), B, H, T, d)
    if buf.numel() * buf.element_size() < need:
        raise ValueError(f"chunk_carry must hold {need} bytes")


def ccq_fwd_chunked_noalloc(rule, q, k, v, log_alpha, beta, w_lambda, b_lambda, o=None,
                            carry_in=None, carry_out=None, segments: int = 0, chunk: int = 64,
                            stream=None, normalize_keys: bool = False, packed_cov: bool = False):
    """ccq_fwd_chunked_noalloc through the C ABI: the prefill with the library's own device array
    as its workspace (nothing is allocated for it; o is allocated here only when not given).
    Returns o."""
    import torch
    lib = load_library()
    if o is None:
        o = torch.empty(q.shape[:-1] + (v.shape[-1],), dtype=q.dtype, device=q.device)
    p = make_fwd_params(rule, q, k, v, log_alpha, beta, w_lambda, b_lambda, o,
                        carry_in, carry_out, segments, chunk, None, normalize_keys, packed_cov)
    st = lib.ccq_fwd_chunked_noalloc(ctypes.byref(p), _stream_handle(stream))
    if st != 0:
        raise CcqError(st, "ccq_fwd_chunked_noalloc")
    return o


def ccq_decode_step(rule, q, k, v, log_alpha, beta, w_lambda, b_lambda, S, C, ksum, n,
                    o=None, stream=None, normalize_keys: bool = False, packed_cov: bool = False):
    """One in-place decode step through the C ABI; returns o [N, H, d_v].  ``normalize_keys``:
    the kernel scales the key to unit L2 norm first (CCQ_FLAG_NORMALIZE_KEYS).  ``packed_cov``:
    C is the packed upper triangle [N, H, d_k (d_k + 1) / 2] (CCQ_FLAG_PACKED_COV)."""
    import torch
    lib = load_library()
    N, H, d_k = q.shape
    d_v = v.shape[-1]
    if o is None:
        o = torch.empty((N, H, d_v), dtype=q.dtype, device=q.device)
    for name, t in (("q", q), ("k", k), ("v", v), ("log_alpha", log_alpha), ("beta", beta), ("o", o)):
        _check_dev(name, t, q.dtype)
    for name, t, dt in (("w_lambda", w_lambda, torch.float32), ("b_lambda", b_lambda, torch.float32),
                        ("S", S, torch.float32), ("C", C, torch.float32), ("ksum", ksum, torch.float32),
                        ("n", n, torch.int64)):
        _check_dev(name, t, dt)
    _check_numel("S", S, N * H * d_v * d_k)
    _check_numel("C", C, N * H * cov_numel(d_k, packed_cov))
    _check_numel("ksum", ksum, N * H * d_k)
    _check_numel("n", n, N * H)
    st = lib.ccq_decode_step(_rule_code(rule), _dtype_code(q), N, H, d_k, d_v,
                             _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                             _ptr(w_lambda), _ptr(b_lambda), _ptr(S), _ptr(C), _ptr(ksum), _ptr(n),
                             _ptr(o), _flags(normalize_keys, packed_cov), _stream_handle(stream))
    if st != 0:
        raise CcqError(st, "ccq_decode_step")
    return o


def ccq_key_subspace(C, ksum, n, k, r: int = 16, needle=None, packed_cov: bool = False, stream=None,
                     iters=None):
    """Key-covariance subspace diagnostic through the C ABI (see ``ccq_key_subspace`` in ccq.h).
    C [B, H, d, d] (or packed [B, H, d (d + 1) / 2]), ksum [B, H, d], n [B, H] int64: the
    statistics; k [B, H, T, d]: the keys to score; needle [B, H, T] bool / uint8 or None;
    iters: optional int32 [B, H] tensor that receives the bisection work per head (multisection
        rounds summed over the eigenvalues).
    Returns (eigvals [B, H, d], basis [B, H, r, d], align [B, H, T], delta_mu [B, H] or None),
    allocated with torch on k's device."""
    import torch
    lib = load_library()
    B, H, T, d = k.shape
    _check_dev("k", k)
    for name, t, dt in (("C", C, torch.float32), ("ksum", ksum, torch.float32), ("n", n, torch.int64)):
        _check_dev(name, t, dt)
    _check_numel("C", C, B * H * cov_numel(d, packed_cov))
    _check_numel("ksum", ksum, B * H * d)
    _check_numel("n", n, B * H)
    dev = k.device
    eig = torch.empty((B, H, d), dtype=torch.float32, device=dev)
    basis = torch.empty((B, H, r, d), dtype=torch.float32, device=dev)
    align = torch.empty((B, H, T), dtype=torch.float32, device=dev)
    if iters is not None:
        _check_dev("iters", iters, torch.int32)
        _check_numel("iters", iters, B * H)
    dmu = None
    nd = None
    if needle is not None:
        nd = needle.to(torch.uint8).contiguous()
        _check_dev("needle", nd)
        _check_numel("needle", nd, B * H * T)
        dmu = torch.empty((B, H), dtype=torch.float32, device=dev)
    st = lib.ccq_key_subspace(_dtype_code(k), B, H, T, d, r, _ptr(C), _ptr(ksum), _ptr(n), _ptr(k), _ptr(nd),
                              _ptr(eig), _ptr(basis), _ptr(align), _ptr(dmu), _ptr(iters),
                              FLAG_PACKED_COV if packed_cov else 0, _stream_handle(stream))
    if st != 0:
        raise CcqError(st, "ccq_key_subspace")
    return eig, basis, align, dmu


def ccq_step_backward(rule, q, k, v, log_alpha, beta, w_lambda, b_lambda, S, C, ksum, n, d_o, dS, dC, dksum,
                      stream=None):
    """Backward of one recurrence step through the C ABI (see ``ccq_step_backward`` in ccq.h).
    The carry before the step (S, C, ksum, n), the token and d_o are inputs; dS, dC, dksum (fp32)
    hold the adjoint of the carry after the step and are overwritten with the adjoint before it.
    Returns a dict of fp32 tensors: dq, dk, dv, dlog_alpha, dbeta (GDN), dw_lambda [N, H, d_k],
    db_lambda [N, H] (per sequence)."""
    import torch
    lib = load_library()
    N, H, d_k = q.shape
    d_v = v.shape[-1]
    for name, t in (("q", q), ("k", k), ("v", v), ("log_alpha", log_alpha), ("beta", beta)):
        _check_dev(name, t, q.dtype)
    for name, t, dt in (("w_lambda", w_lambda, torch.float32), ("b_lambda", b_lambda, torch.float32),
                        ("S", S, torch.float32), ("C", C, torch.float32), ("ksum", ksum, torch.float32),
                        ("n", n, torch.int64), ("d_o", d_o, torch.float32), ("dS", dS, torch.float32),
                        ("dC", dC, torch.float32), ("dksum", dksum, torch.float32)):
        _check_dev(name, t, dt)
    for name, t, cnt in (("S", S, N * H * d_v * d_k), ("C", C, N * H * d_k * d_k), ("ksum", ksum, N * H * d_k),
                         ("n", n, N * H), ("d_o", d_o, N * H * d_v), ("dS", dS, N * H * d_v * d_k),
                         ("dC", dC, N * H * d_k * d_k), ("dksum", dksum, N * H * d_k)):
        _check_numel(name, t, cnt)
    rule_c = _rule_code(rule)
    dev = q.device
    f = dict(dtype=torch.float32, device=dev)
    out = dict(dq=torch.empty((N, H, d_k), **f), dk=torch.empty((N, H, d_k), **f), dv=torch.empty((N, H, d_v), **f),
               dlog_alpha=torch.empty((N, H, d_k) if rule_c == CCQ_RULE_GLA else (N, H), **f),
               dbeta=None if rule_c == CCQ_RULE_GLA else torch.empty((N, H), **f),
               dw_lambda=torch.empty((N, H, d_k), **f), db_lambda=torch.empty((N, H), **f))
    st = lib.ccq_step_backward(rule_c, _dtype_code(q), N, H, d_k, d_v, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                               _ptr(beta), _ptr(w_lambda), _ptr(b_lambda), _ptr(S), _ptr(C), _ptr(ksum), _ptr(n),
                               _ptr(d_o), _ptr(dS), _ptr(dC), _ptr(dksum), _ptr(out["dq"]), _ptr(out["dk"]),
                               _ptr(out["dv"]), _ptr(out["dlog_alpha"]), _ptr(out["dbeta"]), _ptr(out["dw_lambda"]),
                               _ptr(out["db_lambda"]), 0, _stream_handle(stream))
    if st != 0:
        raise CcqError(st, "ccq_step_backward")
    return out


def ccq_bwd_chunked(rule, q, k, v, log_alpha, w_lambda, b_lambda, d_o, carry_in=None, carry_out_adjoint=None,
                    want_carry_in_adjoint: bool = False, workspace=None, stream=None, phase_events=None, beta=None,
                    chunk_carry=None):
    """Chunked backward of the prefill through the C ABI (see ``ccq_bwd_chunked`` in ccq.h).
    q, k, v, d_o: [B, H, T, d] of one dtype; log_alpha: [B, H, T, d] (GLA) or [B, H, T] (Gated
    DeltaNet, with beta [B, H, T]); carry_in: (S0, C0, ksum0, n0) or None; carry_out_adjoint:
    (dS_T, dC_T, dksum_T) fp32 or None.  Returns a dict of fp32 tensors dq, dk, dv, dlog_alpha (the
    shape of log_alpha), dbeta (Gated DeltaNet), dw_lambda [B, H, d], db_lambda [B, H] and, with
    want_carry_in_adjoint, dS0, dC0, dksum0.  ``phase_events``: optional ctypes array of 5
    hipEvent_t handles recorded around the passes.  ``chunk_carry``: the buffer a ccq_fwd_chunked of
    the same inputs filled; the chunk carries are then read from it instead of recomputed."""
    import torch
    lib = load_library()
    B, H, T, d_k = q.shape
    d_v = v.shape[-1]
    rule_c = _rule_code(rule)
    gdn = rule_c == CCQ_RULE_GDN
    if gdn != (beta is not None):
        raise ValueError("beta is given for Gated DeltaNet and only for it")
    for name, t in (("q", q), ("k", k), ("v", v), ("log_alpha", log_alpha), ("d_o", d_o), ("beta", beta)):
        _check_dev(name, t, q.dtype)
        per = d_v if name in ("v", "d_o") else (1 if name == "beta" or (gdn and name == "log_alpha") else d_k)
        _check_numel(name, t, B * H * T * per)
    _check_dev("w_lambda", w_lambda, torch.float32)
    _check_dev("b_lambda", b_lambda, torch.float32)
    p = BwdParams()
    p.rule = rule_c
    p.dtype = _dtype_code(q)
    p.B, p.H, p.T, p.d_k, p.d_v, p.chunk = B, H, T, d_k, d_v, 64
    p.q, p.k, p.v, p.log_alpha, p.d_o = (_ptr(x) for x in (q, k, v, log_alpha, d_o))
    p.w_lambda, p.b_lambda = _ptr(w_lambda), _ptr(b_lambda)
    if carry_in is not None:
        S0, C0, m0, n0 = carry_in
        for name, t, dt, cnt in (("S0", S0, torch.float32, B * H * d_v * d_k), ("C0", C0, torch.float32, B * H * d_k * d_k),
                                 ("ksum0", m0, torch.float32, B * H * d_k), ("n0", n0, torch.int64, B * H)):
            _check_dev(name, t, dt)
            _check_numel(name, t, cnt)
        p.S0, p.C0, p.ksum0, p.n0 = _ptr(S0), _ptr(C0), _ptr(m0), _ptr(n0)
    if carry_out_adjoint is not None:
        dS_T, dC_T, dm_T = carry_out_adjoint
        for name, t, cnt in (("dS_T", dS_T, B * H * d_v * d_k), ("dC_T", dC_T, B * H * d_k * d_k),
                             ("dksum_T", dm_T, B * H * d_k)):
            _check_dev(name, t, torch.float32)
            _check_numel(name, t, cnt)
        p.dS_T, p.dC_T, p.dksum_T = _ptr(dS_T), _ptr(dC_T), _ptr(dm_T)
    f = dict(dtype=torch.float32, device=q.device)
    out = dict(dq=torch.empty((B, H, T, d_k), **f), dk=torch.empty((B, H, T, d_k), **f),
               dv=torch.empty((B, H, T, d_v), **f),
               dlog_alpha=torch.empty((B, H, T) if gdn else (B, H, T, d_k), **f),
               dw_lambda=torch.empty((B, H, d_k), **f), db_lambda=torch.empty((B, H), **f))
    if gdn:
        out["dbeta"] = torch.empty((B, H, T), **f)
        p.beta, p.dbeta = _ptr(beta), _ptr(out["dbeta"])
    if want_carry_in_adjoint:
        out.update(dS0=torch.empty((B, H, d_v, d_k), **f), dC0=torch.empty((B, H, d_k, d_k), **f),
                   dksum0=torch.empty((B, H, d_k), **f))
        p.dS0, p.dC0, p.dksum0 = _ptr(out["dS0"]), _ptr(out["dC0"]), _ptr(out["dksum0"])
    p.dq, p.dk, p.dv, p.dlog_alpha = _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dlog_alpha"])
    p.dw_lambda, p.db_lambda = _ptr(out["dw_lambda"]), _ptr(out["db_lambda"])
    nbytes = int(lib.ccq_bwd_workspace_bytes(ctypes.byref(p)))
    if workspace is None and nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    if workspace is not None:
        _check_dev("workspace", workspace)
        p.workspace = workspace.data_ptr()
        p.workspace_bytes = workspace.numel() * workspace.element_size()
    if phase_events is not None:
        p.phase_events = ctypes.cast(phase_events, ctypes.c_void_p)
    if chunk_carry is not None:
        _check_chunk_carry(chunk_carry, q)
        p.chunk_carry = chunk_carry.data_ptr()
    st = lib.ccq_bwd_chunked(ctypes.byref(p), _stream_handle(stream))
    if st != 0:
        raise CcqError(st, "ccq_bwd_chunked")
    return out


# ---------------------------------------------------------------- operators around the read step
#
# They run on the device of their first tensor, whichever device is current, on the given stream or
# that device's current one; what they allocate belongs to that stream.  A call on a few tokens takes the
# GPU a few microseconds, so the checks here are kept short.

_NORMS = {"none": 0, None: 0, "rms": 1, "l2": 2}
MAX_REORDER_STATES = 16  # CCQ_MAX_REORDER_STATES


class _NoContext:
    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


class _Ops:
    """What every call below looks up, once: torch, its dtypes, and the library's functions."""

    def __init__(self):
        import torch
        lib = load_library()
        self.torch, self.empty, self.empty_strided = torch, torch.empty, torch.empty_strided
        self.f32, self.i32, self.i64, self.u8 = torch.float32, torch.int32, torch.int64, torch.uint8
        self.codes = {torch.float32: CCQ_DTYPE_F32, torch.bfloat16: CCQ_DTYPE_BF16}
        self.current_device, self.raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        self.nowhere = _NoContext()
        for name in ("qk_norm_rope", "qk_norm_rope_backward", "scan", "scan_backward", "beam_select", "beam_reorder",
                     "qk_backward_workspace_bytes", "scan_workspace_bytes", "scan_backward_workspace_bytes",
                     "beam_select_workspace_bytes"):
            setattr(self, name, getattr(lib, "ccq_" + name))

    def dtype_code(self, t):
        code = self.codes.get(t.dtype)
        if code is None:
            raise TypeError(f"unsupported tensor dtype {t.dtype}")
        return code

    def place(self, dev, stream):
        """Context in which a call on tensors of ``dev`` allocates and launches."""
        if dev.type != "cuda":
            raise ValueError("tensors must be device tensors")
        if stream is not None:
            if stream.device != dev:
                raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
            return self.torch.cuda.stream(stream)
        if dev.index != self.current_device():
            return self.torch.cuda.device(dev)
        return self.nowhere


_OPS = None


def _ops():
    global _OPS
    if _OPS is None:
        _OPS = _Ops()
    return _OPS


def _refuse(name, t, dev, dtype, shape, layout):
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, is on {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be {layout}")


def _dense(name, t, dev, dtype, shape):
    """The address of t, which lies on dev, is dense and has this dtype and shape (None: absent)."""
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype or t.device != dev or not t.is_contiguous():
        _refuse(name, t, dev, dtype, shape, "contiguous")
    return t.data_ptr()


def _strided(name, t, dev, dtype, shape):
    """The strides of t, as _dense but dense in its last dimension alone: 0 for the others where there is
    one entry, whose stride means nothing."""
    st = t.stride()
    if t.shape != shape or t.dtype != dtype or t.device != dev or (st[-1] != 1 and shape[-1] != 1):
        _refuse(name, t, dev, dtype, shape, "dense in its last dimension")
    if len(st) == 4:
        return st[0] if shape[0] > 1 else 0, st[1] if shape[1] > 1 else 0, st[2] if shape[2] > 1 else 0
    return st[0] if shape[0] > 1 else 0, st[1] if shape[1] > 1 else 0


def _into(ops, name, t, dev, dtype, shape):
    """An output and its address: the given tensor, checked as by _dense, or a new one."""
    if t is not None:
        return t, _dense(name, t, dev, dtype, shape)
    if len(shape) == 4:
        _, a, b, c = shape
        strides = (a * b * c, b * c, c, 1)
    else:
        _, b, c = shape
        strides = (b * c, c, 1)
    t = ops.empty_strided(shape, strides, dtype=dtype, device=dev)
    return t, t.data_ptr()


def _launch(ops, name, fn, params, dev, size_fn=None, workspace=None):
    """Calls fn, with the workspace that it asks for: the given one, or one allocated here.  The library
    reads its size from the arguments alone, so it is asked first only where one is needed."""
    keep = workspace
    if size_fn is not None:
        if workspace is None:
            need = size_fn(params)
            if need:
                keep = ops.empty(need, dtype=ops.u8, device=dev)
                params.workspace = keep.data_ptr()
                params.workspace_bytes = need
        else:
            if workspace.device != dev or not workspace.is_contiguous():
                raise ValueError(f"workspace must be a contiguous tensor on {dev}")
            params.workspace = workspace.data_ptr()
            params.workspace_bytes = workspace.numel() * workspace.element_size()
    st = fn(params, ops.raw_stream(dev.index))
    if st != 0:
        raise CcqError(st, "ccq_" + name)
    return keep


def _qk_params(ops, q, k, dev, positions, inv_freq, q_weight, k_weight, q_norm, k_norm, eps, interleaved, expand_keys,
               position_offset, q_out, k_out):
    """q_out, k_out: addresses."""
    ref = q if q is not None else k
    dt = ref.dtype
    B, T, _, d = ref.shape
    Hq = Hk = 0
    qs = ks = (0, 0, 0)
    qp = kp = None
    if q is not None:
        Hq = q.shape[2]
        qs, qp = _strided("q", q, dev, dt, (B, T, Hq, d)), q.data_ptr()
    if k is not None:
        if k.dim() != 4:
            raise ValueError("q and k are [B, T, H, d]")
        Hk = k.shape[2]
        ks, kp = _strided("k", k, dev, dt, (B, T, Hk, d)), k.data_ptr()
    if expand_keys and (Hk == 0 or Hq % Hk):
        raise ValueError(f"expand_keys: {Hk} key heads do not divide {Hq} query heads")
    rot, freqs = 0, None
    if inv_freq is not None and inv_freq.numel():
        rot = 2 * inv_freq.numel()
        freqs = _dense("inv_freq", inv_freq, dev, ops.f32, (rot // 2,))
    try:
        norms = _NORMS[q_norm], _NORMS[k_norm]
    except KeyError as e:
        raise ValueError(f"unknown norm {e.args[0]!r}: 'none', 'rms' or 'l2'") from None
    return QkParams(ops.dtype_code(ref), B, T, Hq, Hk, d, *norms, rot, 1 if interleaved else 0, 1 if expand_keys else 0,
                    eps, qp, kp, *qs, *ks, _dense("positions", positions, dev, ops.i64, (B, T)), position_offset, freqs,
                    _dense("q_weight", q_weight, dev, ops.f32, (d,)), _dense("k_weight", k_weight, dev, ops.f32, (d,)),
                    q_out, k_out)


def ccq_qk_norm_rope(q, k, positions=None, inv_freq=None, q_weight=None, k_weight=None, q_norm="rms", k_norm="l2",
                     eps: float = 1e-6, interleaved: bool = False, expand_keys: bool = False,
                     position_offset: int = 0, q_out=None, k_out=None, stream=None):
    """Queries and keys of a projection made ready for the read step (see ``ccq_qk_norm_rope`` in
    ccq.h): every head's row normalised ("rms", "l2" or "none"), weighted, rotated by its position and
    laid out head-major.  q [B, T, H_q, d], k [B, T, H_k, d]: strided views are fine, either may be
    None; positions [B, T] int64, or token t stands at position_offset + t; inv_freq [rot / 2] fp32, or
    None for no rotation.  Returns (q_out [B, H_q, T, d], k_out [B, H_k, T, d], or [B, H_q, T, d] with
    expand_keys), None in the place of an absent side."""
    ref = q if q is not None else k
    if ref is None:
        raise ValueError("q or k must be given")
    if ref.dim() != 4:
        raise ValueError("q and k are [B, T, H, d]")
    ops, dev = _ops(), ref.device
    with ops.place(dev, stream):
        B, T, heads, d = ref.shape
        qp = kp = None
        if q is not None:
            q_out, qp = _into(ops, "q_out", q_out, dev, ref.dtype, (B, heads, T, d))
        elif q_out is not None:
            raise ValueError("q_out is given without q")
        if k is not None:
            k_out, kp = _into(ops, "k_out", k_out, dev, ref.dtype, (B, heads if expand_keys else k.shape[2], T, d))
        elif k_out is not None:
            raise ValueError("k_out is given without k")
        p = _qk_params(ops, q, k, dev, positions, inv_freq, q_weight, k_weight, q_norm, k_norm, eps, interleaved,
                       expand_keys, position_offset, qp, kp)
        _launch(ops, "qk_norm_rope", ops.qk_norm_rope, p, dev)
    return q_out, k_out


def ccq_qk_norm_rope_backward(q, k, dq_out, dk_out, positions=None, inv_freq=None, q_weight=None, k_weight=None,
                              q_norm="rms", k_norm="l2", eps: float = 1e-6, interleaved: bool = False,
                              position_offset: int = 0, dq=None, dk=None, workspace=None, stream=None):
    """Gradient of ``ccq_qk_norm_rope`` (see ``ccq_qk_norm_rope_backward`` in ccq.h).  dq_out, dk_out:
    fp32 gradients of its outputs, dense; dk_out has H_q heads if the keys were expanded.  Returns a
    dict: dq, dk (dtype and shape of q, k, into the given views if any), dq_weight, dk_weight (fp32
    [d], None without that weight)."""
    ref = q if q is not None else k
    if ref is None:
        raise ValueError("q or k must be given")
    if ref.dim() != 4:
        raise ValueError("q and k are [B, T, H, d]")
    ops, dev, dt = _ops(), ref.device, ref.dtype
    with ops.place(dev, stream):
        B, T, _, d = ref.shape
        Hq = 0 if q is None else q.shape[2]
        Hk = 0 if k is None else k.shape[2]
        expand = k is not None and dk_out is not None and dk_out.shape[1] != Hk
        f = _qk_params(ops, q, k, dev, positions, inv_freq, q_weight, k_weight, q_norm, k_norm, eps, interleaved, expand,
                       position_offset, None, None)
        for name, t, heads in (("dq_out", dq_out, Hq), ("dk_out", dk_out, Hk)):
            if (t is None) != (heads == 0):
                raise ValueError(f"{name} is given with its input and only with it")
        qs = ks = (0, 0, 0)
        if q is not None:
            dq = ops.empty((B, T, Hq, d), dtype=dt, device=dev) if dq is None else dq
            qs = _strided("dq", dq, dev, dt, (B, T, Hq, d))
        if k is not None:
            dk = ops.empty((B, T, Hk, d), dtype=dt, device=dev) if dk is None else dk
            ks = _strided("dk", dk, dev, dt, (B, T, Hk, d))
        dwq = None if q_weight is None else ops.empty(d, dtype=ops.f32, device=dev)
        dwk = None if k_weight is None else ops.empty(d, dtype=ops.f32, device=dev)
        p = QkBwdParams(f, _dense("dq_out", dq_out, dev, ops.f32, (B, Hq, T, d)),
                        _dense("dk_out", dk_out, dev, ops.f32, (B, Hq if expand else Hk, T, d)),
                        None if q is None else dq.data_ptr(), None if k is None else dk.data_ptr(), *qs, *ks, _ptr(dwq),
                        _ptr(dwk), None, 0)
        _launch(ops, "qk_norm_rope_backward", ops.qk_norm_rope_backward, p, dev, ops.qk_backward_workspace_bytes, workspace)
    return dict(dq=dq if q is not None else None, dk=dk if k is not None else None, dq_weight=dwq, dk_weight=dwk)


def scan_carry_shape(x):
    """Shape of the chunk-carry tensor of ``ccq_scan`` for inputs x [B, T, D]."""
    B, T, D = x.shape
    return (B, (T + 63) // 64, D)


def ccq_scan(x, log_alpha, h0=None, h_out=None, y=None, lengths=None, complement: bool = False, chunk_carry=None,
             workspace=None, stream=None):
    """Gated linear recurrence h_t = exp(log_alpha_t) h_{t-1} + s_t x_t over [B, T, D] (see ``ccq_scan``
    in ccq.h; s_t is 1, or 1 - exp(log_alpha_t) with complement).  x and log_alpha may be strided
    views; h0, h_out [B, D] fp32 (h_out may be h0: the serving step); lengths [B] int32; chunk_carry:
    fp32 tensor of ``scan_carry_shape(x)`` that receives the state before every 64-token chunk, for
    ``ccq_scan_backward``.  Returns y [B, T, D]: rows at t >= length are left as they were, which in a y
    allocated here (y=None) is whatever the memory held."""
    if x.dim() != 3:
        raise ValueError("x is [B, T, D]")
    ops, dev, dt = _ops(), x.device, x.dtype
    shape = B, T, D = x.shape
    with ops.place(dev, stream):
        y, yp = _into(ops, "y", y, dev, dt, shape)
        p = ScanParams(ops.dtype_code(x), B, T, D, 1 if complement else 0, x.data_ptr(), log_alpha.data_ptr(),
                       *_strided("x", x, dev, dt, shape), *_strided("log_alpha", log_alpha, dev, dt, shape),
                       _dense("lengths", lengths, dev, ops.i32, (B,)), _dense("h0", h0, dev, ops.f32, (B, D)),
                       yp, _dense("h_out", h_out, dev, ops.f32, (B, D)),
                       _dense("chunk_carry", chunk_carry, dev, ops.f32, (B, (T + 63) // 64, D)), None, 0)
        _launch(ops, "scan", ops.scan, p, dev, ops.scan_workspace_bytes, workspace)
    return y


def ccq_scan_backward(x, log_alpha, dy, h0=None, dh_out=None, lengths=None, complement: bool = False,
                      chunk_carry=None, want_dh0: bool = False, dx=None, dlog_alpha=None, workspace=None, stream=None):
    """Gradient of ``ccq_scan`` (see ``ccq_scan_backward`` in ccq.h).  dy [B, T, D]: gradient of y (a
    strided view is fine); dh_out [B, D] fp32: gradient of h_out, or None; chunk_carry: what the
    forward kept, or None to form it again.  Returns a dict: dx, dlog_alpha (dtype of x; zeros at
    t >= length) and, with want_dh0, dh0 fp32."""
    if x.dim() != 3:
        raise ValueError("x is [B, T, D]")
    ops, dev, dt = _ops(), x.device, x.dtype
    shape = B, T, D = x.shape
    with ops.place(dev, stream):
        dx, dxp = _into(ops, "dx", dx, dev, dt, shape)
        dlog_alpha, dgp = _into(ops, "dlog_alpha", dlog_alpha, dev, dt, shape)
        out = dict(dx=dx, dlog_alpha=dlog_alpha)
        if want_dh0:
            out["dh0"] = ops.empty((B, D), dtype=ops.f32, device=dev)
        p = ScanBwdParams(ops.dtype_code(x), B, T, D, 1 if complement else 0, x.data_ptr(), log_alpha.data_ptr(),
                          dy.data_ptr(), *_strided("x", x, dev, dt, shape),
                          *_strided("log_alpha", log_alpha, dev, dt, shape), *_strided("dy", dy, dev, dt, shape),
                          _dense("lengths", lengths, dev, ops.i32, (B,)), _dense("h0", h0, dev, ops.f32, (B, D)),
                          _dense("dh_out", dh_out, dev, ops.f32, (B, D)),
                          _dense("chunk_carry", chunk_carry, dev, ops.f32, (B, (T + 63) // 64, D)),
                          dxp, dgp, _ptr(out.get("dh0")), None, 0)
        _launch(ops, "scan_backward", ops.scan_backward, p, dev, ops.scan_backward_workspace_bytes, workspace)
    return out


def ccq_beam_select(logits, scores, m: int, finished=None, pad_token: int = 0, workspace=None, stream=None):
    """One selection step of beam search (see ``ccq_beam_select`` in ccq.h).  logits [N, K, V] (rows may
    be padded: logits[..., :V] of a wider tensor), scores [N, K] fp32, finished [N, K] bool / uint8 or
    None.  Returns a dict: token, parent (int32 [N, m]) and score (fp32 [N, m]), best first."""
    if logits.dim() != 3:
        raise ValueError("logits is [N, K, V]")
    if m <= 0:
        raise ValueError("m must be positive")
    ops, dev = _ops(), logits.device
    shape = N, K, V = logits.shape
    with ops.place(dev, stream):
        st = _strided("logits", logits, dev, logits.dtype, shape)
        stride = st[1] if K > 1 else st[0] if N > 1 else V
        if N > 1 and K > 1 and st[0] != K * st[1]:
            raise ValueError("the rows of logits must be evenly spaced")
        if finished is not None and finished.dtype == ops.torch.bool:
            finished = finished.view(ops.u8)
        size, strides = (N, m), (m, 1)
        token = ops.empty_strided(size, strides, dtype=ops.i32, device=dev)
        parent = ops.empty_strided(size, strides, dtype=ops.i32, device=dev)
        score = ops.empty_strided(size, strides, dtype=ops.f32, device=dev)
        p = BeamParams(ops.dtype_code(logits), N, K, V, m, logits.data_ptr(), stride,
                       _dense("scores", scores, dev, ops.f32, (N, K)), _dense("finished", finished, dev, ops.u8, (N, K)),
                       pad_token, token.data_ptr(), parent.data_ptr(), score.data_ptr(), None, 0)
        _launch(ops, "beam_select", ops.beam_select, p, dev, ops.beam_select_workspace_bytes, workspace)
    return dict(token=token, parent=parent, score=score)


def ccq_beam_reorder(states, parent, stream=None):
    """Moves every state's rows to the beams that continue them, in place (see ``ccq_beam_reorder`` in
    ccq.h).  states: up to 16 dense tensors [N K, ...] of any dtype whose rows are a multiple of 4
    bytes; parent [N, K] int32, as ``ccq_beam_select`` returns it for m = K."""
    count = len(states)
    if not 0 < count <= MAX_REORDER_STATES:
        raise ValueError(f"1 to {MAX_REORDER_STATES} states, got {count}")
    if parent.dim() != 2:
        raise ValueError("parent is [N, K]")
    ops, dev = _ops(), parent.device
    N, K = parent.shape
    with ops.place(dev, stream):
        at = _dense("parent", parent, dev, ops.i32, (N, K))
        rows = N * K
        for i, t in enumerate(states):
            if t.device != dev or not t.is_contiguous() or t.dim() < 1 or t.shape[0] != rows:
                raise ValueError(f"states[{i}] must be a contiguous tensor on {dev} with {rows} rows")
        ptrs = (ctypes.c_void_p * count)(*[t.data_ptr() for t in states])
        sizes = (ctypes.c_size_t * count)(*[t.nbytes // rows if rows else 0 for t in states])
        st = ops.beam_reorder(count, ptrs, sizes, N, K, at, ops.raw_stream(dev.index))
        if st != 0:
            raise CcqError(st, "ccq_beam_reorder")
