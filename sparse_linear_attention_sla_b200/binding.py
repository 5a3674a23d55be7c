"""Python binding over the C ABI in include/sla.h (argument marshalling only).

Every step of the computation runs in libsla.so's CUDA kernels; this module
checks tensor shapes/dtypes, takes the current torch CUDA stream, allocates
outputs and workspaces with torch, and calls the library through ctypes. There
is no CPU path: without the built library, or without a CUDA device, every
call raises.
"""

from __future__ import annotations

import ctypes
import os
import struct
import threading
from typing import Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsla.so")

SLA_OK = 0
_STATUS = {
    0: "SLA_OK", 1: "SLA_ERR_INVALID_ARG", 2: "SLA_ERR_UNSUPPORTED", 3: "SLA_ERR_WORKSPACE",
    4: "SLA_ERR_CUDA", 5: "SLA_ERR_TIMEOUT", 6: "SLA_ERR_BAD_MASK", 7: "SLA_ERR_BAD_LEN",
}

# Every symbol include/sla.h declares.
EXPORTS = ("sla_counts", "sla_workspace_size", "sla_route", "sla_kv_states", "sla_forward",
           "sla_forward_timed", "sla_check", "sla_last_error", "sla_version", "sla_route_noalloc",
           "sla_selftest_wait_timeout", "sla_workspace_size_fp8", "sla_forward_fp8", "sla_forward_fp8_timed",
           "sla_quantize_kv", "sla_aggregate_states", "sla_forward_launches", "sla_route_variant",
           "sla_forward_variant", "sla_workspace_size_backward", "sla_backward", "sla_workspace_size_pisa",
           "sla_forward_pisa", "sla_pisa_hbar", "sla_lowbit_codes", "sla_rotary", "sla_rotary_backward",
           "sla_workspace_size_attend", "sla_workspace_size_attend_backward", "sla_attend", "sla_attend_backward")


class SlaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS.get(status, status)}: {message}")
        self.status = status


class Variant(ctypes.Structure):
    """sla_variant: feature_map 0 (elu + 1) or 1 (exp); block_score 0 (first order) or 1 (second order);
    linear_scale, drop_threshold: the linear branch is dropped when linear_scale < drop_threshold."""
    _fields_ = [("feature_map", ctypes.c_int), ("block_score", ctypes.c_int), ("linear_scale", ctypes.c_float),
                ("drop_threshold", ctypes.c_float)]


class Problem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("N", ctypes.c_int), ("D", ctypes.c_int),
                ("block_q", ctypes.c_int), ("block_kv", ctypes.c_int),
                ("kh", ctypes.c_float), ("kl", ctypes.c_float)]


class Tensor(ctypes.Structure):
    """sla_tensor: a [B, H, N, D] device tensor with contiguous channels, strides in elements."""
    _fields_ = [("ptr", ctypes.c_void_p), ("stride_b", ctypes.c_int64), ("stride_h", ctypes.c_int64),
                ("stride_n", ctypes.c_int64)]


class RotarySpec(ctypes.Structure):
    """sla_rotary_spec (made by rotary_spec, which keeps the positions tensor alive)."""
    _fields_ = [("n_axes", ctypes.c_int), ("channels", ctypes.c_int * 4), ("grid", ctypes.c_int * 4),
                ("start", ctypes.c_int * 4), ("positions", ctypes.c_void_p), ("positions_stride_b", ctypes.c_int64),
                ("pairing", ctypes.c_int), ("base", ctypes.c_double)]
    positions_tensor = None


_ROTARY_SPEC = struct.Struct("@13iPqid")  # RotarySpec's fields, in C's own alignment
assert _ROTARY_SPEC.size == ctypes.sizeof(RotarySpec)


class AttendProblem(ctypes.Structure):
    """sla_attend_problem."""
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("Hk", ctypes.c_int), ("Nq", ctypes.c_int),
                ("Nk", ctypes.c_int), ("D", ctypes.c_int), ("causal", ctypes.c_int), ("scale", ctypes.c_float)]


_lib = None
_lib_lock = threading.Lock()


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libsla.so and declare its signatures. Raises if the library is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lib_lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with `python -m sparse_linear_attention_sla_b200.build` "
                "(there is no CPU fallback)")
        lib = ctypes.CDLL(path)
        P = ctypes.POINTER(Problem)
        vp, sz = ctypes.c_void_p, ctypes.c_size_t
        ip = ctypes.POINTER(ctypes.c_int)
        lib.sla_counts.argtypes = [P, ip, ip, ip, ip]
        lib.sla_workspace_size.argtypes = [P]
        lib.sla_workspace_size.restype = sz
        lib.sla_route.argtypes = [P, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.sla_kv_states.argtypes = [P, vp, vp, vp, vp, vp, sz, vp]
        lib.sla_forward.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.sla_forward_timed.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, sz, vp, ctypes.POINTER(ctypes.c_float)]
        lib.sla_check.argtypes = [vp, vp]
        lib.sla_workspace_size_fp8.argtypes = [P]
        lib.sla_workspace_size_fp8.restype = sz
        lib.sla_forward_fp8.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.sla_forward_fp8_timed.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, sz, vp, ctypes.POINTER(ctypes.c_float)]
        lib.sla_quantize_kv.argtypes = [P, vp, vp, vp, vp, vp, vp, vp]
        lib.sla_selftest_wait_timeout.argtypes = [vp, sz, ctypes.c_uint, vp]
        lib.sla_selftest_wait_timeout.restype = ctypes.c_int
        lib.sla_aggregate_states.argtypes = [P, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.sla_workspace_size_backward.argtypes = [P]
        lib.sla_workspace_size_backward.restype = sz
        lib.sla_backward.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.sla_workspace_size_pisa.argtypes = [P]
        lib.sla_workspace_size_pisa.restype = sz
        lib.sla_forward_pisa.argtypes = [P, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.sla_pisa_hbar.argtypes = [P, vp, vp, vp, vp, sz, vp]
        pp = ctypes.POINTER(ctypes.c_void_p)
        lib.sla_lowbit_codes.argtypes = [P, vp, sz, pp, pp, pp, pp]
        V = ctypes.POINTER(Variant)
        lib.sla_route_variant.argtypes = [P, V, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.sla_forward_variant.argtypes = [P, V, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.sla_forward_launches.argtypes = [P, ctypes.c_int, ctypes.c_int]
        lib.sla_forward_launches.restype = ctypes.c_int
        R, T, A = ctypes.POINTER(RotarySpec), ctypes.POINTER(Tensor), ctypes.POINTER(AttendProblem)
        i = ctypes.c_int
        lib.sla_rotary.argtypes = [R, i, i, i, i, i, i, T, T, T, T, vp]
        lib.sla_rotary_backward.argtypes = [R, i, i, i, i, i, i, i, T, T, T, T, vp]
        lib.sla_workspace_size_attend.argtypes = [A]
        lib.sla_workspace_size_attend.restype = sz
        lib.sla_workspace_size_attend_backward.argtypes = [A]
        lib.sla_workspace_size_attend_backward.restype = sz
        lib.sla_attend.argtypes = [A, T, T, T, vp, T, vp, vp, sz, vp]
        lib.sla_attend_backward.argtypes = [A, T, T, T, T, vp, T, vp, T, T, T, vp, sz, vp]
        lib.sla_last_error.restype = ctypes.c_char_p
        lib.sla_version.restype = ctypes.c_char_p
        for name in ("sla_counts", "sla_route", "sla_kv_states", "sla_forward", "sla_forward_timed", "sla_check",
                     "sla_forward_fp8", "sla_forward_fp8_timed", "sla_quantize_kv", "sla_forward_pisa",
                     "sla_pisa_hbar", "sla_aggregate_states", "sla_backward", "sla_route_variant",
                     "sla_forward_variant", "sla_lowbit_codes", "sla_rotary", "sla_rotary_backward", "sla_attend",
                     "sla_attend_backward"):
            getattr(lib, name).restype = ctypes.c_int
        _lib = lib
        return lib


def _raise(status: int):
    if status != SLA_OK:
        msg = load_library().sla_last_error().decode(errors="replace")
        raise SlaError(status, msg)


def problem(B, H, N, D, block_q, block_kv, kh=0.0, kl=0.0) -> Problem:
    return Problem(int(B), int(H), int(N), int(D), int(block_q), int(block_kv), float(kh), float(kl))


def counts(p: Problem) -> Tuple[int, int, int, int]:
    """(Nq, Nk, kc, kn) as the library computes them (host only)."""
    out = [ctypes.c_int(0) for _ in range(4)]
    _raise(load_library().sla_counts(ctypes.byref(p), *[ctypes.byref(o) for o in out]))
    return tuple(o.value for o in out)


def workspace_size(p: Problem) -> int:
    return int(load_library().sla_workspace_size(ctypes.byref(p)))


def workspace_size_fp8(p: Problem) -> int:
    return int(load_library().sla_workspace_size_fp8(ctypes.byref(p)))


def new_workspace(p: Problem, device, fp8: bool = False) -> torch.Tensor:
    """A zero-headed workspace for problem p on device (bytes, 256-byte aligned by the allocator);
    fp8=True sizes it for forward_fp8."""
    n = workspace_size_fp8(p) if fp8 else workspace_size(p)
    if n == 0:
        counts(p)  # raises with the library's message
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def _stream_handle(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check_act(name, t, B, H, N, D, device):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16 or tuple(t.shape) != (B, H, N, D) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous bf16 of shape {(B, H, N, D)}, got {t.dtype} {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _ptr(t: Optional[torch.Tensor]):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def route(q, k, block_q, block_kv, kh, kl, want_scores=False, want_crit=False, ws=None):
    """Block labels [B,H,Nq,Nk] int8 (2 critical, 1 marginal, 0 negligible).

    Returns (mask, crit_idx or None, scores or None).
    """
    B, H, N, D = q.shape
    _check_act("q", q, B, H, N, D, q.device)
    _check_act("k", k, B, H, N, D, q.device)
    p = problem(B, H, N, D, block_q, block_kv, kh, kl)
    Nq, Nk, kc, _ = counts(p)
    dev = q.device
    mask = torch.empty(B, H, Nq, Nk, dtype=torch.int8, device=dev)
    crit = torch.empty(B, H, Nq, kc, dtype=torch.int32, device=dev) if want_crit else None
    scores = torch.empty(B, H, Nq, Nk, dtype=torch.float64, device=dev) if want_scores else None
    if ws is None:
        ws = new_workspace(p, dev)
    lib = load_library()
    with torch.cuda.device(dev):
        st = lib.sla_route(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(mask), _ptr(crit), _ptr(scores), _ptr(ws),
                           ctypes.c_size_t(ws.numel()), _stream_handle(dev))
    _raise(st)
    return mask, crit, scores


def kv_states(k, v, block_kv=64, ws=None):
    """Per-KV-block states h [B,H,Nk,D,D] and z [B,H,Nk,D], fp32."""
    B, H, N, D = k.shape
    _check_act("k", k, B, H, N, D, k.device)
    _check_act("v", v, B, H, N, D, k.device)
    p = problem(B, H, N, D, 128 if D == 128 else 64, block_kv)
    _, Nk, _, _ = counts(p)
    dev = k.device
    h = torch.empty(B, H, Nk, D, D, dtype=torch.float32, device=dev)
    z = torch.empty(B, H, Nk, D, dtype=torch.float32, device=dev)
    if ws is None:
        ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    lib = load_library()
    with torch.cuda.device(dev):
        st = lib.sla_kv_states(ctypes.byref(p), _ptr(k), _ptr(v), _ptr(h), _ptr(z), _ptr(ws),
                               ctypes.c_size_t(ws.numel()), _stream_handle(dev))
    _raise(st)
    return h, z


def aggregate_states(k, v, mask, block_q, block_kv=64, ws=None):
    """Per-query-block sums of the marginal blocks' states: H [B,H,Nq,D,D] bf16, Z [B,H,Nq,D] fp32."""
    B, H, N, D = k.shape
    _check_act("k", k, B, H, N, D, k.device)
    _check_act("v", v, B, H, N, D, k.device)
    p = problem(B, H, N, D, block_q, block_kv)
    Nq, Nk, _, _ = counts(p)
    dev = k.device
    if mask.dtype != torch.int8 or tuple(mask.shape) != (B, H, Nq, Nk) or not mask.is_contiguous() \
            or mask.device != dev:
        raise ValueError(f"mask must be contiguous int8 [{B}, {H}, {Nq}, {Nk}] on {dev}")
    Hs = torch.empty(B, H, Nq, D, D, dtype=torch.bfloat16, device=dev)
    Zs = torch.empty(B, H, Nq, D, dtype=torch.float32, device=dev)
    if ws is None:
        ws = new_workspace(p, dev)
    lib = load_library()
    with torch.cuda.device(dev):
        st = lib.sla_aggregate_states(ctypes.byref(p), _ptr(k), _ptr(v), _ptr(mask), _ptr(Hs), _ptr(Zs), _ptr(ws),
                                      ctypes.c_size_t(ws.numel()), _stream_handle(dev))
    _raise(st)
    return Hs, Zs, ws


def route_variant(q, k, block_q, block_kv, kh, kl, feature_map=0, block_score=0, want_scores=False,
                  want_crit=False, ws=None):
    """sla_route_variant: labels [B,H,Nq,Nk] int8 (and crit_idx, scores when asked)."""
    B, H, N, D = q.shape
    _check_act("q", q, B, H, N, D, q.device)
    _check_act("k", k, B, H, N, D, q.device)
    p = problem(B, H, N, D, block_q, block_kv, kh, kl)
    Nq, Nk, kc, _ = counts(p)
    dev = q.device
    mask = torch.empty(B, H, Nq, Nk, dtype=torch.int8, device=dev)
    crit = torch.empty(B, H, Nq, kc, dtype=torch.int32, device=dev) if want_crit else None
    scores = torch.empty(B, H, Nq, Nk, dtype=torch.float64, device=dev) if want_scores else None
    if ws is None:
        ws = new_workspace(p, dev)
    var = Variant(feature_map, block_score, 0.0, 0.0)
    lib = load_library()
    with torch.cuda.device(dev):
        st = lib.sla_route_variant(ctypes.byref(p), ctypes.byref(var), _ptr(q), _ptr(k), _ptr(mask), _ptr(crit),
                                   _ptr(scores), _ptr(ws), ctypes.c_size_t(ws.numel()), _stream_handle(dev))
    _raise(st)
    return mask, crit, scores


def forward_variant(q, k, v, alpha, block_q, block_kv, kh, kl, feature_map=0, block_score=0, mask=None, out=None,
                    ws=None, linear_scale=0.0, drop_threshold=0.0, rotary_by=None):
    """sla_forward_variant: O [B,H,N,D] bf16. rotary_by: as for forward."""
    q, k = _rotated(q, k, rotary_by)
    p, out, ws = _forward_args(q, k, v, alpha, block_q, block_kv, kh, kl, mask, out, ws)
    var = Variant(feature_map, block_score, float(linear_scale), float(drop_threshold))
    lib = load_library()
    dev = q.device
    with torch.cuda.device(dev):
        st = lib.sla_forward_variant(ctypes.byref(p), ctypes.byref(var), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                                     _ptr(mask), _ptr(out), _ptr(ws), ctypes.c_size_t(ws.numel()),
                                     _stream_handle(dev))
    _raise(st)
    return out


def backward(q, k, v, alpha, dO, block_q=128, block_kv=64, kh=0.05, kl=0.10, mask=None, ws=None, rotary_by=None):
    """sla_backward: (dQ, dK, dV [B,H,N,D] fp32, dalpha [H,D] fp32) of sum(dO * O).

    rotary_by: as for forward; dQ and dK are then the gradients of the q and k given here."""
    q, k = _rotated(q, k, rotary_by)
    B, H, N, D = q.shape
    dev = q.device
    for name, t in (("q", q), ("k", k), ("v", v), ("dO", dO)):
        _check_act(name, t, B, H, N, D, dev)
    if alpha.dtype != torch.float32 or tuple(alpha.shape) != (H, D) or not alpha.is_contiguous():
        raise ValueError(f"alpha must be contiguous fp32 [{H}, {D}]")
    p = problem(B, H, N, D, block_q, block_kv, kh, kl)
    Nq, Nk, _, _ = counts(p)
    if mask is not None and (mask.dtype != torch.int8 or tuple(mask.shape) != (B, H, Nq, Nk)
                             or not mask.is_contiguous()):
        raise ValueError(f"mask must be contiguous int8 [{B}, {H}, {Nq}, {Nk}]")
    lib = load_library()
    if ws is None:
        n = lib.sla_workspace_size_backward(ctypes.byref(p))
        if n == 0:
            counts(p)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        ws[:256].zero_()
    dQ, dK, dV = (torch.empty(B, H, N, D, dtype=torch.float32, device=dev) for _ in range(3))
    dalpha = torch.empty(H, D, dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        st = lib.sla_backward(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(mask), _ptr(dO),
                              _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(dalpha), _ptr(ws), ctypes.c_size_t(ws.numel()),
                              _stream_handle(dev))
    _raise(st)
    if rotary_by is not None:
        rotary_backward(dQ, dK, rotary_by, out=(dQ, dK))
    return dQ, dK, dV, dalpha, ws


def lowbit_codes(ws: torch.Tensor, B, H, N, D, block_q=128, block_kv=64):
    """Copies of the e4m3 codes of K and V ([B,H,N,D] uint8) and block exponents ([B,H,Nk] int32)
    that the last forward_fp8 on workspace ws wrote."""
    p = problem(B, H, N, D, block_q, block_kv)
    _, Nk, _, _ = counts(p)
    ptrs = [ctypes.c_void_p() for _ in range(4)]
    _raise(load_library().sla_lowbit_codes(ctypes.byref(p), _ptr(ws), ctypes.c_size_t(ws.numel()),
                                           *[ctypes.byref(x) for x in ptrs]))
    base = ws.data_ptr()
    out = []
    for x, n, dt in ((ptrs[0], B * H * N * D, torch.uint8), (ptrs[1], B * H * N * D, torch.uint8),
                     (ptrs[2], B * H * Nk, torch.int32), (ptrs[3], B * H * Nk, torch.int32)):
        off = x.value - base
        nbytes = n * (4 if dt == torch.int32 else 1)
        out.append(ws[off:off + nbytes].view(dt).clone())
    return (out[0].view(B, H, N, D), out[1].view(B, H, N, D), out[2].view(B, H, Nk), out[3].view(B, H, Nk))


def new_workspace_pisa(p: Problem, device) -> torch.Tensor:
    """A zero-headed workspace of sla_workspace_size_pisa(p) bytes on device."""
    n = int(load_library().sla_workspace_size_pisa(ctypes.byref(p)))
    if n == 0:
        counts(p)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def forward_pisa(q, k, v, block_q=128, block_kv=64, kh=0.05, kl=0.10, labels=None, out=None, ws=None,
                 rotary_by=None):
    """sla_forward_pisa: O [B,H,N,D] bf16. labels [B,H,Nq,Nk] int8 (2 = critical) or None (the router).
    rotary_by: as for forward."""
    q, k = _rotated(q, k, rotary_by)
    B, H, N, D = q.shape
    dev = q.device
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_act(name, t, B, H, N, D, dev)
    p = problem(B, H, N, D, block_q, block_kv, kh, kl)
    Nq, Nk, _, _ = counts(p)
    if labels is not None and (labels.dtype != torch.int8 or tuple(labels.shape) != (B, H, Nq, Nk)
                               or not labels.is_contiguous() or labels.device != dev):
        raise ValueError(f"labels must be contiguous int8 [{B}, {H}, {Nq}, {Nk}] on {dev}")
    if out is None:
        out = torch.empty_like(q)
    if ws is None:
        ws = new_workspace_pisa(p, dev)
    lib = load_library()
    with torch.cuda.device(dev):
        st = lib.sla_forward_pisa(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(labels), _ptr(out), _ptr(ws),
                                  ctypes.c_size_t(ws.numel()), _stream_handle(dev))
    _raise(st)
    return out


def pisa_hbar(k, v, block_kv=64, ws=None):
    """sla_pisa_hbar: Hbar [B,H,D,D] fp32, the mean over KV blocks of (K_j - kbar_j)^T V_j."""
    B, H, N, D = k.shape
    dev = k.device
    for name, t in (("k", k), ("v", v)):
        _check_act(name, t, B, H, N, D, dev)
    p = problem(B, H, N, D, 128, block_kv)
    if ws is None:
        ws = new_workspace_pisa(p, dev)
    out = torch.empty(B, H, D, D, dtype=torch.float32, device=dev)
    lib = load_library()
    with torch.cuda.device(dev):
        st = lib.sla_pisa_hbar(ctypes.byref(p), _ptr(k), _ptr(v), _ptr(out), _ptr(ws), ctypes.c_size_t(ws.numel()),
                               _stream_handle(dev))
    _raise(st)
    return out


def forward_launches(p, with_mask=False, low_bit=False) -> int:
    """Kernel launches one sla_forward (or sla_forward_fp8) call enqueues for problem p."""
    n = load_library().sla_forward_launches(ctypes.byref(p), int(bool(with_mask)), int(bool(low_bit)))
    if n < 0:
        raise SlaError(1, "invalid problem")
    return n


def _forward_args(q, k, v, alpha, block_q, block_kv, kh, kl, mask, out, ws, fp8=False):
    B, H, N, D = q.shape
    dev = q.device
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_act(name, t, B, H, N, D, dev)
    if alpha.dtype != torch.float32 or tuple(alpha.shape) != (H, D) or not alpha.is_contiguous() or alpha.device != dev:
        raise ValueError(f"alpha must be contiguous fp32 [{H}, {D}] on {dev}")
    p = problem(B, H, N, D, block_q, block_kv, kh, kl)
    Nq, Nk, _, _ = counts(p)
    if mask is not None:
        if mask.dtype != torch.int8 or tuple(mask.shape) != (B, H, Nq, Nk) or not mask.is_contiguous() \
                or mask.device != dev:
            raise ValueError(f"mask must be contiguous int8 [{B}, {H}, {Nq}, {Nk}] on {dev}")
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_act("out", out, B, H, N, D, dev)
    if ws is None:
        ws = new_workspace(p, dev, fp8)
    return p, out, ws


def _rotated(q, k, spec):
    """q and k as the attention takes them: themselves, or turned by the rotary_spec."""
    return (q, k) if spec is None else rotary(q, k, spec)


def forward(q, k, v, alpha, block_q=128, block_kv=64, kh=0.05, kl=0.10, mask=None, out=None, ws=None,
            rotary_by=None):
    """Fused SLA forward: O = alpha * O_s + (1 - alpha) * O_l, bf16 [B,H,N,D].

    rotary_by: a rotary_spec by whose positions q and k are turned first. They may then have any
    strides with contiguous channels (a projection's [B,N,H,D] output as its transpose(1, 2))."""
    q, k = _rotated(q, k, rotary_by)
    p, out, ws = _forward_args(q, k, v, alpha, block_q, block_kv, kh, kl, mask, out, ws)
    lib = load_library()
    with torch.cuda.device(q.device):
        st = lib.sla_forward(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(mask), _ptr(out),
                             _ptr(ws), ctypes.c_size_t(ws.numel()), _stream_handle(q.device))
    _raise(st)
    return out


def forward_timed(q, k, v, alpha, block_q=128, block_kv=64, kh=0.05, kl=0.10, mask=None, out=None, ws=None):
    """forward() plus per-stage device milliseconds (precompute, route, aggregate, attention).

    Synchronises the current stream."""
    p, out, ws = _forward_args(q, k, v, alpha, block_q, block_kv, kh, kl, mask, out, ws)
    ms = (ctypes.c_float * 4)()
    lib = load_library()
    with torch.cuda.device(q.device):
        st = lib.sla_forward_timed(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(mask), _ptr(out),
                                   _ptr(ws), ctypes.c_size_t(ws.numel()), _stream_handle(q.device), ms)
    _raise(st)
    return out, [float(x) for x in ms]


def forward_fp8(q, k, v, alpha, block_q=128, block_kv=64, kh=0.05, kl=0.10, mask=None, out=None, ws=None,
                rotary_by=None):
    """forward() with the low-bit (e4m3) sparse branch (include/sla.h states the reading); D = 128."""
    q, k = _rotated(q, k, rotary_by)
    p, out, ws = _forward_args(q, k, v, alpha, block_q, block_kv, kh, kl, mask, out, ws, fp8=True)
    lib = load_library()
    with torch.cuda.device(q.device):
        st = lib.sla_forward_fp8(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(mask), _ptr(out),
                                 _ptr(ws), ctypes.c_size_t(ws.numel()), _stream_handle(q.device))
    _raise(st)
    return out


def forward_fp8_timed(q, k, v, alpha, block_q=128, block_kv=64, kh=0.05, kl=0.10, mask=None, out=None, ws=None):
    """forward_fp8() plus per-stage device milliseconds (precompute, route, aggregate, quantise,
    attention). Synchronises the current stream."""
    p, out, ws = _forward_args(q, k, v, alpha, block_q, block_kv, kh, kl, mask, out, ws, fp8=True)
    ms = (ctypes.c_float * 5)()
    lib = load_library()
    with torch.cuda.device(q.device):
        st = lib.sla_forward_fp8_timed(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(mask),
                                       _ptr(out), _ptr(ws), ctypes.c_size_t(ws.numel()), _stream_handle(q.device), ms)
    _raise(st)
    return out, [float(x) for x in ms]


def quantize_kv(k, v, block_kv=64):
    """e4m3 codes of K and V ([B,H,N,D] uint8) and their per-KV-block scale exponents
    ([B,H,Nk] int32): code * 2^exp approximates the input."""
    B, H, N, D = k.shape
    _check_act("k", k, B, H, N, D, k.device)
    _check_act("v", v, B, H, N, D, k.device)
    p = problem(B, H, N, D, 128 if D == 128 else 64, block_kv)
    _, Nk, _, _ = counts(p)
    dev = k.device
    k8 = torch.empty(B, H, N, D, dtype=torch.uint8, device=dev)
    v8 = torch.empty(B, H, N, D, dtype=torch.uint8, device=dev)
    kexp = torch.empty(B, H, Nk, dtype=torch.int32, device=dev)
    vexp = torch.empty(B, H, Nk, dtype=torch.int32, device=dev)
    lib = load_library()
    with torch.cuda.device(dev):
        st = lib.sla_quantize_kv(ctypes.byref(p), _ptr(k), _ptr(v), _ptr(k8), _ptr(v8), _ptr(kexp), _ptr(vexp),
                                 _stream_handle(dev))
    _raise(st)
    return k8, v8, kexp, vexp


def rotary_spec(axes, grid=None, positions=None, start=None, base=10000.0, pairing=0) -> RotarySpec:
    """What rotary and rotary_backward turn by.

    axes: channels of each axis (even; one to four axes, together at most D; channels behind them
    are copied). Positions are either a grid, one extent per axis (token n at its n-th cell, the
    last axis fastest, the first cell at `start`; tokens behind the last cell are copied), or an
    int32 tensor [N, len(axes)] or [B, N, len(axes)]. pairing: 0 neighbouring channels, 1 the two
    halves of an axis' channels.
    """
    axes = tuple(map(int, axes))
    n = len(axes)
    if not 1 <= n <= 4:
        raise ValueError(f"one to four axes, got {n}")
    if (grid is None) == (positions is None):
        raise ValueError("give either grid or positions")
    if grid is not None:
        grid = tuple(map(int, grid))
        start = tuple(map(int, start)) if start is not None else (0,) * n
        if len(grid) != n or len(start) != n:
            raise ValueError(f"grid and start need one entry per axis ({n})")
        where, stride = 0, 0
    else:
        if start is not None:
            raise ValueError("start goes with grid")
        if not isinstance(positions, torch.Tensor) or not positions.is_cuda or positions.dtype != torch.int32 \
                or positions.dim() not in (2, 3) or positions.shape[-1] != n or not positions.is_contiguous():
            raise ValueError(f"positions must be a contiguous int32 CUDA tensor [N, {n}] or [B, N, {n}]")
        grid = start = (0,) * n
        where, stride = positions.data_ptr(), positions.shape[-2] * n if positions.dim() == 3 else 0
    none = (0,) * (4 - n)
    try:  # packed in one step: filling the structure field by field takes longer than the kernel's launch
        spec = RotarySpec.from_buffer_copy(_ROTARY_SPEC.pack(n, *axes, *none, *grid, *none, *start, *none, where, stride,
                                                             int(pairing), float(base)))
    except struct.error as e:
        raise ValueError(f"channels, grid, start and pairing must fit 32 bits: {e}") from None
    spec.positions_tensor = positions
    return spec


def _check_heads(name, t, B, H, N, D, dtype, device):
    """A [B, H, N, D] tensor whose channels are contiguous (the library checks the other strides), as
    the library takes it."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    strides = t.stride()
    if t.dtype is not dtype or t.shape != (B, H, N, D) or strides[3] != 1:
        raise ValueError(f"{name} must be {dtype} of shape {(B, H, N, D)} with contiguous channels, got {t.dtype} "
                         f"{tuple(t.shape)} with strides {strides}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return Tensor(t.data_ptr(), strides[0], strides[1], strides[2])


def _new_heads(device, B, H, N, D, dtype):
    """A contiguous [B, H, N, D] tensor, and as the library takes it."""
    n = N * D
    t = torch.empty_strided((B, H, N, D), (H * n, n, D, 1), dtype=dtype, device=device)
    return t, Tensor(t.data_ptr(), H * n, n, D)


def _address(t: Optional[torch.Tensor]):
    return t.data_ptr() if t is not None else None


class _Call:
    """Calls a library function with the device of its tensors current, on torch's current stream there. (Where
    that device is current already, as it nearly always is, nothing is switched.)"""

    def __init__(self, device):
        self.device = device
        self.stream = torch._C._cuda_getCurrentRawStream(device.index)

    def __call__(self, f, *args):
        if torch._C._cuda_getDevice() == self.device.index:
            status = f(*args, self.stream)
        else:
            with torch.cuda.device(self.device):
                status = f(*args, self.stream)
        if status != SLA_OK:
            _raise(status)


def _span(t):
    """The bytes [first, last) that a tensor's elements lie in."""
    first = t.data_ptr()
    return first, first + (sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) * t.element_size()


def _check_apart(name, y, *others):
    """The output y shares no memory with the other tensors. Heads or tokens of one buffer that lie between
    each other's rows are apart where neither's rows reach into the other's."""
    c, d = _span(y)
    for x in others:
        a, b = _span(x)
        if a < d and c < b and not _interleaved(x, y):
            raise ValueError(f"{name} overlaps another tensor of the call")


def _interleaved(x, y):
    """x and y are slices of one buffer that never meet: every step between rows is a multiple of the smallest, and
    within that one their row blocks lie apart."""
    steps = [s * t.element_size() for t in (x, y) for n, s in zip(t.shape[:3], t.stride()) if n > 1 and s > 0]
    for period in sorted(set(steps)):
        def block(t):  # bytes of the dimensions that stay within the period
            return (sum((n - 1) * s for n, s in zip(t.shape, t.stride()) if s * t.element_size() < period) + 1) \
                * t.element_size()
        if any(s % period and s > period for s in steps):
            continue
        gap = (y.data_ptr() - x.data_ptr()) % period
        if block(x) <= gap and block(y) <= period - gap:
            return True
    return False


def _check_in_place(name, x, y):
    """y is x itself, or apart from it: tensors that share part of their memory cannot be rotated."""
    if y.data_ptr() == x.data_ptr() and y.stride() == x.stride() and y.dtype == x.dtype:
        return
    _check_apart(name, y, x)


def _rotary_call(q, k, spec, out, dtype, names, backward):
    if not isinstance(spec, RotarySpec):
        raise ValueError("spec must come from rotary_spec")
    first = q if q is not None else k
    if first is None:
        raise ValueError(f"give {names[0]} or {names[1]}")
    if not isinstance(first, torch.Tensor) or first.dim() != 4:
        raise ValueError(f"{names[0]} and {names[1]} must be [B, H, N, D] tensors")
    (B, _, N, D), dev, in_dtype = first.shape, first.device, first.dtype
    if max(first.shape) >= 2 ** 31:
        raise ValueError(f"sizes must fit 32 bits, got {tuple(first.shape)}")
    if in_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"{names[0]} and {names[1]} must be bf16 or fp32, got {in_dtype}")
    dtype = in_dtype if dtype is None else dtype
    if dtype != in_dtype and (in_dtype, dtype) != (torch.float32, torch.bfloat16):
        raise ValueError(f"{in_dtype} gradients cannot be given back as {dtype}")
    pos = spec.positions_tensor
    if pos is not None and (pos.device != dev or pos.shape[-2] != N or (pos.dim() == 3 and pos.shape[0] != B)):
        raise ValueError(f"positions {tuple(pos.shape)} on {pos.device} do not fit {B} sequences of {N} tokens on {dev}")
    outs, args, heads = [None, None], [None] * 4, [0, 0]
    for w, x in enumerate((q, k)):
        if x is None:
            continue
        H = heads[w] = x.shape[1] if isinstance(x, torch.Tensor) and x.dim() == 4 else 0
        args[2 * w] = _check_heads(names[w], x, B, H, N, D, in_dtype, dev)
        y = out[w] if out is not None else None
        if y is None:
            outs[w], args[2 * w + 1] = _new_heads(dev, B, H, N, D, dtype)
        else:
            args[2 * w + 1] = _check_heads(f"out of {names[w]}", y, B, H, N, D, dtype, dev)
            _check_in_place(f"out of {names[w]}", x, y)
            outs[w] = y
    if out is not None and args[0] is not None and args[2] is not None:  # one's output may not be the other's
        _check_apart(f"out of {names[0]}", outs[0], k, outs[1])
        _check_apart(f"out of {names[1]}", outs[1], q)
    lib, call = load_library(), _Call(dev)
    in_code, out_code = int(in_dtype is torch.float32), int(dtype is torch.float32)  # SLA_BF16, SLA_F32
    if backward:
        call(lib.sla_rotary_backward, spec, B, heads[0], heads[1], N, D, in_code, out_code, *args)
    else:
        call(lib.sla_rotary, spec, B, heads[0], heads[1], N, D, in_code, *args)
    return outs[0], outs[1]


def rotary(q, k, spec, out=None):
    """sla_rotary: q [B,H,N,D] and k [B,Hk,N,D] (bf16 or fp32; either may be None) turned by their
    tokens' positions.

    Any strides with contiguous channels: a projection's [B,N,H,D] output goes in as its
    transpose(1, 2). Returns contiguous tensors, or the pair `out` (an entry may be its own input:
    in place)."""
    return _rotary_call(q, k, spec, out, None, ("q", "k"), False)


def rotary_backward(dq, dk, spec, dtype=None, out=None):
    """sla_rotary_backward: the gradients of rotary's inputs from those of its outputs. dtype: of
    the result (the gradients' own, or bf16 for fp32 gradients, as backward gives them)."""
    return _rotary_call(dq, dk, spec, out, dtype, ("dq", "dk"), True)


def attend_problem(q, k, causal=False, scale=None) -> AttendProblem:
    """The sla_attend_problem of q [B,H,Nq,D] and k [B,Hk,Nk,D]."""
    if not isinstance(q, torch.Tensor) or not isinstance(k, torch.Tensor) or q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be [B, H, N, D] tensors")
    B, H, Nq, D = q.shape
    _, Hk, Nk, _ = k.shape
    if max(B, H, Nq, Hk, Nk, D) >= 2 ** 31:
        raise ValueError(f"sizes must fit 32 bits, got {tuple(q.shape)} and {tuple(k.shape)}")
    scale = float(scale) if scale is not None else max(D, 1) ** -0.5
    return AttendProblem(B, H, Hk, Nq, Nk, D, int(bool(causal)), scale)


def new_workspace_attend(p: AttendProblem, device, backward: bool = False) -> torch.Tensor:
    """A zero-headed workspace for attend (backward=True: attend_backward) of problem p on device."""
    ws = _attend_space(p, device, backward)
    ws[:256].zero_()
    return ws


def _attend_space(p, device, backward):
    lib = load_library()
    n = (lib.sla_workspace_size_attend_backward if backward else lib.sla_workspace_size_attend)(p)
    if n == 0:
        raise SlaError(1, lib.sla_last_error().decode(errors="replace"))
    return torch.empty(n, dtype=torch.uint8, device=device)


def _given_space(ws, dev):
    if not isinstance(ws, torch.Tensor) or ws.device != dev or ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise ValueError(f"ws must be a workspace of new_workspace_attend on {dev}")
    return ws


def _attend_inputs(q, k, v, kv_lens, causal, scale):
    p = attend_problem(q, k, causal, scale)
    (B, H, Nq, D), (_, Hk, Nk, _) = q.shape, k.shape
    dev, bf16 = q.device, torch.bfloat16
    args = (_check_heads("q", q, B, H, Nq, D, bf16, dev), _check_heads("k", k, B, Hk, Nk, D, bf16, dev),
            _check_heads("v", v, B, Hk, Nk, D, bf16, dev))
    if kv_lens is not None and (not isinstance(kv_lens, torch.Tensor) or kv_lens.dtype != torch.int32
                                or tuple(kv_lens.shape) != (B,) or not kv_lens.is_contiguous()
                                or kv_lens.device != dev):
        raise ValueError(f"kv_lens must be contiguous int32 [{B}] on {dev}")
    return p, (B, H, Hk, Nq, Nk, D), dev, args


def attend(q, k, v, kv_lens=None, causal=False, scale=None, out=None, ws=None):
    """sla_attend: (out [B,H,Nq,D] bf16, lse [B,H,Nq] fp32) of softmax(scale q k^T) v.

    q [B,H,Nq,D], k and v [B,Hk,Nk,D] bf16 with contiguous channels and any other strides; Hk
    divides H. kv_lens: int32 [B] keys of each sequence (None: Nk). causal: query i sees the keys
    j <= i + len - Nq. scale: 1 / sqrt(D) if None. A query without keys gives 0 and lse = -inf.
    ws: new_workspace_attend's, kept where a device-side error is to be asked for with check(ws): without one of
    the caller's, a length outside [0, Nk] or a wait that ran out shows nowhere."""
    p, (B, H, Hk, Nq, Nk, D), dev, args = _attend_inputs(q, k, v, kv_lens, causal, scale)
    if out is None:
        out, o = _new_heads(dev, B, H, Nq, D, torch.bfloat16)
    else:
        o = _check_heads("out", out, B, H, Nq, D, torch.bfloat16, dev)
        _check_apart("out", out, q, k, v)
    lse = q.new_empty((B, H, Nq), dtype=torch.float32)
    ws = _attend_space(p, dev, False) if ws is None else _given_space(ws, dev)
    _Call(dev)(load_library().sla_attend, p, *args, _address(kv_lens), o, lse.data_ptr(), ws.data_ptr(), ws.numel())
    return out, lse


def attend_backward(q, k, v, out, lse, dO, kv_lens=None, causal=False, scale=None, ws=None):
    """sla_attend_backward: (dq [B,H,Nq,D], dk, dv [B,Hk,Nk,D]) bf16 of sum(dO * out), from attend's
    out and lse of the same arguments. Equal calls give equal bits. ws: new_workspace_attend's with
    backward=True; as for attend."""
    p, (B, H, Hk, Nq, Nk, D), dev, args = _attend_inputs(q, k, v, kv_lens, causal, scale)
    o = _check_heads("out", out, B, H, Nq, D, torch.bfloat16, dev)
    g = _check_heads("dO", dO, B, H, Nq, D, torch.bfloat16, dev)
    if not isinstance(lse, torch.Tensor) or lse.dtype != torch.float32 or lse.shape != (B, H, Nq) \
            or not lse.is_contiguous() or lse.device != dev:
        raise ValueError(f"lse must be contiguous fp32 [{B}, {H}, {Nq}] on {dev}")
    dq, a = _new_heads(dev, B, H, Nq, D, torch.bfloat16)
    dk, b = _new_heads(dev, B, Hk, Nk, D, torch.bfloat16)
    dv, c = _new_heads(dev, B, Hk, Nk, D, torch.bfloat16)
    ws = _attend_space(p, dev, True) if ws is None else _given_space(ws, dev)
    _Call(dev)(load_library().sla_attend_backward, p, *args, o, lse.data_ptr(), g, _address(kv_lens), a, b, c,
               ws.data_ptr(), ws.numel())
    return dq, dk, dv


def check(ws: torch.Tensor):
    """Synchronise and raise if a kernel recorded a device-side error in ws."""
    lib = load_library()
    with torch.cuda.device(ws.device):
        _raise(lib.sla_check(_ptr(ws), _stream_handle(ws.device)))


def selftest_wait_timeout(ws: torch.Tensor, limit_us: int = 50000):
    """Enqueue the device self-test of the bounded-wait path (see include/sla.h); a
    following check(ws) raises SlaError with status SLA_ERR_TIMEOUT."""
    lib = load_library()
    with torch.cuda.device(ws.device):
        _raise(lib.sla_selftest_wait_timeout(_ptr(ws), ctypes.c_size_t(ws.numel()), ctypes.c_uint(int(limit_us)),
                                             _stream_handle(ws.device)))


def version() -> str:
    return load_library().sla_version().decode()
