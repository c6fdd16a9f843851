"""Python binding of the lbq C ABI (include/lbq.h).

Argument marshalling only: every computation runs in the CUDA kernels of
liblbq.so.  The low-level functions (`lbq_quantize`, `lbq_linear_fwd`, ...)
have the C names and take raw integers (device pointers, sizes, stream
handles) and `lbq_qweight` structures.  The helpers below them accept torch
tensors, allocate outputs and workspaces with torch (device memory is the one
thing PyTorch supplies) and pass pointers through.

There is no fallback: importing this module fails when liblbq.so is missing,
and every call raises `LbqError` when the library returns a non-OK status.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import re
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "liblbq.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "lbq.h")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m qlora_quantized_linear_b200.build`")
_L = ctypes.CDLL(LIB_PATH)

LBQ_OK, LBQ_EINVAL, LBQ_EALIGN, LBQ_EUNSUPPORTED, LBQ_ECUDA, LBQ_ETIMEOUT, LBQ_EWORKSPACE = range(7)
LBQ_MINMAX_ASYM, LBQ_CODEBOOK4 = 0, 1
LBQ_F32, LBQ_BF16, LBQ_F16 = 0, 1, 2
STATUS_TIMEOUT, STATUS_BAD_TABLE = 1, 2


class lbq_qweight(ctypes.Structure):
    _fields_ = [
        ("n", ctypes.c_int32), ("k", ctypes.c_int32),
        ("bits", ctypes.c_int32), ("group", ctypes.c_int32),
        ("scheme", ctypes.c_int32), ("double_quant", ctypes.c_int32),
        ("packed", ctypes.c_void_p),
        ("scale", ctypes.c_void_p), ("zero", ctypes.c_void_p),
        ("absmax", ctypes.c_void_p),
        ("absmax_q8", ctypes.c_void_p), ("absmax_s2", ctypes.c_void_p), ("absmax_offset", ctypes.c_void_p),
        ("codebook", ctypes.c_void_p),
    ]


class lbq_qweight_mix(ctypes.Structure):
    _fields_ = [("hi", lbq_qweight), ("lo", lbq_qweight), ("perm", ctypes.c_void_p)]


class lbq_fwd_problem(ctypes.Structure):
    _fields_ = [("X", ctypes.c_void_p), ("q", ctypes.POINTER(lbq_qweight)), ("A", ctypes.c_void_p),
                ("B", ctypes.c_void_p), ("rank", ctypes.c_int32), ("s", ctypes.c_float),
                ("Y", ctypes.c_void_p), ("T_save", ctypes.c_void_p)]


class lbq_bwd_problem(ctypes.Structure):
    _fields_ = [("dY", ctypes.c_void_p), ("q", ctypes.POINTER(lbq_qweight)), ("A", ctypes.c_void_p),
                ("B", ctypes.c_void_p), ("rank", ctypes.c_int32), ("s", ctypes.c_float),
                ("dX", ctypes.c_void_p), ("U_save", ctypes.c_void_p)]


class lbq_mix_problem(ctypes.Structure):
    _fields_ = [("X", ctypes.c_void_p), ("q", ctypes.POINTER(lbq_qweight_mix)), ("A", ctypes.c_void_p),
                ("B", ctypes.c_void_p), ("rank", ctypes.c_int32), ("s", ctypes.c_float),
                ("Y", ctypes.c_void_p), ("T_save", ctypes.c_void_p)]


class lbq_i8weight(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("k", ctypes.c_int32), ("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


class lbq_grad(ctypes.Structure):
    _fields_ = [("g", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_vp, _int, _f32, _sz, _u32p = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.POINTER(ctypes.c_uint32)
_QP, _MP = ctypes.POINTER(lbq_qweight), ctypes.POINTER(lbq_qweight_mix)
_PP, _QPP, _I64P = ctypes.POINTER(lbq_fwd_problem), ctypes.POINTER(ctypes.POINTER(lbq_qweight)), ctypes.POINTER(ctypes.c_int64)
_BPP = ctypes.POINTER(lbq_bwd_problem)
_MPP = ctypes.POINTER(lbq_mix_problem)
_IP, _GP = ctypes.POINTER(lbq_i8weight), ctypes.POINTER(lbq_grad)
_SIGS = {
    "lbq_status_string": (ctypes.c_char_p, [_int]),
    "lbq_quantize_workspace_size": (_sz, [_QP]),
    "lbq_quantize": (_int, [_vp, _QP, _vp, _sz, _vp]),
    "lbq_dequantize": (_int, [_QP, _vp, _vp]),
    "lbq_linear_fwd_workspace_size": (_sz, [_int, _QP, _int]),
    "lbq_linear_fwd": (_int, [_vp, _int, _QP, _vp, _vp, _int, _f32, _vp, _vp, _vp, _sz, _vp]),
    "lbq_linear_fwd_noalloc": (_int, [_vp, _int, _QP, _vp, _vp, _int, _f32, _vp, _vp, _vp]),
    "lbq_linear_fwd_mix_workspace_size": (_sz, [_int, _MP, _int]),
    "lbq_linear_fwd_mix": (_int, [_vp, _int, _MP, _vp, _vp, _int, _f32, _vp, _vp, _vp, _sz, _vp]),
    "lbq_linear_bwd_workspace_size": (_sz, [_int, _QP, _int]),
    "lbq_linear_bwd": (_int, [_vp, _int, _QP, _vp, _vp, _int, _f32, _vp, _vp, _vp, _sz, _vp]),
    "lbq_lora_grads": (_int, [_vp, _vp, _int, _int, _int, _vp, _vp, _int, _f32, _vp, _vp, _vp]),
    "lbq_device_status": (_int, [_u32p]),
    "lbq_merge_lora": (_int, [_QP, _vp, _vp, _int, _f32, _vp, _vp]),
    "lbq_gemv_plan": (_int, [_int, _QPP, _int, _int, _I64P, _I64P]),
    "lbq_linear_fwd_grouped_workspace_size": (_sz, [_int, _PP, _int]),
    "lbq_linear_fwd_grouped": (_int, [_int, _PP, _int, _vp, _sz, _vp]),
    "lbq_linear_bwd_grouped_workspace_size": (_sz, [_int, _BPP, _int]),
    "lbq_linear_bwd_grouped": (_int, [_int, _BPP, _int, _vp, _sz, _vp]),
    "lbq_unmerge_lora": (_int, [_vp, _int, _int, _vp, _vp, _int, _f32, _vp, _vp]),
    "lbq_linear_fwd_noalloc_reset": (_int, [_vp]),
    "lbq_channel_mix_select_workspace_size": (_sz, [_int, _int]),
    "lbq_channel_mix_select": (_int, [_vp, _int, _int, _vp, _int, _int, _vp, _vp, _vp, _sz, _vp]),
    "lbq_gather_rows": (_int, [_vp, _int, _int, _vp, _int, _vp, _vp]),
    "lbq_selftest_wait_timeout": (_int, [ctypes.c_uint32, _vp]),
    "lbq_linear_fwd_mix_grouped_workspace_size": (_sz, [_int, _MPP, _int]),
    "lbq_linear_fwd_mix_grouped": (_int, [_int, _MPP, _int, _vp, _sz, _vp]),
    "lbq_quantize_i8": (_int, [_vp, _int, _int, _int, _vp, _vp, _vp]),
    "lbq_linear_i8_fwd_workspace_size": (_sz, [_int, _IP, _int]),
    "lbq_linear_i8_fwd": (_int, [_vp, _int, _IP, _vp, _vp, _int, _f32, _vp, _vp, _vp, _sz, _vp]),
    "lbq_linear_i8_bwd_workspace_size": (_sz, [_int, _IP, _int]),
    "lbq_linear_i8_bwd": (_int, [_vp, _int, _IP, _vp, _vp, _int, _f32, _vp, _vp, _vp, _sz, _vp]),
    "lbq_grad_norm_workspace_size": (_sz, [_int]),
    "lbq_grad_norm": (_int, [_GP, _int, _vp, _vp, _sz, _vp]),
    "lbq_clip_grad_norm": (_int, [_GP, _int, _f32, _vp, _vp, _sz, _vp]),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_L, _name)
    _f.restype, _f.argtypes = _res, _args


def header_functions():
    """Names of the functions that include/lbq.h declares."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\*?\s+\*?(lbq_\w+)\(", text, re.M)))


# --------------------------------------------------------------------------- C names
lbq_status_string = _L.lbq_status_string
lbq_quantize_workspace_size = _L.lbq_quantize_workspace_size
lbq_quantize = _L.lbq_quantize
lbq_dequantize = _L.lbq_dequantize
lbq_linear_fwd_workspace_size = _L.lbq_linear_fwd_workspace_size
lbq_linear_fwd = _L.lbq_linear_fwd
lbq_linear_fwd_noalloc = _L.lbq_linear_fwd_noalloc
lbq_linear_fwd_mix_workspace_size = _L.lbq_linear_fwd_mix_workspace_size
lbq_linear_fwd_mix = _L.lbq_linear_fwd_mix
lbq_linear_bwd_workspace_size = _L.lbq_linear_bwd_workspace_size
lbq_linear_bwd = _L.lbq_linear_bwd
lbq_lora_grads = _L.lbq_lora_grads
lbq_device_status = _L.lbq_device_status
lbq_merge_lora = _L.lbq_merge_lora
lbq_gemv_plan = _L.lbq_gemv_plan
lbq_linear_fwd_grouped_workspace_size = _L.lbq_linear_fwd_grouped_workspace_size
lbq_linear_fwd_grouped = _L.lbq_linear_fwd_grouped
lbq_linear_bwd_grouped_workspace_size = _L.lbq_linear_bwd_grouped_workspace_size
lbq_linear_bwd_grouped = _L.lbq_linear_bwd_grouped
lbq_unmerge_lora = _L.lbq_unmerge_lora
lbq_linear_fwd_noalloc_reset = _L.lbq_linear_fwd_noalloc_reset
lbq_channel_mix_select_workspace_size = _L.lbq_channel_mix_select_workspace_size
lbq_channel_mix_select = _L.lbq_channel_mix_select
lbq_gather_rows = _L.lbq_gather_rows
lbq_selftest_wait_timeout = _L.lbq_selftest_wait_timeout
lbq_linear_fwd_mix_grouped_workspace_size = _L.lbq_linear_fwd_mix_grouped_workspace_size
lbq_linear_fwd_mix_grouped = _L.lbq_linear_fwd_mix_grouped
lbq_quantize_i8 = _L.lbq_quantize_i8
lbq_linear_i8_fwd_workspace_size = _L.lbq_linear_i8_fwd_workspace_size
lbq_linear_i8_fwd = _L.lbq_linear_i8_fwd
lbq_linear_i8_bwd_workspace_size = _L.lbq_linear_i8_bwd_workspace_size
lbq_linear_i8_bwd = _L.lbq_linear_i8_bwd
lbq_grad_norm_workspace_size = _L.lbq_grad_norm_workspace_size
lbq_grad_norm = _L.lbq_grad_norm
lbq_clip_grad_norm = _L.lbq_clip_grad_norm


class LbqError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {lbq_status_string(code).decode()} (status {code})")


def _check(code: int, what: str) -> None:
    if code != LBQ_OK:
        raise LbqError(code, what)


# --------------------------------------------------------------------------- torch helpers
def _torch():
    import torch
    return torch


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _on(stream):
    """Makes a caller's stream the current one while a helper allocates and launches: a temporary is then filled in
    that stream's order and its memory goes back to that stream."""
    torch = _torch()
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _bf16_2d(t, name):
    torch = _torch()
    if t.dtype != torch.bfloat16 or t.dim() != 2 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-D bf16 CUDA tensor")
    return t


class QuantizedWeight:
    """Device buffers of one quantized weight plus its `lbq_qweight` view.

    scheme "minmax": bits 4 (group 128) or 2 (group 64).
    scheme "codebook": 4-bit codes, absmax per 64, optional double quantization;
    `codebook` is 16 sorted floats in [-1, 1] with an exact 0.
    """

    def __init__(self, n: int, k: int, scheme: str = "minmax", bits: int = 4, group: Optional[int] = None,
                 double_quant: bool = False, codebook=None, device="cuda"):
        torch = _torch()
        self.n, self.k, self.scheme, self.bits = int(n), int(k), scheme, int(bits)
        self.double_quant = bool(double_quant)
        u8, f32 = torch.uint8, torch.float32
        if scheme == "minmax":
            self.group = int(group or (128 if bits == 4 else 64))
            self.packed = torch.empty((n, k * bits // 8), dtype=u8, device=device)
            self.scale = torch.empty((n, k // self.group), dtype=torch.float16, device=device)
            self.zero = torch.empty((n, k // self.group), dtype=torch.float16, device=device)
            self.absmax = self.q8 = self.s2 = self.offset = self.codebook = None
        elif scheme == "codebook":
            self.group, self.bits = 64, 4
            nb = n * k // 64
            self.packed = torch.empty((n, k // 2), dtype=u8, device=device)
            self.scale = self.zero = None
            self.absmax = torch.empty(nb, dtype=f32, device=device)
            self.codebook = torch.as_tensor(codebook, dtype=f32).to(device).contiguous()
            if self.double_quant:
                self.q8 = torch.empty(nb, dtype=torch.int8, device=device)
                self.s2 = torch.empty((nb + 255) // 256, dtype=f32, device=device)
                self.offset = torch.empty(4, dtype=f32, device=device)  # 1 used; 16-byte buffer
            else:
                self.q8 = self.s2 = self.offset = None
        else:
            raise ValueError(f"unknown scheme {scheme!r}")
        self.struct = self._make_struct()

    def _make_struct(self) -> lbq_qweight:
        return lbq_qweight(
            n=self.n, k=self.k, bits=self.bits, group=self.group,
            scheme=LBQ_MINMAX_ASYM if self.scheme == "minmax" else LBQ_CODEBOOK4,
            double_quant=int(self.double_quant),
            packed=_ptr(self.packed), scale=_ptr(self.scale), zero=_ptr(self.zero), absmax=_ptr(self.absmax),
            absmax_q8=_ptr(self.q8), absmax_s2=_ptr(self.s2), absmax_offset=_ptr(self.offset),
            codebook=_ptr(self.codebook))

    def quantize(self, W, stream=None) -> "QuantizedWeight":
        torch = _torch()
        W = _bf16_2d(W, "W")
        assert tuple(W.shape) == (self.n, self.k)
        nws = lbq_quantize_workspace_size(ctypes.byref(self.struct))
        ws = torch.empty(max(nws, 16), dtype=torch.uint8, device=W.device) if nws else None
        _check(lbq_quantize(W.data_ptr(), ctypes.byref(self.struct), _ptr(ws), nws, _stream(stream)), "lbq_quantize")
        self._keep = ws
        return self

    def dequantize(self, stream=None):
        torch = _torch()
        out = torch.empty((self.n, self.k), dtype=torch.float32, device=self.packed.device)
        _check(lbq_dequantize(ctypes.byref(self.struct), out.data_ptr(), _stream(stream)), "lbq_dequantize")
        return out


class ChannelMixWeight:
    """Channel-mix weight: INT4 g128 rows `hi`, INT2 g64 rows `lo`, and perm
    (stored row -> original output channel; rows of hi first)."""

    def __init__(self, hi: QuantizedWeight, lo: QuantizedWeight, perm):
        torch = _torch()
        self.hi, self.lo = hi, lo
        self.perm = torch.as_tensor(perm, dtype=torch.int32).to(hi.packed.device).contiguous()
        self.n, self.k = hi.n + lo.n, hi.k
        self.struct = lbq_qweight_mix(hi=hi.struct, lo=lo.struct, perm=self.perm.data_ptr())


def channel_mix_select(W, X_calib, n4: int, stream=None):
    """(perm int32 [n], score fp64 [n]) on the device: the n4 channels of W
    whose INT4 -> INT2 error rise, weighted by the calibration activations'
    second moments, is largest come first (lbq_channel_mix_select)."""
    torch = _torch()
    W, X_calib = _bf16_2d(W, "W"), _bf16_2d(X_calib, "X_calib")
    n, k = W.shape
    perm = torch.empty(n, dtype=torch.int32, device=W.device)
    score = torch.empty(n, dtype=torch.float64, device=W.device)
    nws = lbq_channel_mix_select_workspace_size(n, k)
    ws = torch.empty(max(nws, 16), dtype=torch.uint8, device=W.device)
    _check(lbq_channel_mix_select(W.data_ptr(), n, k, X_calib.data_ptr(), X_calib.shape[0], int(n4), score.data_ptr(),
                                  perm.data_ptr(), ws.data_ptr(), nws, _stream(stream)), "lbq_channel_mix_select")
    return perm, score


def gather_rows(W, rows, stream=None):
    """W[rows] (bf16 rows gathered on the device by lbq_gather_rows)."""
    torch = _torch()
    W = _bf16_2d(W, "W")
    rows = torch.as_tensor(rows, dtype=torch.int32, device=W.device).contiguous()
    out = torch.empty((rows.numel(), W.shape[1]), dtype=torch.bfloat16, device=W.device)
    _check(lbq_gather_rows(W.data_ptr(), W.shape[0], W.shape[1], rows.data_ptr(), rows.numel(), out.data_ptr(),
                           _stream(stream)), "lbq_gather_rows")
    return out


def channel_mix_weight(W, X_calib, frac_int4: float = 0.25, stream=None):
    """A ChannelMixWeight of W: the round(frac_int4 * n) most sensitive channels
    (lbq_channel_mix_select) as INT4 g128 rows, the others as INT2 g64 rows."""
    n, k = W.shape
    n4 = int(round(frac_int4 * n))
    perm, _ = channel_mix_select(W, X_calib, n4, stream=stream)
    hi = QuantizedWeight(n4, k, "minmax", 4).quantize(gather_rows(W, perm[:n4], stream=stream), stream=stream)
    lo = QuantizedWeight(n - n4, k, "minmax", 2).quantize(gather_rows(W, perm[n4:], stream=stream), stream=stream)
    return ChannelMixWeight(hi, lo, perm)


def _workspace(nbytes: int, device):
    torch = _torch()
    # zero-filled once: the library leaves its counters at zero after every call
    return torch.zeros(max(int(nbytes), 16), dtype=torch.uint8, device=device) if nbytes else None


def linear_fwd(X, qw, A=None, B=None, s: float = 0.0, Y=None, T=None, workspace=None, stream=None):
    """Y = X W^T + s (X A^T) B^T; returns (Y fp32 [m, n], T fp32 [m, rank] or None)."""
    torch = _torch()
    X = _bf16_2d(X, "X")
    m = X.shape[0]
    rank = 0 if A is None else int(A.shape[0])
    if Y is None:
        Y = torch.empty((m, qw.n), dtype=torch.float32, device=X.device)
    if rank > 0 and T is None:
        T = torch.empty((m, rank), dtype=torch.float32, device=X.device)
    mix = isinstance(qw, ChannelMixWeight)
    size_fn = lbq_linear_fwd_mix_workspace_size if mix else lbq_linear_fwd_workspace_size
    nws = size_fn(m, ctypes.byref(qw.struct), rank)
    if workspace is None:
        workspace = _workspace(nws, X.device)
    fn = lbq_linear_fwd_mix if mix else lbq_linear_fwd
    _check(fn(X.data_ptr(), m, ctypes.byref(qw.struct), _ptr(A), _ptr(B), rank, float(s), Y.data_ptr(), _ptr(T),
              _ptr(workspace), nws, _stream(stream)), fn.__name__)
    return Y, T


def linear_fwd_grouped(problems, workspace=None, stream=None):
    """Several forwards with the same token count in one call.  `problems` is a
    list of (X, qw) or (X, qw, A, B, s) tuples; returns the list of Y (and T
    when an adapter is given) as linear_fwd would."""
    torch = _torch()
    arr = (lbq_fwd_problem * len(problems))()
    outs, keep = [], []
    m = None
    for i, pr in enumerate(problems):
        X, qw = _bf16_2d(pr[0], "X"), pr[1]
        A, B, s = (pr[2], pr[3], pr[4]) if len(pr) > 2 else (None, None, 0.0)
        m = X.shape[0] if m is None else m
        if X.shape[0] != m:
            raise ValueError("all problems of a grouped call have the same token count")
        rank = 0 if A is None else int(A.shape[0])
        Y = torch.empty((m, qw.n), dtype=torch.float32, device=X.device)
        T = torch.empty((m, rank), dtype=torch.float32, device=X.device) if rank else None
        arr[i] = lbq_fwd_problem(X=X.data_ptr(), q=ctypes.pointer(qw.struct), A=_ptr(A), B=_ptr(B), rank=rank,
                                 s=float(s), Y=Y.data_ptr(), T_save=_ptr(T))
        outs.append((Y, T))
        keep.append((X, A, B))
    nws = lbq_linear_fwd_grouped_workspace_size(m, arr, len(problems))
    if workspace is None:
        workspace = _workspace(nws, problems[0][0].device)
    _check(lbq_linear_fwd_grouped(m, arr, len(problems), _ptr(workspace), nws, _stream(stream)),
           "lbq_linear_fwd_grouped")
    return outs


def linear_fwd_mix_grouped(problems, workspace=None, stream=None):
    """Several channel-mix forwards with the same token count in one call.
    `problems` is a list of (X, ChannelMixWeight) or (X, ChannelMixWeight, A,
    B, s) tuples; returns the list of (Y, T) as linear_fwd would."""
    torch = _torch()
    arr = (lbq_mix_problem * len(problems))()
    outs, keep = [], []
    m = None
    for i, pr in enumerate(problems):
        X, mw = _bf16_2d(pr[0], "X"), pr[1]
        A, B, s = (pr[2], pr[3], pr[4]) if len(pr) > 2 else (None, None, 0.0)
        m = X.shape[0] if m is None else m
        if X.shape[0] != m:
            raise ValueError("all problems of a grouped call have the same token count")
        rank = 0 if A is None else int(A.shape[0])
        Y = torch.empty((m, mw.n), dtype=torch.float32, device=X.device)
        T = torch.empty((m, rank), dtype=torch.float32, device=X.device) if rank else None
        arr[i] = lbq_mix_problem(X=X.data_ptr(), q=ctypes.pointer(mw.struct), A=_ptr(A), B=_ptr(B), rank=rank,
                                 s=float(s), Y=Y.data_ptr(), T_save=_ptr(T))
        outs.append((Y, T))
        keep.append((X, A, B))
    nws = lbq_linear_fwd_mix_grouped_workspace_size(m, arr, len(problems))
    if workspace is None:
        workspace = _workspace(nws, problems[0][0].device)
    _check(lbq_linear_fwd_mix_grouped(m, arr, len(problems), _ptr(workspace), nws, _stream(stream)),
           "lbq_linear_fwd_mix_grouped")
    return outs


def linear_bwd(dY, qw, A=None, B=None, s: float = 0.0, dX=None, U=None, workspace=None, stream=None):
    """dX = dY W + s (dY B) A; returns (dX fp32 [m, k], U fp32 [m, rank] or None)."""
    torch = _torch()
    dY = _bf16_2d(dY, "dY")
    m = dY.shape[0]
    rank = 0 if A is None else int(A.shape[0])
    if dX is None:
        dX = torch.empty((m, qw.k), dtype=torch.float32, device=dY.device)
    if rank > 0 and U is None:
        U = torch.empty((m, rank), dtype=torch.float32, device=dY.device)
    nws = lbq_linear_bwd_workspace_size(m, ctypes.byref(qw.struct), rank)
    if workspace is None:
        workspace = _workspace(nws, dY.device)
    _check(lbq_linear_bwd(dY.data_ptr(), m, ctypes.byref(qw.struct), _ptr(A), _ptr(B), rank, float(s), dX.data_ptr(),
                          _ptr(U), _ptr(workspace), nws, _stream(stream)), "lbq_linear_bwd")
    return dX, U


def linear_bwd_grouped(problems, workspace=None, stream=None):
    """Several backward passes with the same token count in one call.
    `problems` is a list of (dY, qw) or (dY, qw, A, B, s) tuples; returns the
    list of (dX, U) as linear_bwd would."""
    torch = _torch()
    arr = (lbq_bwd_problem * len(problems))()
    outs, keep = [], []
    m = None
    for i, pr in enumerate(problems):
        dY, qw = _bf16_2d(pr[0], "dY"), pr[1]
        A, B, s = (pr[2], pr[3], pr[4]) if len(pr) > 2 else (None, None, 0.0)
        m = dY.shape[0] if m is None else m
        if dY.shape[0] != m:
            raise ValueError("all problems of a grouped call have the same token count")
        rank = 0 if A is None else int(A.shape[0])
        dX = torch.empty((m, qw.k), dtype=torch.float32, device=dY.device)
        U = torch.empty((m, rank), dtype=torch.float32, device=dY.device) if rank else None
        arr[i] = lbq_bwd_problem(dY=dY.data_ptr(), q=ctypes.pointer(qw.struct), A=_ptr(A), B=_ptr(B), rank=rank,
                                 s=float(s), dX=dX.data_ptr(), U_save=_ptr(U))
        outs.append((dX, U))
        keep.append((dY, A, B))
    nws = lbq_linear_bwd_grouped_workspace_size(m, arr, len(problems))
    if workspace is None:
        workspace = _workspace(nws, problems[0][0].device)
    _check(lbq_linear_bwd_grouped(m, arr, len(problems), _ptr(workspace), nws, _stream(stream)),
           "lbq_linear_bwd_grouped")
    return outs


def lora_grads(X, dY, T, U, s: float, dA=None, dB=None, stream=None):
    """dA = s U^T X [rank, k], dB = s dY^T T [n, rank] (fp32)."""
    torch = _torch()
    X, dY = _bf16_2d(X, "X"), _bf16_2d(dY, "dY")
    m, k = X.shape
    n = dY.shape[1]
    rank = int(T.shape[1])
    if dA is None:
        dA = torch.empty((rank, k), dtype=torch.float32, device=X.device)
    if dB is None:
        dB = torch.empty((n, rank), dtype=torch.float32, device=X.device)
    _check(lbq_lora_grads(X.data_ptr(), dY.data_ptr(), m, n, k, T.data_ptr(), U.data_ptr(), rank, float(s),
                          dA.data_ptr(), dB.data_ptr(), _stream(stream)), "lbq_lora_grads")
    return dA, dB


def merge_lora(qw, A=None, B=None, s: float = 0.0, out=None, stream=None):
    """bf16 [n, k]: the dequantized weight plus s B A (the adapter merged in)."""
    torch = _torch()
    rank = 0 if A is None else int(A.shape[0])
    if rank:
        A, B = _bf16_2d(A, "A"), _bf16_2d(B, "B")
    if out is None:
        out = torch.empty((qw.n, qw.k), dtype=torch.bfloat16, device=qw.packed.device)
    _check(lbq_merge_lora(ctypes.byref(qw.struct), _ptr(A) if rank else None, _ptr(B) if rank else None, rank,
                          float(s), out.data_ptr(), _stream(stream)), "lbq_merge_lora")
    return out


def unmerge_lora(W, A=None, B=None, s: float = 0.0, out=None, stream=None):
    """bf16 [n, k]: W minus s B A (a merged adapter removed); out may be W."""
    torch = _torch()
    W = _bf16_2d(W, "W")
    n, k = W.shape
    rank = 0 if A is None else int(A.shape[0])
    if rank:
        A, B = _bf16_2d(A, "A"), _bf16_2d(B, "B")
    if out is None:
        out = torch.empty_like(W)
    _check(lbq_unmerge_lora(W.data_ptr(), n, k, _ptr(A) if rank else None, _ptr(B) if rank else None, rank,
                            float(s), out.data_ptr(), _stream(stream)), "lbq_unmerge_lora")
    return out


# --------------------------------------------------------------------------- 8-bit linear layers
def _dtype_code(t, name):
    torch = _torch()
    code = {torch.float32: LBQ_F32, torch.bfloat16: LBQ_BF16, torch.float16: LBQ_F16}.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be fp32, bf16 or fp16, not {t.dtype}")
    return code


def _same_device(dev, **tensors):
    """The library launches on the current device, so every tensor of a call has to live there."""
    torch = _torch()
    if dev.type != "cuda" or dev.index != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {dev}, not on the current CUDA device")
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, not on {dev}")


def _out(t, shape, dtype, name, like):
    """A caller's output, checked, or a new one."""
    torch = _torch()
    if t is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")
    return t


def quantize_i8(X, codes=None, scale=None, stream=None):
    """(codes int8 [rows, k], scale fp32 [rows]): the rows of X (fp32, bf16 or fp16) quantized to 8 bits with
    one symmetric scale per row (lbq_quantize_i8)."""
    torch = _torch()
    if X.dim() != 2 or not X.is_cuda or not X.is_contiguous():
        raise ValueError("X must be a contiguous 2-D CUDA tensor")
    code = _dtype_code(X, "X")
    rows, k = X.shape
    with _on(stream):
        codes = _out(codes, (rows, k), torch.int8, "codes", X)
        scale = _out(scale, (rows,), torch.float32, "scale", X)
        _same_device(X.device, codes=codes, scale=scale)
        _check(lbq_quantize_i8(X.data_ptr(), code, rows, k, codes.data_ptr(), scale.data_ptr(), _stream(None)),
               "lbq_quantize_i8")
    return codes, scale


class Int8Weight:
    """A frozen weight [n, k] in 8-bit integers: codes int8 [n, k] and one fp32 scale per output channel, with
    their `lbq_i8weight` view.  Fill it with `quantize`, or pass codes and scale that are there already."""

    def __init__(self, n: int, k: int, codes=None, scale=None, device="cuda"):
        torch = _torch()
        self.n, self.k = int(n), int(k)
        if (codes is None) != (scale is None):
            raise ValueError("codes and scale come together")
        if codes is None:
            codes = torch.empty((n, k), dtype=torch.int8, device=device)
            scale = torch.empty(n, dtype=torch.float32, device=device)
        self.codes = _out(codes, (self.n, self.k), torch.int8, "codes", codes)
        self.scale = _out(scale, (self.n,), torch.float32, "scale", scale)
        if self.codes.device != self.scale.device or not self.codes.is_cuda:
            raise ValueError("codes and scale must be on one CUDA device")
        self.device_index = self.codes.get_device()
        self.struct = lbq_i8weight(n=self.n, k=self.k, codes=self.codes.data_ptr(), scale=self.scale.data_ptr())
        self._ref = ctypes.byref(self.struct)

    def quantize(self, W, stream=None) -> "Int8Weight":
        if tuple(W.shape) != (self.n, self.k):
            raise ValueError(f"W must have shape {(self.n, self.k)}")
        quantize_i8(W, self.codes, self.scale, stream=stream)
        return self

    def dequantize(self):
        """fp32 [n, k]: codes times scale."""
        return self.codes.float() * self.scale[:, None]


def linear_i8_fwd_workspace(m: int, qw: Int8Weight, rank: int = 0):
    """A workspace tensor for linear_i8_fwd with m tokens (any contents; not shared by calls that may overlap)."""
    torch = _torch()
    return torch.empty(lbq_linear_i8_fwd_workspace_size(m, qw._ref, rank), dtype=torch.uint8, device=qw.codes.device)


def linear_i8_bwd_workspace(m: int, qw: Int8Weight, rank: int = 0):
    """A workspace tensor for linear_i8_bwd with m tokens (any contents; not shared by calls that may overlap)."""
    torch = _torch()
    return torch.empty(lbq_linear_i8_bwd_workspace_size(m, qw._ref, rank), dtype=torch.uint8, device=qw.codes.device)


def _f32_out(t, m, n, name, like):
    """An fp32 [m, n] output of the caller, checked, or a new one."""
    torch = _torch()
    if t is None:
        return torch.empty((m, n), dtype=torch.float32, device=like.device)
    if t.dtype is not torch.float32 or t.shape != (m, n) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous fp32 tensor of shape {(m, n)}")
    return t


def _linear_i8(call, what, space, x, name, width_in, width_out, qw, A, B, s, out, out_name, saved, saved_name,
               workspace, stream):
    if stream is not None:
        with _on(stream):
            return _linear_i8(call, what, space, x, name, width_in, width_out, qw, A, B, s, out, out_name, saved,
                              saved_name, workspace, None)
    torch = _torch()
    dev, bf16 = qw.device_index, torch.bfloat16
    if x.dtype is not bf16 or x.dim() != 2 or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-D bf16 CUDA tensor")
    m, width = x.shape
    if width != width_in:
        raise ValueError(f"{name} must have {width_in} columns")
    out = _f32_out(out, m, width_out, out_name, x)
    a = b = t = None
    rank = 0
    if A is None and B is None:
        saved = None
    elif A is None or B is None:
        raise ValueError("A and B come together")
    else:
        rank = A.shape[0]
        if A.dtype is not bf16 or B.dtype is not bf16 or A.shape != (rank, qw.k) or B.shape != (qw.n, rank) or \
                not A.is_contiguous() or not B.is_contiguous():
            raise ValueError(f"A must be contiguous bf16 [rank, {qw.k}] and B [{qw.n}, rank]")
        saved = _f32_out(saved, m, rank, saved_name, x)
        if A.get_device() != dev or B.get_device() != dev or saved.get_device() != dev:
            raise ValueError(f"A, B and {saved_name} must be on the weight's device")
        a, b, t = A.data_ptr(), B.data_ptr(), saved.data_ptr()
    if workspace is None:
        workspace = space(m, qw, rank)
    if x.get_device() != dev or out.get_device() != dev or workspace.get_device() != dev:
        raise ValueError(f"{name}, {out_name} and the workspace must be on the weight's device")
    # the library launches on the current device
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"the tensors are on cuda:{dev}, not on the current CUDA device")
    st = torch._C._cuda_getCurrentRawStream(dev)
    rc = call(x.data_ptr(), m, qw._ref, a, b, rank, s, out.data_ptr(), t, workspace.data_ptr(), workspace.nbytes, st)
    if rc != LBQ_OK:
        raise LbqError(rc, what)
    return out, saved


def linear_i8_fwd(X, qw: Int8Weight, A=None, B=None, s: float = 0.0, Y=None, T=None, workspace=None, stream=None):
    """Y = (Xq Wq^T) sx sw + s (X A^T) B^T with the tokens of X (bf16 [m, k]) quantized to 8 bits in the call;
    returns (Y fp32 [m, n], T = X A^T fp32 [m, rank] or None)."""
    return _linear_i8(lbq_linear_i8_fwd, "lbq_linear_i8_fwd", linear_i8_fwd_workspace, X, "X", qw.k, qw.n, qw, A, B, s,
                      Y, "Y", T, "T", workspace, stream)


def linear_i8_bwd(dY, qw: Int8Weight, A=None, B=None, s: float = 0.0, dX=None, U=None, workspace=None, stream=None):
    """dX = (Vq Wq) sv + s (dY B) A with V = dY times the channel scales, its tokens quantized to 8 bits in the
    call; returns (dX fp32 [m, k], U = dY B fp32 [m, rank] or None)."""
    return _linear_i8(lbq_linear_i8_bwd, "lbq_linear_i8_bwd", linear_i8_bwd_workspace, dY, "dY", qw.n, qw.k, qw, A, B,
                      s, dX, "dX", U, "U", workspace, stream)


# --------------------------------------------------------------------------- gradient norm and clipping
class GradClip:
    """The norm and the clipping of one list of gradients, step after step: keeps the list's table, the norm and
    the workspace.  `grads` are contiguous fp32, bf16 or fp16 CUDA tensors; `outs` (default: the gradients
    themselves) get the scaled copies, with the same types and sizes.  The tensors are held, so their memory
    stays theirs; calls of one GradClip that may run at the same time race on its workspace, which is zeroed on
    the stream that is current here: the first call on another stream waits for that.  (Not a call that is being
    captured, which cannot wait for work outside its graph: `torch.cuda.graph` waits for the device when it begins,
    and so has to whoever begins a capture by hand before the workspace is zeroed.  A plan made inside a capture is
    that graph's alone.)"""

    def __init__(self, grads, outs=None, *, _one_call=False):
        torch = _torch()
        self.grads = list(grads)
        self.outs = self.grads if outs is None else list(outs)
        if not self.grads:
            raise ValueError("no gradients")
        if len(self.outs) != len(self.grads):
            raise ValueError("one output for each gradient")
        dev = self.grads[0].device
        self.table = (lbq_grad * len(self.grads))()
        for i, (g, o) in enumerate(zip(self.grads, self.outs)):
            if not g.is_contiguous() or not o.is_contiguous():
                raise ValueError(f"gradient {i} and its output must be contiguous")
            if o.dtype != g.dtype or o.numel() != g.numel():
                raise ValueError(f"output {i} must have its gradient's type and size")
            if g.device != dev or o.device != dev:
                raise ValueError(f"gradient {i} and its output must be on {dev}")
            self.table[i] = lbq_grad(g=g.data_ptr(), out=o.data_ptr(), numel=g.numel(),
                                     dtype=_dtype_code(g, f"gradient {i}"), reserved=0)
        if dev.type != "cuda":
            raise ValueError("the gradients must be CUDA tensors")
        self.total_norm = torch.empty(1, dtype=torch.float32, device=dev)
        self.workspace = torch.zeros(lbq_grad_norm_workspace_size(len(self.grads)), dtype=torch.uint8, device=dev)
        # streams whose work comes after the zero fill, and what others wait for (an event takes 6 us: not where the
        # only call follows here)
        self._ordered = {torch._C._cuda_getCurrentRawStream(dev.index)}
        self._zeroed = None
        if not _one_call and not torch.cuda.is_current_stream_capturing():
            self._zeroed = torch.cuda.current_stream(dev).record_event()

    def _order(self, stream):
        """Puts a stream's work after the workspace's zero fill, which another stream was given."""
        torch = _torch()
        if stream is None:
            stream = torch.cuda.current_stream(self.total_norm.device)
        with torch.cuda.stream(stream):
            if self._zeroed is None or torch.cuda.is_current_stream_capturing():
                return
            stream.wait_event(self._zeroed)
            for t in (self.total_norm, self.workspace):      # their memory is not reused before this stream is done
                t.record_stream(stream)
        self._ordered.add(stream.cuda_stream)

    def norm(self, stream=None):
        """The Euclidean norm of all gradients together (fp32 [1], on the device)."""
        _same_device(self.total_norm.device)
        st = _stream(stream)
        if st not in self._ordered:
            self._order(stream)
        _check(lbq_grad_norm(self.table, len(self.grads), self.total_norm.data_ptr(), self.workspace.data_ptr(),
                             self.workspace.numel(), st), "lbq_grad_norm")
        return self.total_norm

    def clip(self, max_norm: float, stream=None):
        """Scale the gradients by min(1, max_norm / (norm + 1e-6)); returns their norm before."""
        torch = _torch()
        dev = self.total_norm.get_device()
        if dev != torch._C._cuda_getDevice():
            raise ValueError(f"the gradients are on cuda:{dev}, not on the current CUDA device")
        st = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
        if st not in self._ordered:
            self._order(stream)
        _check(lbq_clip_grad_norm(self.table, len(self.grads), max_norm, self.total_norm.data_ptr(),
                                  self.workspace.data_ptr(), self.workspace.nbytes, st), "lbq_clip_grad_norm")
        return self.total_norm


def grad_norm(grads, stream=None):
    """The Euclidean norm of all `grads` together (fp32 [1], on the device)."""
    with _on(stream):
        return GradClip(grads, _one_call=True).norm()


def clip_grad_norm(grads, max_norm: float, outs=None, stream=None):
    """Clip `grads` to max_norm, in place or into `outs`; returns their norm before (fp32 [1], on the device)."""
    with _on(stream):
        return GradClip(grads, outs, _one_call=True).clip(max_norm)


def device_status() -> int:
    """The device status word (timeouts, bad codebooks) since the last read."""
    v = ctypes.c_uint32(0)
    _check(lbq_device_status(ctypes.byref(v)), "lbq_device_status")
    return int(v.value)
