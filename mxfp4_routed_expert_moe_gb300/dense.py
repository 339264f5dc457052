"""The dense half of a serving step around the layer (``include/moe_dense.h``): residual norm, MX matrices (MXFP4,
MXFP8) and their product, log probabilities of given tokens.  Argument marshalling only, as in the package
itself."""
from __future__ import annotations

import ctypes

from . import DT_BF16, DT_F32, MoeError, _check, lib
from . import serve
from .serve import _same_gpu, _status, _stream

__all__ = ["MXMatrix", "mx_quantize", "mx_dequantize", "mx_linear", "rms_norm", "token_logprobs", "DENSE_EXPORTS",
           "DENSE_MAX_COLS", "DENSE_MAX_STRIDE", "MX_MAX_VALUES", "LINEAR_MAX_ROWS", "LINEAR_MAX_OUTS", "LOGPROBS_MAX_ROWS",
           "LOGPROBS_MAX_VOCAB", "LOGPROBS_MAX_TOP"]

# Every symbol moe_dense.h declares (checked by the tests against the .so).
DENSE_EXPORTS = ("moe_mx_quantize", "moe_mx_dequantize", "moe_rms_norm", "moe_mx_linear", "moe_token_logprobs")
DENSE_MAX_COLS = 16384          # MOE_DENSE_MAX_COLS
DENSE_MAX_STRIDE = 1 << 38      # MOE_DENSE_MAX_STRIDE
MX_MAX_VALUES = 34359730144     # MOE_MX_MAX_VALUES
LINEAR_MAX_ROWS = 65536         # MOE_LINEAR_MAX_ROWS
LINEAR_MAX_OUTS = 262144        # MOE_LINEAR_MAX_OUTS
LOGPROBS_MAX_ROWS = 16777216    # MOE_LOGPROBS_MAX_ROWS
LOGPROBS_MAX_VOCAB = 262144     # MOE_LOGPROBS_MAX_VOCAB
LOGPROBS_MAX_TOP = 32           # MOE_LOGPROBS_MAX_TOP

KINDS = {"e2m1": 0, "e4m3": 1}  # MOE_MX_E2M1, MOE_MX_E4M3


class _Mx(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("s", ctypes.c_void_p), ("type", ctypes.c_int32), ("rows", ctypes.c_int32),
                ("cols", ctypes.c_int32), ("q_stride", ctypes.c_int64), ("s_stride", ctypes.c_int64)]


_READY = _TYPES = None
torch = None  # imported with the library: a build needs neither


def _lib():
    """The loaded library with the argument types of this module's calls."""
    global _READY, torch, _TYPES
    if _READY is None:
        import torch as _torch
        serve._lib()  # the shared checks of arguments
        L = lib()
        vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
        M = ctypes.POINTER(_Mx)
        L.moe_mx_quantize.argtypes = [vp, i32, i64, M, vp]
        L.moe_mx_dequantize.argtypes = [M, vp, i32, i64, vp]
        L.moe_rms_norm.argtypes = [i32, i32, vp, i32, i64, vp, vp, i32, i64, vp, f32, vp, i32, i64, M, vp]
        L.moe_mx_linear.argtypes = [M, M, vp, i64, vp, i32, i64, vp, vp]
        L.moe_token_logprobs.argtypes = [i32, i32, vp, i32, i64, vp, vp, vp, vp, i32, vp, vp, vp]
        torch = _torch
        _TYPES = {torch.float32: DT_F32, torch.bfloat16: DT_BF16}
        _READY = L
    return _READY


class MXMatrix:
    """An MX matrix [rows][cols] over two uint8 tensors: codes ``q`` [rows][cols / 2] (``kind`` "e2m1", MXFP4: element
    2i in the low nibble of byte i) or [rows][cols] ("e4m3", MXFP8), and scales ``s`` [rows][cols / 32], value
    2^(s - 127).  Views with a row stride are taken as they are.  The tensors are kept and may be written between
    calls."""

    def __init__(self, q, s, kind="e2m1"):
        _lib()
        if kind not in KINDS:
            raise ValueError(f"kind must be one of {tuple(KINDS)}, not {kind!r}")
        for t, what in ((q, "q"), (s, "s")):
            if t.dtype is not torch.uint8:
                raise TypeError(f"{what} must be torch.uint8, not {t.dtype}")
            if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
                raise ValueError(f"{what} must have two dimensions, contiguous in the last")
        rows, cols = q.shape[0], q.shape[1] * (2 if kind == "e2m1" else 1)
        if cols % 32 or s.shape != (rows, cols // 32):
            raise ValueError(f"codes of [{rows}][{cols}] need cols a multiple of 32 and scales [rows][cols / 32], not {tuple(s.shape)}")
        if q.get_device() != s.get_device():
            raise ValueError("q and s of an MX matrix must be on one device")
        self.q, self.s, self.kind, self.rows, self.cols, self.shape = q, s, kind, rows, cols, (rows, cols)
        # One row has any stride.
        qs, ss = (q.stride(0), s.stride(0)) if rows > 1 else (q.shape[1] + -q.shape[1] % 32, cols // 32 + -(cols // 32) % 4)
        self.struct = _Mx(q.data_ptr(), s.data_ptr(), KINDS[kind], rows, cols, qs, ss)
        self.ref = ctypes.byref(self.struct)
        self.device = q.get_device()

    @classmethod
    def empty(cls, rows, cols, kind="e2m1", device="cuda"):
        """An uninitialised matrix with contiguous rows."""
        import torch
        if kind not in KINDS:
            raise ValueError(f"kind must be one of {tuple(KINDS)}, not {kind!r}")
        if cols % 32:
            raise ValueError("cols must be a multiple of 32")
        return cls(torch.empty(rows, cols if kind == "e4m3" else cols // 2, dtype=torch.uint8, device=device),
                   torch.empty(rows, cols // 32, dtype=torch.uint8, device=device), kind)

    def get_device(self):
        return self.device


def _mx(a, what):
    if not isinstance(a, MXMatrix):
        raise TypeError(f"{what} must be an MXMatrix")
    return a


def _matrix(x, what, shape):
    """[rows][cols] of fp32 or bf16, contiguous in the last: its type and the stride between rows."""
    dt = _TYPES.get(x.dtype)
    if dt is None:
        raise TypeError(f"{what} must be torch.float32 or torch.bfloat16, not {x.dtype}")
    if x.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, not {tuple(x.shape)}")
    if x.is_contiguous():
        return dt, shape[1]
    row, one = x.stride()
    if one != 1 and shape[1] > 1:
        raise ValueError(f"{what} must be contiguous in the last dimension")
    return dt, row if shape[0] > 1 else shape[1]


def mx_quantize(x, out: MXMatrix, stream=None):
    """moe_mx_quantize: x [rows][cols] (fp32 or bf16, any row stride that is a multiple of 16 bytes) into ``out``."""
    _mx(out, "out")
    dt, xs = _matrix(x, "x", out.shape)
    if not (x.get_device() == out.device >= 0):
        _same_gpu(out.device, ((x, "x"),))
    _check(_READY.moe_mx_quantize(x.data_ptr(), dt, xs, out.ref, _stream(stream, x)), "moe_mx_quantize")


def mx_dequantize(x: MXMatrix, out, stream=None):
    """moe_mx_dequantize: what ``x`` stands for into ``out`` [rows][cols] (fp32 or bf16)."""
    _mx(x, "x")
    dt, os = _matrix(out, "out", x.shape)
    if not (out.get_device() == x.device >= 0):
        _same_gpu(x.device, ((out, "out"),))
    _check(_READY.moe_mx_dequantize(x.ref, out.data_ptr(), dt, os, _stream(stream, out)), "moe_mx_dequantize")


def rms_norm(x, out, weight=None, residual=None, residual_out=None, eps=1e-6, stream=None):
    """moe_rms_norm: ``out`` (a tensor [rows][cols] or an :class:`MXMatrix`) receives the norm of x + residual times
    ``weight`` ([cols] fp32 or None); ``residual_out`` (with a residual; may be the residual itself) the sum."""
    L = _lib()
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x must be [rows][cols]")
    dt, xs = _matrix(x, "x", shape)
    gpu = x.get_device()
    fine = gpu >= 0
    rp = rop = wp = op = mp = None
    rdt = rs = odt = os = 0
    if residual is not None:
        if residual_out is None:
            raise ValueError("a residual needs residual_out (it may be the residual)")
        rdt, rs = _matrix(residual, "residual", shape)
        rp = rop = residual.data_ptr()
        fine = fine and residual.get_device() == gpu
        if residual_out is not residual:
            if _matrix(residual_out, "residual_out", shape) != (rdt, rs):
                raise ValueError("residual_out must have the type and strides of residual")
            rop = residual_out.data_ptr()
            fine = fine and residual_out.get_device() == gpu
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    if weight is not None:
        if weight.dtype is not torch.float32 or weight.dim() != 1 or weight.shape[0] != shape[1] or not weight.is_contiguous():
            raise ValueError(f"weight must be a contiguous torch.float32 [{shape[1]}]")
        wp = weight.data_ptr()
        fine = fine and weight.get_device() == gpu
    if isinstance(out, MXMatrix):
        if out.shape != shape:
            raise ValueError(f"out must have shape {tuple(shape)}, not {out.shape}")
        mp = out.ref
    else:
        odt, os = _matrix(out, "out", shape)
        op = out.data_ptr()
    if not (fine and out.get_device() == gpu):
        _same_gpu(gpu, ((out, "out"), (residual, "residual"), (residual_out, "residual_out"), (weight, "weight")))
    _check(L.moe_rms_norm(shape[0], shape[1], x.data_ptr(), dt, xs, rp, rop, rdt, rs, wp, eps, op, odt, os, mp,
                          _stream(stream, x)), "moe_rms_norm")


def mx_linear(x: MXMatrix, w: MXMatrix, out, add=None, status=None, stream=None):
    """moe_mx_linear: out [rows of x][rows of w] (fp32 or bf16, any row stride) = x w^T (+ ``add``, of out's type; it may
    be ``out`` itself).  ``w`` is MXFP4 ("e2m1"), x either kind."""
    _mx(x, "x"), _mx(w, "w")
    shape = (x.rows, w.rows)
    if x.cols != w.cols:
        raise ValueError(f"x has rows of {x.cols}, w of {w.cols}")
    dt, os = _matrix(out, "out", shape)
    ap, as_ = None, 0
    if add is not None:
        adt, as_ = _matrix(add, "add", shape)
        if adt != dt:
            raise TypeError("add and out must have one type")
        ap = add.data_ptr()
    gpu = x.device
    if not (gpu == w.device == out.get_device() and gpu >= 0 and (add is None or add.get_device() == gpu)):
        _same_gpu(gpu, ((w, "w"), (out, "out"), (add, "add")))
    _check(_READY.moe_mx_linear(x.ref, w.ref, ap, as_, out.data_ptr(), dt, os, _status(status, gpu), _stream(stream, out)),
           "moe_mx_linear")


def token_logprobs(logits, tokens=None, logprob=None, rank=None, entropy=None, top_ids=None, top_logprobs=None,
                   stream=None):
    """moe_token_logprobs: for rows of ``logits`` [rows][vocab] (fp32 or bf16, any row stride) the log probability of
    ``tokens`` [rows] int32 into ``logprob`` [rows] fp32 and its rank into ``rank`` [rows] int32, the row's entropy
    into ``entropy`` [rows] fp32, and the best alternatives into ``top_ids`` [rows][n] int32 and ``top_logprobs``
    [rows][n] fp32 (n <= LOGPROBS_MAX_TOP).  Any of the outputs may be None."""
    L = _lib()
    if logits.dim() != 2:
        raise ValueError("logits must be [rows][vocab]")
    rows, vocab = logits.shape
    dt = _TYPES.get(logits.dtype)
    if dt is None:
        raise TypeError(f"logits must be torch.float32 or torch.bfloat16, not {logits.dtype}")
    stride, one = logits.stride()
    if vocab > 1 and one != 1:
        raise ValueError("logits must be contiguous in the last dimension")
    top = 0
    if (top_ids is None) != (top_logprobs is None):
        raise ValueError("top_ids and top_logprobs go together")
    if top_ids is not None:
        if top_ids.dim() != 2:
            raise ValueError("top_ids must be [rows][n]")
        top = top_ids.shape[1]
    f32, i32, row = torch.float32, torch.int32, (rows,)
    ptrs = []
    gpu = logits.get_device()
    fine = gpu >= 0
    for t, what, dtype, shape in ((tokens, "tokens", i32, row), (logprob, "logprob", f32, row), (rank, "rank", i32, row),
                                  (entropy, "entropy", f32, row), (top_ids, "top_ids", i32, (rows, top)),
                                  (top_logprobs, "top_logprobs", f32, (rows, top))):
        if t is None:
            ptrs.append(None)
            continue
        if t.dtype is not dtype:
            raise TypeError(f"{what} must be {dtype}, not {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{what} must have shape {shape}, not {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{what} must be contiguous")
        fine = fine and t.get_device() == gpu
        ptrs.append(t.data_ptr())
    if not fine:
        _same_gpu(gpu, ((tokens, "tokens"), (logprob, "logprob"), (rank, "rank"), (entropy, "entropy"), (top_ids, "top_ids"),
                        (top_logprobs, "top_logprobs")))
    _check(L.moe_token_logprobs(rows, vocab, logits.data_ptr(), dt, stride if rows > 1 else vocab, *ptrs[:4], top, *ptrs[4:],
                                _stream(stream, logits)), "moe_token_logprobs")
