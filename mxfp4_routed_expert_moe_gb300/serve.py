"""The operators around the layer in a serving step (``include/moe_serve.h``): new keys and values into
a paged cache with rotary positions on the way, attention of a batch that shares a prefix over that cache,
and sampling from logits.  Argument marshalling only, as in the package itself.

What a kernel finds wrong in the values of its arguments (a page id, length or position out of range, a wait
that gave up) it can only write down: pass ``status``, a GPU int32 word, and read it when the results matter.
Without one such a call leaves unspecified outputs and no sign."""
from __future__ import annotations

import ctypes

from . import DT_BF16, DT_F32, MoeError, _check, lib

__all__ = ["KVCache", "KVBatch", "kv_append", "prefix_attention", "attention_workspace_bytes", "sample",
           "rope_table", "SERVE_EXPORTS", "SAMPLE_MAX_VOCAB", "SERVE_MAX_BATCH",
           "SERVE_MAX_LEN"]

# Every symbol moe_serve.h declares (checked by the tests against the .so).
SERVE_EXPORTS = ("moe_kv_append", "moe_attention_workspace_bytes", "moe_prefix_attention", "moe_sample")
SAMPLE_MAX_VOCAB = 1 << 18   # MOE_SAMPLE_MAX_VOCAB
SERVE_MAX_BATCH = 4096       # MOE_SERVE_MAX_BATCH
SERVE_MAX_LEN = 1 << 30      # MOE_SERVE_MAX_LEN


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class _Batch(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("tokens", ctypes.c_int32), ("max_q", ctypes.c_int32),
                ("table_stride", ctypes.c_int32), ("table_pages", ctypes.c_int32), ("prefix_len", ctypes.c_int32),
                ("q_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("prefix_table", ctypes.c_void_p)]


_READY = _TYPES = None
torch = None  # imported with the library: a build needs neither


def _lib():
    """The loaded library with the argument types of this module's calls."""
    global _READY, torch, _TYPES
    if _READY is None:
        import torch as _torch
        L = lib()
        vp, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
        P = ctypes.POINTER
        L.moe_kv_append.argtypes = [P(_Cache), P(_Batch), i32, vp, vp, vp, i32, i64, i64, i64, vp, i64, vp, i32, i32,
                                    i32, vp, vp]
        L.moe_attention_workspace_bytes.restype = sz
        L.moe_attention_workspace_bytes.argtypes = [P(_Cache), P(_Batch), i32]
        L.moe_prefix_attention.argtypes = [P(_Cache), P(_Batch), vp, i32, i64, f32, vp, i64, vp, vp, sz, vp, vp]
        L.moe_sample.argtypes = [i32, i32, vp, i32, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        torch = _torch
        _TYPES = {torch.float32: DT_F32, torch.bfloat16: DT_BF16}
        _READY = L
    return _READY


def _stream(stream, t):
    """The raw stream: the given one, or the current one of the tensor's device."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(t.get_device())
    return stream if isinstance(stream, int) else stream.cuda_stream


def _dtype_of(t, what):
    dt = _TYPES.get(t.dtype)
    if dt is None:
        raise TypeError(f"{what} must be torch.float32 or torch.bfloat16, not {t.dtype}")
    return dt


def _want(t, what, dtype, shape=None):
    """Address of a tensor argument, after checks of its type, shape (None: any) and contiguity."""
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _same_gpu(device, tensors):
    """Every (tensor or None, name) has to be on the GPU ``device``: the kernels would follow a host address."""
    if device < 0:
        raise ValueError("the tensors of a call must be on a GPU")
    for t, what in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"{what} must be on GPU {device}, as the others")


def _status(status, device):
    """Address of a status word: None, an address, or a GPU int32 tensor."""
    if status is None or isinstance(status, int):
        return status
    if status.dtype is not torch.int32 or status.numel() < 1:
        raise TypeError("status must be a torch.int32 word")
    _same_gpu(device, ((status, "status"),))
    return status.data_ptr()


class KVCache:
    """A paged cache over two bf16 tensors [num_pages][page_size][kv_heads][head_dim].  Views of another
    order (head-major pages, one tensor that holds both) are taken as they are, by their strides."""

    def __init__(self, k, v):
        _lib()
        for t, what in ((k, "k"), (v, "v")):
            if t.dtype is not torch.bfloat16:
                raise TypeError(f"the cache's {what} must be torch.bfloat16, not {t.dtype}")
            if t.dim() != 4 or t.stride(3) != 1:
                raise ValueError(f"the cache's {what} must be [pages][page_size][kv_heads][head_dim], contiguous in the last")
        if k.shape != v.shape or k.stride() != v.stride():
            raise ValueError("k and v of a cache must have the same shape and strides")
        self.k, self.v = k, v
        pages, size, heads, dim = k.shape
        self.struct = _Cache(k.data_ptr(), v.data_ptr(), pages, size, heads, dim, *k.stride()[:3])
        self.ref = ctypes.byref(self.struct)
        self.heads, self.dim = heads, dim
        self.device = k.get_device()
        if v.get_device() != self.device:
            raise ValueError("k and v of a cache must be on one device")


class KVBatch:
    """A batch of sequences over one cache: their lengths and page tables on the device, and the prefix
    that all of them share.

    ``kv_len`` [B] int32: tokens of each sequence's own part, the new ones included; ``table`` [B][pages]
    int32: their pages; ``q_start`` [B + 1] int32: first row of each sequence among the ``tokens`` new ones
    (None: one token each), at most ``max_q`` a sequence; ``prefix_table`` int32: the pages of the first
    ``prefix_len`` tokens that every sequence sees before its own.  The tensors are kept and may be updated
    in place between calls."""

    def __init__(self, kv_len, table, tokens=None, q_start=None, max_q=1, prefix_table=None, prefix_len=0):
        _lib()
        B = kv_len.shape[0]
        if table.dim() != 2 or table.shape[0] != B or (table.shape[1] > 1 and table.stride(1) != 1):
            raise ValueError("table must be [batch][pages], contiguous in the last")
        if table.dtype is not torch.int32:
            raise TypeError(f"table must be torch.int32, not {table.dtype}")
        if prefix_len > 0 and (prefix_table is None or prefix_table.numel() < 1):
            raise ValueError("a prefix needs its page table")
        stride = table.stride(0) if B > 1 else max(table.stride(0), table.shape[1])
        self.kv_len, self.table, self.q_start, self.prefix_table = kv_len, table, q_start, prefix_table
        self.struct = _Batch(B, B if tokens is None else tokens, max_q, stride, table.shape[1], prefix_len,
                             None if q_start is None else _want(q_start, "q_start", torch.int32, (B + 1,)),
                             _want(kv_len, "kv_len", torch.int32, (B,)), table.data_ptr(),
                             None if prefix_table is None else _want(prefix_table, "prefix_table", torch.int32))
        self.prefix_tokens = 0 if prefix_table is None else prefix_table.numel()
        self.ref = ctypes.byref(self.struct)
        self.tokens = self.struct.tokens
        self.device = kv_len.get_device()
        for t in (table, q_start, prefix_table):
            if t is not None and t.get_device() != self.device:
                raise ValueError("the tensors of a batch must be on one device")

    def get_device(self):
        return self.device

    def check_prefix(self, cache):
        if self.struct.prefix_len > self.prefix_tokens * cache.struct.page_size:
            raise ValueError("prefix_len is more than the prefix's pages hold")


def _rows(x, what, tokens, heads, dim):
    """[tokens][heads][dim] with the heads of a token side by side: the stride between tokens."""
    if x.shape != (tokens, heads, dim):
        raise ValueError(f"{what} must have shape {(tokens, heads, dim)}, not {tuple(x.shape)}")
    row, head, one = x.stride()
    if one != 1 or (heads > 1 and head != dim):
        raise ValueError(f"{what}: the heads of a token must be contiguous")
    return row if tokens > 1 else heads * dim


def rope_table(positions: int, rot_dim: int, base: float = 10000.0, device="cuda"):
    """Cosines and sines of positions 0 .. positions - 1 for :func:`kv_append`: fp32 [positions][rot_dim],
    the rot_dim / 2 cosines of angles position * base^(-2i / rot_dim), then the sines (computed in fp64:
    an angle of a long context has too few bits in fp32)."""
    import torch
    inv = float(base) ** (-torch.arange(0, rot_dim, 2, device=device, dtype=torch.float64) / rot_dim)
    a = torch.arange(positions, device=device, dtype=torch.float64)[:, None] * inv
    return torch.cat((a.cos(), a.sin()), 1).float()


def kv_append(cache: KVCache, batch: KVBatch, k, v, q=None, q_out=None, rope=None, rot_dim=0, interleaved=False,
              status=None, stream=None):
    """moe_kv_append: k, v [tokens][kv_heads][dim] (fp32 or bf16, any token stride) into the cache at each
    token's place, with the first ``rot_dim`` values of each key head, and of the queries q -> q_out, rotated
    by the rows of ``rope`` (see :func:`rope_table`)."""
    n, dim = batch.tokens, cache.dim
    ks, vs = _rows(k, "k", n, cache.heads, dim), _rows(v, "v", n, cache.heads, dim)
    dt = _dtype_of(k, "k")
    if v.dtype is not k.dtype or (q is not None and q.dtype is not k.dtype):
        raise TypeError("q, k and v must have one type")
    qh = qs = os = rows = 0
    qp = op = rp = None
    if q is not None:
        qh = q.shape[1]
        qs = _rows(q, "q", n, qh, dim)
        qp = q.data_ptr()
    if q_out is not None:
        if q_out.dtype is not torch.bfloat16:
            raise TypeError(f"q_out must be torch.bfloat16, not {q_out.dtype}")
        os = _rows(q_out, "q_out", n, qh, dim)
        op = q_out.data_ptr()
    if rope is not None:
        rows = rope.shape[0]
        rp = _want(rope, "rope", torch.float32, (rows, rot_dim))
    sp = _status(status, cache.device)
    gpu = cache.device
    # One expression where all is well: a list of names each time would be a tenth of the call.
    if not (batch.device == gpu == k.get_device() == v.get_device() and gpu >= 0 and (q is None or q.get_device() == gpu)
            and (q_out is None or q_out.get_device() == gpu) and (rope is None or rope.get_device() == gpu)):
        _same_gpu(gpu, ((batch, "the batch"), (k, "k"), (v, "v"), (q, "q"), (q_out, "q_out"), (rope, "rope")))
    _check(_READY.moe_kv_append(cache.ref, batch.ref, dt, qp, k.data_ptr(), v.data_ptr(), qh, qs, ks, vs, op, os, rp, rows,
                                rot_dim, bool(interleaved), sp, _stream(stream, k)), "moe_kv_append")


def attention_workspace_bytes(cache: KVCache, batch: KVBatch, q_heads: int) -> int:
    """moe_attention_workspace_bytes; raises MoeError where moe_prefix_attention would refuse the arguments."""
    n = int(_READY.moe_attention_workspace_bytes(cache.ref, batch.ref, int(q_heads)))
    if n == 0:
        raise MoeError(1, "moe_attention_workspace_bytes")
    return n


def prefix_attention(cache: KVCache, batch: KVBatch, q, out, ws, scale=None, lse=None, status=None, stream=None):
    """moe_prefix_attention: q, out bf16 [tokens][q_heads][dim] (any token stride); ``scale`` defaults to
    dim^-1/2; ``lse`` is None or fp32 [tokens][q_heads]; ``ws`` a uint8 tensor of at least
    :func:`attention_workspace_bytes`."""
    n, dim = batch.tokens, cache.dim
    qh = q.shape[1]
    qs, os = _rows(q, "q", n, qh, dim), _rows(out, "out", n, qh, dim)
    if q.dtype is not torch.bfloat16 or out.dtype is not torch.bfloat16:
        raise TypeError(f"q and out must be torch.bfloat16, not {q.dtype} and {out.dtype}")
    batch.check_prefix(cache)
    lp = None if lse is None else _want(lse, "lse", torch.float32, (n, qh))
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    sp = _status(status, cache.device)
    gpu = cache.device
    if not (batch.device == gpu == q.get_device() == out.get_device() == ws.get_device() and gpu >= 0
            and (lse is None or lse.get_device() == gpu)):
        _same_gpu(gpu, ((batch, "the batch"), (q, "q"), (out, "out"), (ws, "ws"), (lse, "lse")))
    _check(_READY.moe_prefix_attention(cache.ref, batch.ref, q.data_ptr(), qh, qs, dim ** -0.5 if scale is None else scale,
                                       out.data_ptr(), os, lp, ws.data_ptr(), ws.nbytes, sp,
                                       _stream(stream, q)), "moe_prefix_attention")


def sample(logits, u, token, temperature=None, top_k=None, top_p=None, min_p=None, logprob=None, kept=None,
           probs=None, stream=None):
    """moe_sample: one token per row of ``logits`` [rows][vocab] (fp32 or bf16, any row stride) into ``token``
    [rows] int32, drawn by ``u`` [rows] in [0, 1).  ``temperature``, ``top_p``, ``min_p`` (fp32) and ``top_k``
    (int32) are [rows] device tensors or None; ``logprob`` [rows] fp32, ``kept`` [rows] int32 and ``probs``
    [rows][vocab] fp32 receive the token's log-probability, the number of tokens kept and their
    probabilities."""
    L = _lib()
    rows, vocab = logits.shape
    stride, one = logits.stride()
    if vocab > 1 and one != 1:
        raise ValueError("logits must be contiguous in the last dimension")
    f32, i32, row = torch.float32, torch.int32, (rows,)
    args = (rows, vocab, logits.data_ptr(), _dtype_of(logits, "logits"), stride if rows > 1 else vocab,
            _want(u, "u", f32, row),
            None if temperature is None else _want(temperature, "temperature", f32, row),
            None if top_k is None else _want(top_k, "top_k", i32, row),
            None if top_p is None else _want(top_p, "top_p", f32, row),
            None if min_p is None else _want(min_p, "min_p", f32, row), _want(token, "token", i32, row),
            None if logprob is None else _want(logprob, "logprob", f32, row),
            None if kept is None else _want(kept, "kept", i32, row),
            None if probs is None else _want(probs, "probs", f32, (rows, vocab)))
    gpu = logits.get_device()
    if not (gpu == u.get_device() == token.get_device() and gpu >= 0
            and (temperature is None or temperature.get_device() == gpu) and (top_k is None or top_k.get_device() == gpu)
            and (top_p is None or top_p.get_device() == gpu) and (min_p is None or min_p.get_device() == gpu)
            and (logprob is None or logprob.get_device() == gpu) and (kept is None or kept.get_device() == gpu)
            and (probs is None or probs.get_device() == gpu)):
        _same_gpu(gpu, ((u, "u"), (token, "token"), (temperature, "temperature"), (top_k, "top_k"), (top_p, "top_p"),
                        (min_p, "min_p"), (logprob, "logprob"), (kept, "kept"), (probs, "probs")))
    _check(L.moe_sample(*args, _stream(stream, logits)), "moe_sample")
