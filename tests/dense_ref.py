"""Plain 64-bit forms of the operators of moe_dense.h, in numpy."""
from __future__ import annotations

import numpy as np

from serve_ref import torch  # noqa: F401

EMAX = {"e2m1": 2, "e4m3": 8}
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)


def _e4m3():
    v = [m * 2.0 ** -9 for m in range(8)]
    v += [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return np.array(v[:127], dtype=np.float64)  # code 127 is NaN


E4M3 = _e4m3()
GRID = {"e2m1": E2M1, "e4m3": E4M3}


def nearest(a, kind):
    """Codes of magnitudes: the nearest value of the type, ties to the even code, saturating."""
    g = GRID[kind]
    mid = (g[1:] + g[:-1]) / 2
    lo = np.searchsorted(mid, a, side="left")   # a tie goes down
    hi = np.searchsorted(mid, a, side="right")  # a tie goes up
    return np.where(lo % 2 == 0, lo, hi)


def quantize(x, kind):
    """fp64 values [r][c] -> codes [r][c] (sign in the top bit of 4 or 8) and scales uint8 [r][c / 32]."""
    r, c = x.shape
    b = x.reshape(r, c // 32, 32)
    with np.errstate(invalid="ignore"):
        most = np.abs(b).max(-1)
    bad = ~np.isfinite(b).all(-1)
    m = np.where(bad | (most == 0), 1.0, most)
    e = np.frexp(m)[1] - 1 - EMAX[kind]
    e = np.where(most == 0, -127, np.maximum(e, -127))
    s = np.where(bad, 255, e + 127).astype(np.uint8)
    a = np.where(bad[..., None], 0.0, b)
    code = nearest(np.abs(np.ldexp(a, -e[..., None])), kind)
    code = code + np.where(np.signbit(a), 8 if kind == "e2m1" else 128, 0)
    return code.astype(np.uint8).reshape(r, c), s


def pack(code, kind):
    return code if kind == "e4m3" else (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)


def unpack(q, kind):
    if kind == "e4m3":
        return q
    out = np.empty((q.shape[0], q.shape[1] * 2), dtype=np.uint8)
    out[:, 0::2], out[:, 1::2] = q & 15, q >> 4
    return out


def values(code, s, kind):
    """What codes [r][c] and scales stand for, fp64."""
    top = 8 if kind == "e2m1" else 128
    g = np.concatenate((GRID[kind], [np.nan])) if kind == "e4m3" else GRID[kind]
    v = g[code % top] * np.where(code >= top, -1.0, 1.0)
    scale = np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(np.int64) - 127))
    return v * np.repeat(scale, 32, axis=1)


def random_mx(rng, rows, cols, kind, spread=3, scales=None):
    """Random codes without NaN, scales within `spread` powers of two around 1: codes, scales."""
    if kind == "e2m1":
        code = rng.integers(0, 16, (rows, cols), dtype=np.uint8)
    else:
        code = rng.integers(0, 127, (rows, cols)).astype(np.uint8) | (rng.integers(0, 2, (rows, cols)).astype(np.uint8) << 7)
    s = rng.integers(127 - spread, 128 + spread, (rows, cols // 32)).astype(np.uint8) if scales is None else scales
    return code, s


def matrix(moe, code, s, kind, pad=0):
    """An MXMatrix on the GPU; pad > 0: rows `pad` x 32 bytes (codes) and `pad` x 4 bytes (scales) longer, the gaps full of NaN."""
    t = torch()
    q = pack(code, kind)
    qt = t.full((q.shape[0], q.shape[1] + 32 * pad), 0xFF, dtype=t.uint8, device="cuda")
    st = t.full((s.shape[0], s.shape[1] + 4 * pad), 0xFF, dtype=t.uint8, device="cuda")
    qv, sv = qt[:, :q.shape[1]], st[:, :s.shape[1]]
    qv.copy_(t.from_numpy(q))
    sv.copy_(t.from_numpy(s))
    return moe.MXMatrix(qv, sv, kind)


def host(t):
    return t.double().cpu().numpy()
