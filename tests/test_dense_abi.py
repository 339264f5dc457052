"""moe_dense.h: the library exports what it declares, the binding knows every symbol and limit, and bad arguments are
refused before anything is launched (no GPU needed: these calls return before touching CUDA)."""
import ctypes
import os
import re

import pytest

from conftest import ROOT

HEADER = os.path.join(ROOT, "include", "moe_dense.h")
A = 1 << 20  # a fake, never-dereferenced address
B, C, D, E = A + 4096, A + 8192, A + 12288, A + 16384


@pytest.fixture(scope="module")
def moe():
    import mxfp4_routed_expert_moe_gb300 as m
    import mxfp4_routed_expert_moe_gb300.build as b
    b.build()
    m.lib()
    return m


@pytest.fixture(scope="module")
def dense(moe):
    from mxfp4_routed_expert_moe_gb300 import dense as d
    d._lib()
    return d


def test_header_binding_and_library_agree(moe):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^[A-Za-z_][\w\s\*]*?\b(moe_\w+)\s*\(", src, flags=re.M)))
    assert names == sorted(moe.DENSE_EXPORTS)
    L = ctypes.CDLL(moe.LIB_PATH)
    for name in names:
        assert hasattr(L, name), name
    for name in ("DENSE_MAX_COLS", "LINEAR_MAX_ROWS", "LINEAR_MAX_OUTS", "LOGPROBS_MAX_VOCAB", "LOGPROBS_MAX_TOP"):
        assert getattr(moe, name) == int(re.search(rf"MOE_{name} (\d+)", src).group(1)), name


def mx(dense, **kw):
    m = dense._Mx(A, A, 1, 4, 256, 256, 8)
    for k, v in kw.items():
        setattr(m, k, v)
    return m


BAD_MX = [(dict(q=None), 1), (dict(s=None), 1), (dict(q=A + 8), 1), (dict(type=2), 1), (dict(type=-1), 1), (dict(rows=0), 1),
          (dict(cols=0), 1), (dict(cols=16), 1), (dict(cols=40), 1), (dict(q_stride=240), 1), (dict(q_stride=264), 1),
          (dict(q_stride=-256), 1), (dict(s_stride=7), 1), (dict(cols=16416, q_stride=1 << 15, s_stride=1 << 10), 2),
          (dict(q_stride=1 << 40), 2), (dict(s_stride=1 << 40), 2)]


def quantize(dense, m, x=B, dtype=1, stride=256):
    return dense._lib().moe_mx_quantize(x, dtype, stride, None if m is None else ctypes.byref(m), None)


def dequantize(dense, m, out=B, dtype=1, stride=256):
    return dense._lib().moe_mx_dequantize(None if m is None else ctypes.byref(m), out, dtype, stride, None)


def norm(dense, rows=4, cols=256, x=B, xt=1, xs=256, res=C, ro=C, rt=0, rs=256, w=D, eps=1e-6, out=E, ot=1, os=256, m=None):
    return dense._lib().moe_rms_norm(rows, cols, x, xt, xs, res, ro, rt, rs, w, eps, out, ot, os,
                                     None if m is None else ctypes.byref(m), None)


def linear(dense, x, w, add=None, adds=0, out=A, dt=0, os=8, status=None):
    return dense._lib().moe_mx_linear(ctypes.byref(x), ctypes.byref(w), add, adds, out, dt, os, status, None)


def scores(dense, rows=2, vocab=100, x=A, dt=0, stride=100, tokens=A, lp=A, rank=A, ent=A, top=3, ids=A, tlp=A):
    return dense._lib().moe_token_logprobs(rows, vocab, x, dt, stride, tokens, lp, rank, ent, top, ids, tlp, None)


@pytest.mark.parametrize("kw,want", BAD_MX)
def test_bad_matrix_is_refused(dense, kw, want):
    m = mx(dense, **kw)
    assert quantize(dense, m, stride=1 << 14) == want
    assert dequantize(dense, m, stride=1 << 14) == want
    assert norm(dense, cols=m.cols if 0 < m.cols <= 16384 and m.cols % 8 == 0 else 256, rs=1 << 14, xs=1 << 14, out=None, m=m) == want
    if "cols" not in kw:
        w = mx(dense, type=0, q_stride=128)
        assert linear(dense, m, w) == want
        if "type" not in kw:
            assert linear(dense, mx(dense), mx(dense, **{"type": 0, **kw})) == want


def test_null_matrix_is_refused(dense):
    assert quantize(dense, None) == dequantize(dense, None) == 1
    L = dense._lib()
    assert L.moe_mx_linear(None, ctypes.byref(mx(dense)), None, 0, A, 0, 8, None, None) == 1
    assert L.moe_mx_linear(ctypes.byref(mx(dense)), None, None, 0, A, 0, 8, None, None) == 1


@pytest.mark.parametrize("kw,want", [(dict(x=None), 1), (dict(x=A + 8), 1), (dict(dtype=2), 1), (dict(stride=260), 1),
                                     (dict(dtype=0, stride=258), 1), (dict(stride=1 << 38), 2)])
def test_conversion_refusals(dense, kw, want):
    assert quantize(dense, mx(dense), **kw) == want
    if "x" in kw:
        kw = {"out": kw["x"]}
    assert dequantize(dense, mx(dense), **kw) == want


def test_output_rows_over_one_another_are_refused(dense):
    for stride in (248, -248, 0):
        assert dequantize(dense, mx(dense), stride=stride) == 1
        assert norm(dense, os=stride) == 1
        assert norm(dense, rs=stride) == 1
    assert linear(dense, mx(dense), mx(dense, type=0, q_stride=128, rows=9), os=8) == 1


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), 1), (dict(cols=0), 1), (dict(cols=252), 1), (dict(cols=16392, xs=1 << 15, rs=1 << 15, os=1 << 15), 2),
    (dict(x=None), 1), (dict(x=A + 4), 1), (dict(xt=3), 1), (dict(xs=252), 1), (dict(res=None), 1), (dict(ro=None), 1),
    (dict(res=A + 8), 1), (dict(ro=A + 8), 1), (dict(rt=2), 1), (dict(rs=258), 1), (dict(w=A + 4), 1), (dict(eps=0.0), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(out=None), 1), (dict(out=A + 2), 1),
    (dict(ot=5), 1), (dict(os=260), 1), (dict(xs=1 << 39), 2)])
def test_norm_refusals(dense, kw, want):
    assert norm(dense, **kw) == want


def test_norm_takes_one_output_of_the_right_size(dense):
    assert norm(dense, m=mx(dense)) == 1                       # both
    assert norm(dense, out=None, m=mx(dense, rows=5)) == 1
    assert norm(dense, out=None, m=mx(dense, cols=128)) == 1
    assert norm(dense, cols=264, xs=264, rs=264, out=None, m=mx(dense)) == 1


@pytest.mark.parametrize("xkw,wkw,kw,want", [
    (dict(), dict(cols=128), dict(), 1), (dict(), dict(), dict(out=None), 1), (dict(), dict(), dict(dt=2), 1),
    (dict(), dict(), dict(out=A + 2), 1), (dict(), dict(), dict(dt=1, out=A + 1), 1), (dict(), dict(), dict(add=A + 1), 1),
    (dict(q=A + 16), dict(), dict(), 1), (dict(q_stride=272), dict(), dict(), 1), (dict(), dict(q=A + 16), dict(), 1),
    (dict(), dict(q_stride=144), dict(), 1), (dict(s=A + 2), dict(), dict(), 1), (dict(), dict(s_stride=10), dict(), 1),
    (dict(), dict(), dict(os=3), 1), (dict(), dict(), dict(status=A + 1), 1), (dict(), dict(), dict(add=A, adds=12), 1),
    (dict(), dict(type=1, q_stride=256), dict(), 2), (dict(cols=160, q_stride=160), dict(cols=160, q_stride=96), dict(), 2),
    (dict(rows=65537), dict(), dict(), 2), (dict(), dict(rows=262145), dict(os=1 << 19), 2),
    (dict(), dict(), dict(os=1 << 39), 2), (dict(), dict(), dict(add=A + 4, adds=-(1 << 39)), 2)])
def test_linear_refusals(dense, xkw, wkw, kw, want):
    assert linear(dense, mx(dense, **xkw), mx(dense, **{"type": 0, "q_stride": 128, **wkw}), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), 1), (dict(vocab=0), 1), (dict(x=None), 1), (dict(x=A + 2), 1), (dict(dt=1, x=A + 1), 1), (dict(dt=3), 1),
    (dict(stride=99), 1), (dict(stride=-99), 1), (dict(tokens=None), 1), (dict(tokens=None, lp=None), 1), (dict(top=-1), 1),
    (dict(top=0), 1), (dict(ids=None), 1), (dict(tlp=None), 1), (dict(top=0, ids=None, tlp=None, lp=None, rank=None, ent=None), 1),
    (dict(tokens=A + 1), 1), (dict(lp=A + 2), 1), (dict(rank=A + 3), 1), (dict(ent=A + 1), 1), (dict(ids=A + 2), 1),
    (dict(tlp=A + 2), 1), (dict(vocab=262145, stride=1 << 20), 2), (dict(rows=(1 << 24) + 1), 2), (dict(top=33), 2),
    (dict(stride=1 << 39), 2)])
def test_logprobs_refusals(dense, kw, want):
    assert scores(dense, **kw) == want


# ---------------------------------------------------------------------------------------- binding --

def cpu(*shape, dtype=None):
    import torch
    return torch.zeros(*shape, dtype=dtype or torch.float32)


def test_binding_refuses_before_a_call(moe, dense, monkeypatch):
    """Types, shapes, strides and devices that the kernels would misread never reach the library."""
    import torch
    u8, i32, bf = torch.uint8, torch.int32, torch.bfloat16
    calls = []
    fake = type("L", (), {n: staticmethod(lambda *a, n=n: calls.append(n) or 0) for n in moe.DENSE_EXPORTS})()
    monkeypatch.setattr(dense, "_READY", fake)
    M = moe.MXMatrix
    with pytest.raises(ValueError):
        M(cpu(4, 64, dtype=u8), cpu(4, 2, dtype=u8), "e5m2")
    with pytest.raises(ValueError):
        M.empty(4, 64, "fp4", device="cpu")
    with pytest.raises(ValueError):
        M.empty(4, 48, device="cpu")
    with pytest.raises(TypeError):
        M(cpu(4, 64), cpu(4, 2, dtype=u8), "e4m3")
    with pytest.raises(TypeError):
        M(cpu(4, 64, dtype=u8), cpu(4, 2), "e4m3")
    with pytest.raises(ValueError):
        M(cpu(64, 4, dtype=u8).T, cpu(4, 2, dtype=u8), "e4m3")
    with pytest.raises(ValueError):
        M(cpu(4, 64, dtype=u8), cpu(4, 3, dtype=u8), "e4m3")
    with pytest.raises(ValueError):
        M(cpu(4, 24, dtype=u8), cpu(4, 1, dtype=u8))
    a, w = M.empty(4, 64, "e4m3", device="cpu"), M.empty(8, 64, device="cpu")
    for bad in (cpu(4, 64, dtype=torch.float16), cpu(4, 64, dtype=i32)):
        with pytest.raises(TypeError):
            moe.mx_quantize(bad, a)
        with pytest.raises(TypeError):
            moe.mx_dequantize(a, bad)
        with pytest.raises(TypeError):
            moe.rms_norm(bad, a)
        with pytest.raises(TypeError):
            moe.token_logprobs(bad, entropy=cpu(4))
    for bad in (cpu(4, 32), cpu(64, 4).T, cpu(3, 64)):
        with pytest.raises(ValueError):
            moe.mx_quantize(bad, a)
        with pytest.raises(ValueError):
            moe.rms_norm(bad, a)
    with pytest.raises(TypeError):
        moe.mx_quantize(cpu(4, 64), cpu(4, 64))
    # On the host: refused by the device check.
    for call in (lambda: moe.mx_quantize(cpu(4, 64), a), lambda: moe.mx_dequantize(a, cpu(4, 64)), lambda: moe.rms_norm(cpu(4, 64), a),
                 lambda: moe.mx_linear(a, w, cpu(4, 8)), lambda: moe.token_logprobs(cpu(4, 64), entropy=cpu(4))):
        with pytest.raises(ValueError):
            call()
    x = cpu(4, 64)
    with pytest.raises(ValueError):
        moe.rms_norm(x, a, residual=x)
    with pytest.raises(ValueError):
        moe.rms_norm(x, a, residual_out=x)
    with pytest.raises(ValueError):
        moe.rms_norm(x, a, residual=x, residual_out=cpu(4, 64, dtype=bf))
    with pytest.raises(ValueError):
        moe.rms_norm(x, a, residual=x, residual_out=cpu(4, 128)[:, :64])
    with pytest.raises(ValueError):
        moe.rms_norm(x, a, weight=cpu(32))
    with pytest.raises(ValueError):
        moe.rms_norm(x, a, weight=cpu(64, dtype=bf))
    with pytest.raises(ValueError):
        moe.mx_linear(a, M.empty(8, 96, device="cpu"), cpu(4, 8))
    with pytest.raises(ValueError):
        moe.mx_linear(a, w, cpu(4, 9))
    with pytest.raises(TypeError):
        moe.mx_linear(a, w, cpu(4, 8), add=cpu(4, 8, dtype=bf))
    with pytest.raises(TypeError):
        moe.token_logprobs(x, cpu(4), cpu(4))
    with pytest.raises(ValueError):
        moe.token_logprobs(x, cpu(5, dtype=i32), cpu(4))
    with pytest.raises(ValueError):
        moe.token_logprobs(x, top_ids=cpu(4, 3, dtype=i32))
    with pytest.raises(ValueError):
        moe.token_logprobs(x, top_ids=cpu(4, 3, dtype=i32), top_logprobs=cpu(4, 2))
    with pytest.raises(ValueError):
        moe.token_logprobs(cpu(64, 4).T, entropy=cpu(4))
    assert calls == []


def test_a_single_row_has_any_stride(moe):
    """One row of a wider tensor, and a view whose single row has another stride: the struct holds lengths that fit."""
    import torch
    q, s = torch.zeros(3, 100, dtype=torch.uint8)[1:2, :32], torch.zeros(3, 7, dtype=torch.uint8)[1:2, :2]
    m = moe.MXMatrix(q, s)
    assert (m.rows, m.cols, m.struct.q_stride, m.struct.s_stride) == (1, 64, 32, 4)


@pytest.mark.parametrize("kw", [dict(out=B, ot=0), dict(out=B, os=512), dict(out=C), dict(out=C, ot=0, os=512), dict(ro=B), dict(ro=E),
                                dict(out=C, ot=0)])
def test_norm_over_its_inputs_in_another_form_is_refused(dense, kw):
    """A row's results over rows that other CTAs have yet to read, or two results in one place."""
    assert norm(dense, **kw) == 1


def test_codes_over_their_values_are_refused(dense):
    assert quantize(dense, mx(dense), x=A) == 1 and dequantize(dense, mx(dense), out=A) == 1
    for at in (B, C):
        assert norm(dense, out=None, m=mx(dense, q=at)) == 1
