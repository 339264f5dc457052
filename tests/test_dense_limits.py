"""Limits of moe_dense.h: declared, known to the binding, and where the library refuses (no GPU needed: refused calls
return before touching CUDA)."""
import os
import re

import pytest

from conftest import ROOT
from test_dense_abi import HEADER, dense, dequantize, linear, moe, mx, norm, quantize, scores  # noqa: F401

INT64_MIN = -(1 << 63)


def test_every_limit_is_declared_and_bound(moe):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    limits = dict(re.findall(r"^#define MOE_(\w*_MAX_\w+) \(?(\d+(?:LL << \d+)?)\)?\s*(?:LL)?", src, flags=re.M))
    assert set(limits) == {"DENSE_MAX_COLS", "DENSE_MAX_STRIDE", "MX_MAX_VALUES", "LINEAR_MAX_ROWS", "LINEAR_MAX_OUTS",
                           "LOGPROBS_MAX_ROWS", "LOGPROBS_MAX_VOCAB", "LOGPROBS_MAX_TOP"}
    for name, value in limits.items():
        assert getattr(moe, name) == eval(value.replace("LL", "")), name
    # Each is a limit of the code, under its name.
    code = open(os.path.join(ROOT, "mxfp4_routed_expert_moe_gb300", "csrc", "dense.cu")).read()
    for name in limits:
        assert "MOE_" + name in code, name


def test_refused_beyond_each_limit(moe, dense):
    most = moe.MX_MAX_VALUES
    for cols in (32, 7168, 16384):
        rows = most // cols + 1
        if rows > (1 << 31) - 1:
            continue
        m = mx(dense, rows=rows, cols=cols, q_stride=cols, s_stride=cols // 32)
        assert quantize(dense, m, stride=cols) == 2 and dequantize(dense, m, stride=cols) == 2
    assert scores(dense, rows=moe.LOGPROBS_MAX_ROWS + 1) == 2
    assert scores(dense, vocab=moe.LOGPROBS_MAX_VOCAB + 1, stride=1 << 20) == 2
    assert scores(dense, top=moe.LOGPROBS_MAX_TOP + 1) == 2
    far = moe.DENSE_MAX_STRIDE
    w = mx(dense, type=0, q_stride=128)
    for stride in (far, -far, 1 << 61, -(1 << 61)):
        assert quantize(dense, mx(dense), stride=stride) == dequantize(dense, mx(dense), stride=stride) == 2
        assert norm(dense, xs=stride) == norm(dense, rs=stride) == norm(dense, os=stride) == 2
        assert linear(dense, mx(dense), w, os=stride) == linear(dense, mx(dense), w, add=1 << 21, adds=stride) == 2
        assert scores(dense, stride=stride) == 2
    for stride in (4 * far, 1 << 62):
        assert quantize(dense, mx(dense, q_stride=stride)) == quantize(dense, mx(dense, s_stride=stride)) == 2


def test_the_lowest_stride_is_refused(moe, dense):
    """-2^63 has no magnitude in 64 bits."""
    w = mx(dense, type=0, q_stride=128)
    assert quantize(dense, mx(dense), stride=INT64_MIN) == 2
    assert dequantize(dense, mx(dense), stride=INT64_MIN) == 2
    assert norm(dense, xs=INT64_MIN) == norm(dense, rs=INT64_MIN) == norm(dense, os=INT64_MIN) == 2
    assert linear(dense, mx(dense), w, os=INT64_MIN) == linear(dense, mx(dense), w, add=1 << 21, adds=INT64_MIN) == 2
    assert scores(dense, stride=INT64_MIN) == 2
