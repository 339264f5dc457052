"""moe_rms_norm over the whole range of eps."""
import numpy as np
import pytest

import dense_ref as ref
from serve_ref import torch
from test_gpu_mx import FP32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch().cuda.is_available():
        pytest.skip("no CUDA device")
    import mxfp4_routed_expert_moe_gb300 as m
    return m


@pytest.mark.parametrize("cols", [8, 64, 768, 1024, 7168, 16384])
@pytest.mark.parametrize("eps", [1e-45, 1e-38, 1e-6, 1.0, 1e20, 1.7e38, 3.3e38, 3.39e38])
def test_any_eps(moe, cols, eps):
    """Rows whose sum of squares is near fp32's largest, beyond it, and small, with an eps that may not be added to their
    mean in fp32.  Bounds as of other norms: none of these rows' mean and eps comes near fp32's smallest numbers but for
    eps itself, beside a mean of 0 or one that hides it."""
    t = torch()
    rng = np.random.default_rng(cols)
    sizes = np.sqrt(np.array([2.9e38, 2.99e38, 1e38, 3.1e38, 1e30, 1.0, 1e-10, 0.0]) / cols)
    x = (rng.integers(0, 2, (len(sizes), cols)) * 2 - 1) * sizes[:, None]
    x = t.from_numpy(x.astype(np.float32)).cuda()
    out = t.empty_like(x)
    moe.rms_norm(x, out, eps=eps)
    h, e = ref.host(x), float(np.float32(eps))
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + e)
    assert np.all(np.abs(ref.host(out) - y) <= FP32 * np.abs(y) + 2.0 ** -149)
