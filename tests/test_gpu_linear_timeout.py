"""moe_mx_linear with a limit of one cycle for its waits: results whose sum is not whole are NaN, all others as ever."""
import numpy as np
import pytest

import dense_ref as ref
from serve_ref import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch().cuda.is_available():
        pytest.skip("no CUDA device")
    import mxfp4_routed_expert_moe_gb300 as m
    return m


@pytest.mark.parametrize("kind", ["e4m3", "e2m1"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,K,addend", [
    (4, 512, 7168, True), (1, 9216, 7168, False),      # clusters; two CTAs an SM
    (64, 1407, 7168, True),                            # clusters, a column a thread
    (32, 30000, 2048, False), (1, 1, 128, True),       # single CTAs
    (1024, 2048, 1024, True), (700, 4099, 1408, False),  # pairs
    (4100, 5000, 512, True)])                          # pairs of several tiles
def test_no_sum_is_passed_off_as_whole(moe, T, N, K, addend, out, kind):
    t = torch()
    rng = np.random.default_rng(T + N)
    xc, xs = ref.random_mx(rng, T, K, kind)
    wc, ws = ref.random_mx(rng, N, K, "e2m1")
    x, w = ref.matrix(moe, xc, xs, kind), ref.matrix(moe, wc, ws, "e2m1")
    dt = t.float32 if out == "f32" else t.bfloat16
    start = t.from_numpy(rng.standard_normal((T, N)).astype(np.float32)).cuda().to(dt)
    good = t.empty(T, N, dtype=dt, device="cuda")
    moe.mx_linear(x, w, good, add=start if addend else None)
    assert not good.isnan().any()
    status = t.zeros(1, dtype=t.int32, device="cuda")
    for st in (status, None):
        got = start.clone()
        t.cuda.synchronize()
        moe.set_wait_limit(1)
        try:
            moe.mx_linear(x, w, got, add=got if addend else None, status=st)
            t.cuda.synchronize()
        finally:
            moe.set_wait_limit(0)
        lost = got.isnan()
        assert lost.any()  # no first slice is there within a cycle
        assert t.all(lost | (got == good))
    assert int(status.item()) == moe.MOE_ERR_TIMEOUT
    status.zero_()
    got = start.clone()
    moe.mx_linear(x, w, got, add=got if addend else None, status=status)
    assert int(status.item()) == 0 and t.equal(got, good)
