"""Operators one behind the other on buffers that each step writes anew: a kernel that starts while the one before it
still runs reads what that one has written, scales, tokens, logits and weights of a norm among it."""
import numpy as np
import pytest

from serve_ref import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch().cuda.is_available():
        pytest.skip("no CUDA device")
    import mxfp4_routed_expert_moe_gb300 as m
    return m


@pytest.mark.parametrize("T,H,N", [(1, 512, 1003), (5, 1408, 4099), (64, 512, 2051), (300, 1024, 4099)])
def test_each_step_reads_what_the_one_before_wrote(moe, T, H, N):
    t = torch()
    g = t.Generator("cuda").manual_seed(T + N)
    f32, i32 = dict(device="cuda"), dict(device="cuda", dtype=t.int32)
    w = moe.MXMatrix.empty(N, H, "e2m1")
    moe.mx_quantize(t.randn(N, H, generator=g, **f32), w)
    steps = 24
    # Inputs of very different size, so that scales, codes and drawn tokens change from step to step.
    size = 2.0 ** t.randint(-8, 9, (steps, T, H // 32, 1), generator=g, **f32)
    x = (t.randn(steps, T, H // 32, 32, generator=g, **f32) * size).reshape(steps, T, H)
    gain = t.randn(steps, H, generator=g, **f32)
    u = t.rand(steps, T, generator=g, **f32)

    def run(wait):
        a8, y = moe.MXMatrix.empty(T, H, "e4m3"), t.empty(T, H, **f32)
        weight, logits = t.empty(H, **f32), t.empty(T, N, **f32)
        token, logprob, rank = t.zeros(T, **i32), t.empty(T, **f32), t.empty(T, **i32)
        got = []
        for k in range(steps):
            moe.rms_norm(gain[k][None], weight[None])  # a weight that a kernel writes
            wait()
            moe.rms_norm(x[k], y, weight=weight)
            wait()
            moe.mx_quantize(y, a8)
            wait()
            moe.mx_linear(a8, w, logits)
            wait()
            moe.sample(logits, u[k], token)
            wait()
            moe.token_logprobs(logits, token, logprob, rank=rank)
            wait()
            got.append((logits.clone(), token.clone(), logprob.clone(), rank.clone()))
        t.cuda.synchronize()
        return got

    want = run(t.cuda.synchronize)
    assert len({tuple(o[1].tolist()) for o in want}) > steps // 2
    for _ in range(3):
        for a, b in zip(run(lambda: None), want):
            assert all(t.equal(p, q) for p, q in zip(a, b))
