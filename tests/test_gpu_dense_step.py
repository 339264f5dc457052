"""The dense operators together, as a step uses them: stage by stage against 64-bit forms of what each was given, the
example's microscaled model, sampling and scoring of one distribution, and experts quantised into their table."""
import importlib.util
import os

import numpy as np
import pytest

import dense_ref as ref
from conftest import ROOT
from serve_ref import torch
from test_gpu_linear import bound, product
from test_gpu_mx import FP32, check_mx

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch().cuda.is_available():
        pytest.skip("no CUDA device")
    import mxfp4_routed_expert_moe_gb300 as m
    return m


@pytest.fixture(scope="module")
def example(moe):
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("T", [1, 5, 130, 700])
def test_norm_product_residual_norm_product_scores(moe, T):
    """rms_norm -> mx_linear -> mx_quantize -> mx_linear into the residual -> rms_norm -> mx_linear -> token_logprobs in
    one captured graph, replayed on new inputs; each stage's result against the formula on that stage's own inputs."""
    t = torch()
    H, N, V = 512, 384, 1003
    rng = np.random.default_rng(T)
    f32 = dict(device="cuda")

    def mx(rows, cols, kind):
        return moe.MXMatrix.empty(rows, cols, kind)

    def weights(rows, cols):
        w = mx(rows, cols, "e2m1")
        moe.mx_quantize(t.from_numpy(rng.standard_normal((rows, cols)).astype(np.float32) * cols ** -0.5).cuda(), w)
        return w

    x = t.empty(T, H, dtype=t.bfloat16, device="cuda")
    res, res2 = t.empty(T, H, **f32), t.empty(T, H, **f32)
    gain = t.from_numpy(1 + 0.1 * rng.standard_normal(H).astype(np.float32)).cuda()
    w1, w2, w3 = weights(N, H), weights(H, N), weights(V, H)
    a8, b8, c4 = mx(T, H, "e4m3"), mx(T, N, "e4m3"), mx(T, H, "e2m1")
    mid, logits = t.empty(T, N, dtype=t.bfloat16, device="cuda"), t.empty(T, V, **f32)
    token = t.from_numpy(rng.integers(0, V, T).astype(np.int32)).cuda()
    logprob, rank = t.empty(T, **f32), t.empty(T, dtype=t.int32, device="cuda")
    status = t.zeros(1, dtype=t.int32, device="cuda")

    def step():
        moe.rms_norm(x, a8, weight=gain, residual=res, residual_out=res2)
        moe.mx_linear(a8, w1, mid, status=status)
        moe.mx_quantize(mid, b8)
        moe.mx_linear(b8, w2, res2, add=res2, status=status)
        moe.rms_norm(res2, c4, weight=gain)
        moe.mx_linear(c4, w3, logits, status=status)
        moe.token_logprobs(logits, token, logprob, rank=rank)

    def fill(seed):
        r = np.random.default_rng(seed)
        x.copy_(t.from_numpy(r.standard_normal((T, H)).astype(np.float32)))
        res.copy_(t.from_numpy(r.standard_normal((T, H)).astype(np.float32) * 2))

    fill(1)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    graph = t.cuda.CUDAGraph()
    with t.cuda.stream(side):
        step()
        with t.cuda.graph(graph, stream=side):
            step()
    t.cuda.current_stream().wait_stream(side)
    fill(2)
    graph.replay()
    t.cuda.synchronize()
    assert int(status.item()) == 0

    def parts(m):
        return ref.unpack(m.q.cpu().numpy(), m.kind), m.s.cpu().numpy()

    def values(m):
        return ref.values(*parts(m), m.kind)

    def normed(h):
        return h / np.sqrt((h * h).mean(1, keepdims=True) + 1e-6) * ref.host(gain)

    h = ref.host(x) + ref.host(res)
    check_mx(*parts(a8), normed(h), "e4m3")
    y, mag = product(values(a8), values(w1))
    assert np.all(np.abs(ref.host(mid) - y) <= bound("e4m3", H, mag, y, "bf16"))
    code, s = ref.quantize(ref.host(mid), "e4m3")
    assert np.array_equal(parts(b8)[0], code) and np.array_equal(parts(b8)[1], s)
    y, mag = product(values(b8), values(w2))
    # The residual of the first norm is h rounded to fp32 before the product is added.
    assert np.all(np.abs(ref.host(res2) - (y + h)) <= bound("e4m3", N, mag + np.abs(h), y + h, "f32") + 2.0 ** -24 * np.abs(h))
    check_mx(*parts(c4), normed(ref.host(res2)), "e2m1")
    y, mag = product(values(c4), values(w3))
    assert np.all(np.abs(ref.host(logits) - y) <= bound("e2m1", H, mag, y, "f32"))
    z = ref.host(logits)
    lp = z - z.max(1, keepdims=True)
    lp -= np.log(np.exp(lp).sum(1, keepdims=True))
    at = token.cpu().numpy()
    assert np.all(np.abs(ref.host(logprob) - lp[np.arange(T), at]) <= 2.0 ** -18)
    order = np.argsort(-z, axis=1, kind="stable")
    assert np.array_equal(rank.cpu().numpy(), (order == at[:, None]).argmax(1))


def test_sampled_and_scored_log_probabilities_agree(moe):
    """Without filters, sample's log probability of the token it drew is token_logprobs' of that token: integer weights
    of 2^-31 against fp32 sums of 4,099 terms, each within 2^-18 for tokens that are drawn with some probability."""
    t = torch()
    g = t.Generator("cuda").manual_seed(5)
    logits = (t.randn(300, 4099, generator=g, device="cuda") * 3).bfloat16()
    token, drawn, scored = t.empty(300, dtype=t.int32, device="cuda"), t.empty(300, device="cuda"), t.empty(300, device="cuda")
    rank = t.empty_like(token)
    moe.sample(logits, t.rand(300, generator=g, device="cuda"), token, logprob=drawn)
    moe.token_logprobs(logits, token, scored, rank=rank)
    likely = drawn > -9
    assert likely.any() and float((drawn - scored)[likely].abs().max()) <= 2.0 ** -18
    # Greedy rows draw the token of rank 0.
    moe.sample(logits, t.zeros(300, device="cuda"), token, temperature=t.zeros(300, device="cuda"))
    moe.token_logprobs(logits, token, scored, rank=rank)
    assert t.all(rank == 0)


def test_example_in_microscaled_formats(example):
    """The example with --mx runs, repeats, draws valid tokens and scores a text."""
    t = torch()
    model = example.Model(mx=True)
    prompt = t.randint(0, 4099, (45,), generator=t.Generator().manual_seed(3)).cuda()
    tokens, logits, lp = example.generate(model, prompt, sequences=3, steps=4)
    again, logits2, lp2 = example.generate(model, prompt, sequences=3, steps=4)
    assert t.equal(tokens, again) and t.equal(logits, logits2) and t.equal(lp, lp2)
    assert t.all((tokens >= 0) & (tokens < 4099)) and t.all(lp < 0)
    s = example.score(model, t.cat((prompt, tokens[0, :1].long())), top=5)
    assert t.all(s["rank"] >= 0) and t.all(s["entropy"] > 0) and t.all(s["top_logprobs"][:, :-1] >= s["top_logprobs"][:, 1:])
    assert t.all(s["logprob"] <= s["top_logprobs"][:, 0]) and t.all((s["rank"] == 0) == (s["top_ids"][:, 0] == t.cat((prompt[1:], tokens[0, :1].long()))))
    assert int(model.status.item()) == 0


def test_experts_quantised_into_the_table(moe):
    """ExpertTable.quantize writes what mx_quantize defines, and weights that are on the MXFP4 grid already give the
    layer they came from."""
    import synth
    from harness import DeviceLayer
    t = torch()
    wl = synth.WORKLOADS["tiny"]
    inp = synth.make_inputs(wl)
    L = DeviceLayer(inp)
    base, _, _ = L.forward(path=1)
    table = moe.ExpertTable(wl.E, wl.H, wl.I, "cuda:0")
    for e in range(wl.E):
        dense = []
        for j, shape in ((0, (wl.I, wl.H)), (2, (wl.I, wl.H)), (4, (wl.H, wl.I))):
            w = t.empty(shape, device="cuda")
            moe.mx_dequantize(moe.MXMatrix(L.table.tensor(e, j), L.table.tensor(e, j + 1)), w)
            dense.append(w)
        table.quantize(e, *dense)
        for j, w in zip((0, 2, 4), dense):
            back = t.empty_like(w)
            moe.mx_dequantize(moe.MXMatrix(table.tensor(e, j), table.tensor(e, j + 1)), back)
            assert t.equal(back, w)
    L.table = table
    got, _, _ = L.forward(path=1)
    # Equal weights in other codes and scales: exact block sums either way, fp32 sums of the blocks.
    assert float((got - base).abs().max()) <= 1e-5 * float(base.abs().max())
