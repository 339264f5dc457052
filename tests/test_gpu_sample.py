"""moe_sample against its definition: weights by the fp32 exponential, everything after it in exact integers."""
import numpy as np
import pytest

from serve_ref import sample_row, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch().cuda.is_available():
        pytest.skip("no CUDA device")
    import mxfp4_routed_expert_moe_gb300 as m
    return m


def scaled(logits, temperature):
    """z and exp(z - max) in fp32, as the definition has them (NaN as -inf)."""
    t = torch()
    x = logits.float()
    one = t.ones_like(temperature)
    z = x * t.where(temperature == 0, one, 1.0 / temperature)[:, None]
    z = t.where(z.isnan(), -float("inf"), z)
    m = z.amax(1, keepdim=True)
    w = t.where(m == float("inf"), (z == m).float(), t.exp(z - m))
    return z.cpu().numpy(), w.nan_to_num(0.0).cpu().numpy()


def run(moe, logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
    t = torch()
    rows, vocab = logits.shape
    dev = lambda a, dt: None if a is None else t.tensor(a, dtype=dt, device="cuda")  # noqa: E731
    token = t.full((rows,), -9, dtype=t.int32, device="cuda")
    kept = t.full((rows,), -9, dtype=t.int32, device="cuda")
    logprob = t.full((rows,), 9.0, device="cuda")
    probs = t.full((rows, vocab), 9.0, device="cuda")
    moe.sample(logits, dev(u, t.float32), token, temperature=dev(temperature, t.float32), top_k=dev(top_k, t.int32),
               top_p=dev(top_p, t.float32), min_p=dev(min_p, t.float32), logprob=logprob, kept=kept, probs=probs)
    # The optional outputs change nothing.
    alone = t.empty_like(token)
    moe.sample(logits, dev(u, t.float32), alone, temperature=dev(temperature, t.float32), top_k=dev(top_k, t.int32),
               top_p=dev(top_p, t.float32), min_p=dev(min_p, t.float32))
    assert t.equal(alone, token)
    return token.cpu().numpy(), kept.cpu().numpy(), logprob.cpu().numpy(), probs.cpu().numpy()


def check(moe, logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
    t = torch()
    rows = logits.shape[0]
    token, kept, logprob, probs = run(moe, logits, u, temperature, top_k, top_p, min_p)
    temp = t.tensor(temperature if temperature is not None else [1.0] * rows, dtype=t.float32, device="cuda")
    z, w = scaled(logits, temp)
    at = lambda a, i, off: off if a is None else a[i]  # noqa: E731
    for i in range(rows):
        if float(temp[i]) == 0:
            want, n, f = int(np.argmax(z[i])), 1, None
            assert logprob[i] == 0 and probs[i].sum() == 1 and probs[i][want] == 1
        else:
            want, n, f = sample_row(z[i], w[i], u[i], at(top_k, i, 0), at(top_p, i, 1.0), at(min_p, i, 0.0))
            p = f / f.sum()
            # W and S to fp32 (2^-24 each), a reciprocal, a product, a logarithm: within 4 units of 2^-23.
            np.testing.assert_allclose(probs[i], p, rtol=4 * 2.0 ** -23, atol=0)
            lp = np.log(p[want])
            assert abs(logprob[i] - lp) <= 4 * 2.0 ** -23 * (1 + abs(lp)), (i, logprob[i], lp)
        assert (token[i], kept[i]) == (want, n), (i, token[i], want, kept[i], n)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 7), (5, 1000), (2, 32001), (1, 100003), (33, 50257), (4, 262144),
                                        (300, 4099)])
def test_filters(moe, rows, vocab, dtype):
    t = torch()
    rng = np.random.default_rng(rows * 1000 + vocab)
    logits = t.from_numpy((rng.standard_normal((rows, vocab)) * 3).astype(np.float32)).cuda()
    if dtype == "bf16":
        logits = logits.bfloat16()  # many ties
    u = rng.random(rows).astype(np.float32).tolist()
    temp = np.where(rng.random(rows) < 0.2, 0, rng.uniform(0.2, 2, rows)).astype(np.float32).tolist()
    k = np.where(rng.random(rows) < 0.3, 0, rng.integers(1, vocab + 2, rows)).tolist()
    small_k = rng.integers(1, min(vocab, 60) + 1, rows).tolist()
    p = np.where(rng.random(rows) < 0.2, 1, rng.random(rows)).astype(np.float32).tolist()
    mp = np.where(rng.random(rows) < 0.3, 0, rng.random(rows) * 0.2).astype(np.float32).tolist()
    check(moe, logits, u)
    check(moe, logits, u, temp)
    check(moe, logits, u, temp, top_k=small_k)
    check(moe, logits, u, None, top_p=p)
    check(moe, logits, u, temp, min_p=mp)
    check(moe, logits, u, temp, top_k=k, top_p=p, min_p=mp)


def test_weights_are_the_exponential(moe):
    """Unfiltered probabilities against 64 bits: exp to 2 units in the last place, the fixed-point unit, and
    the fp32 quotient."""
    t = torch()
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((2, 5000)) * 4).astype(np.float32)
    _, _, _, probs = run(moe, t.from_numpy(x).cuda(), [0.5, 0.5])
    e = np.exp(x.astype(np.float64) - x.max(1, keepdims=True).astype(np.float64))
    s = e.sum(1, keepdims=True)
    # z - m rounds (2^-24 |z - m| <= 2^-24 * 32 in the exponent), W by half a unit of 2^-31.
    assert np.all(np.abs(probs - e / s) <= (e * (32 * 2.0 ** -24 + 6 * 2.0 ** -23) + 2.0 ** -31) / s)


def test_ties_and_crowded_bins(moe):
    """Equal scores rank by index, also where one histogram bin holds thousands of them."""
    t = torch()
    for vocab in (9, 5000, 70001):
        flat = t.zeros(4, vocab, device="cuda")
        check(moe, flat, [0.0, 0.3, 0.999999, 0.5], None, top_k=[1, 3, vocab, vocab - 1])
        check(moe, flat, [0.0, 0.3, 0.999999, 0.5], None, top_p=[0.0, 0.1, 0.5, 0.9999])
    near = t.from_numpy((np.random.default_rng(0).random((3, 40000)) * 1e-3).astype(np.float32)).cuda()
    near[:, ::7] = 5e-4
    check(moe, near, [0.1, 0.5, 0.9], None, top_k=[20000, 0, 3], top_p=[0.5, 0.2, 0.7])


def test_extreme_scores(moe):
    t = torch()
    inf, nan = float("inf"), float("nan")
    low = float(np.finfo(np.float32).min)
    x = t.tensor([[1.0, -inf, nan, 0.0, -inf, low], [inf, 1.0, inf, -inf, nan, inf], [low] * 6,
                  [-0.0, 0.0, -1.0, -0.0, -40.0, -15.0]], device="cuda")
    u = [0.9, 0.6, 0.4, 0.3]
    check(moe, x, u)
    check(moe, x, u, None, top_k=[2, 2, 4, 2], top_p=[0.9, 0.5, 0.5, 0.6], min_p=[0.1, 0.1, 1.0, 7.0])
    check(moe, x, u, [0.0] * 4)
    # Nothing to choose from, or a temperature that means nothing.
    token, kept, logprob, probs = run(moe, t.tensor([[-inf] * 6, [nan] * 6, [1.0] * 6, [1.0] * 6], device="cuda"),
                                      [0.5] * 4, [1.0, 0.0, -1.0, nan], top_k=[2] * 4, top_p=[0.5] * 4)
    assert token.tolist() == [-1] * 4 and kept.tolist() == [0] * 4
    assert np.all(logprob == -inf) and np.all(probs == 0)


def test_uniform_numbers_out_of_range_and_at_the_ends(moe):
    t = torch()
    x = t.zeros(5, 4, device="cuda")
    token, _, _, _ = run(moe, x, [0.0, float(np.nextafter(np.float32(1), np.float32(0))), 1.0, -3.0, float("nan")])
    assert token.tolist() == [0, 3, 3, 0, 0]


def test_strided_and_unaligned_rows(moe):
    """Rows of a wider matrix, starting at every offset within 16 bytes."""
    t = torch()
    rng = np.random.default_rng(5)
    for dt in (t.float32, t.bfloat16):
        wide = t.from_numpy((rng.standard_normal((6, 4111)) * 3).astype(np.float32)).cuda().to(dt)
        for off in range(8):
            view = wide[:, off:off + 4001]
            a = run(moe, view, [0.7] * 6, None, [50] * 6, [0.9] * 6)
            b = run(moe, view.contiguous(), [0.7] * 6, None, [50] * 6, [0.9] * 6)
            for x, y in zip(a, b):
                np.testing.assert_array_equal(x, y)


def test_frequencies(moe):
    """u on a grid gives each token its share."""
    t = torch()
    n = 4096
    x = t.log(t.tensor([4.0, 1.0, 2.0, 1.0], device="cuda")).repeat(n, 1).contiguous()
    token, _, _, _ = run(moe, x, ((np.arange(n) + 0.5) / n).astype(np.float32).tolist())
    counts = np.bincount(token, minlength=4)
    assert np.all(np.abs(counts - n * np.array([0.5, 0.125, 0.25, 0.125])) <= 1)


def test_graph_follows_the_parameters(moe):
    """A captured call reads its parameters and numbers at each replay, on its own stream."""
    t = torch()
    rng = np.random.default_rng(8)
    x = t.from_numpy((rng.standard_normal((4, 5001)) * 3).astype(np.float32)).cuda()
    u = t.full((4,), 0.5, device="cuda")
    k = t.full((4,), 5, dtype=t.int32, device="cuda")
    token = t.empty(4, dtype=t.int32, device="cuda")
    kept = t.empty(4, dtype=t.int32, device="cuda")
    moe.sample(x, u, token, top_k=k, kept=kept)
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        moe.sample(x, u, token, top_k=k, kept=kept)
    k.fill_(17)
    u.fill_(0.9)
    g.replay()
    t.cuda.synchronize()
    assert kept.tolist() == [17] * 4
    z, w = scaled(x, t.ones(4, device="cuda"))
    assert token.tolist() == [sample_row(z[i], w[i], 0.9, 17)[0] for i in range(4)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_candidate_lists_of_all_lengths(moe, dtype):
    """Few to many candidates in one CTA's list, kept alone and cut further, at both ends of u."""
    t = torch()
    ks = [1, 2, 31, 32, 33, 127, 128, 129, 255, 256, 257, 511, 512, 513, 900, 1023, 1024, 1025, 2000]
    rng = np.random.default_rng(77)
    x = t.from_numpy((rng.standard_normal((len(ks), 50021)) * 2).astype(np.float32)).cuda()
    if dtype == "bf16":
        x = x.bfloat16()
    temp = [1.7] * len(ks)  # flat: many tokens weigh alike
    for u in (0.0, 0.37, 0.99999994):
        check(moe, x, [u] * len(ks), temp, top_k=ks)
        check(moe, x, [u] * len(ks), temp, top_k=ks, top_p=[0.9] * len(ks))
        check(moe, x, [u] * len(ks), temp, top_k=ks, min_p=[0.2] * len(ks))
    peaked = [0.25] * len(ks)
    check(moe, x, rng.random(len(ks)).astype(np.float32).tolist(), peaked, top_p=np.linspace(0.05, 0.999, len(ks)).astype(np.float32).tolist())


@pytest.mark.parametrize("top", [4194304.5, 5000000.5, 8000001.0, -5210070.5, 4e7, -4e7, 1e8, 1.2e8, 3e8, 2.0 ** 31])
def test_large_scaled_scores(moe, top):
    """Floats of this size have none at the cut below which weights are 0: scores on both sides of it, and between it
    and the maximum, rank in their order."""
    rng = np.random.default_rng(12)
    below = np.concatenate([[0, 0, 4, 4, 8, 16, 20, 21.5, 22, 22.25, 22.5, 23, 24, 24, 26, 28, 32, 64], rng.uniform(0, 40, 3000)])
    x = np.tile((np.float64(top) - below).astype(np.float32), (6, 1))
    for row in x[1:]:
        rng.shuffle(row)
    logits = torch().from_numpy(x).cuda()
    u = [0.0, 0.2, 0.5, 0.9, 0.999, 0.99999994]
    check(moe, logits, u)
    check(moe, logits, u, None, top_k=[1, 2, 3, 40, 1500, 3017])
    check(moe, logits, u, None, top_p=[0.1, 0.5, 0.9, 0.99, 0.9999, 0.99999994])
    check(moe, logits, u, None, min_p=[0.5, 1e-3, 1e-6, 1e-9, 1e-10, 0.0])
    check(moe, logits, u, None, top_k=[2, 3, 100, 2000, 5000, 3000], top_p=[0.99, 0.9, 0.999, 0.9999, 0.999, 0.5], min_p=[0.0, 1e-4, 0.0, 1e-9, 0.0, 1e-2])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_small_temperatures(moe, dtype):
    """Ordinary logits over temperatures that take them to such sizes."""
    t = torch()
    rng = np.random.default_rng(13)
    x = t.from_numpy((5 + rng.random((5, 30011)) * 2.5e-5).astype(np.float32)).cuda()
    x[:, 7::1001] = 5.0000224
    if dtype == "bf16":
        x = x.bfloat16()
        x[:, ::1000] = 5.03125
    temp, u = [1e-6, 3e-7, 1.3e-7, 5e-8, 2e-6], [0.1, 0.4, 0.6, 0.9, 0.3]
    check(moe, x, u, temp)
    check(moe, x, u, temp, top_k=[2, 50, 700, 5000, 30011], top_p=[0.9, 0.99, 0.5, 0.9999, 0.3])
    check(moe, x, u, temp, top_p=[0.9, 0.99, 0.5, 0.9999, 0.3], min_p=[0.0, 0.1, 0.0, 1e-9, 0.2])


@pytest.mark.parametrize("rows", [1, 7, 400])
@pytest.mark.parametrize("vocab", [4097, 8193, 16385, 32776])
def test_uneven_pieces_of_a_cluster(moe, rows, vocab):
    """The last CTA of a cluster has a piece of few or no scores and gives its maximum while the others still load;
    the row's largest score lies in the first piece, or in the last one."""
    t = torch()
    rng = np.random.default_rng(vocab)
    x = t.from_numpy(rng.standard_normal((rows, vocab)).astype(np.float32)).cuda()
    x[:, 3] = 9
    x[::2, -1] = 11
    want = [vocab - 1 if r % 2 == 0 else 3 for r in range(rows)]
    token = t.empty(rows, dtype=t.int32, device="cuda")
    u = t.full((rows,), 0.5, device="cuda")
    zero, k = t.zeros(rows, device="cuda"), t.ones(rows, dtype=t.int32, device="cuda")
    for _ in range(20):
        for kw in (dict(temperature=zero), dict(top_k=k), dict(top_p=zero + 0.01)):
            token.fill_(-5)
            moe.sample(x, u, token, **kw)
            assert token.tolist() == want, kw.keys()
