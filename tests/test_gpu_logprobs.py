"""moe_token_logprobs against its definition in 64 bits."""
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


def expected(z, tokens, top):
    """Row by row in 64 bits: logprob, rank, entropy, top ids, top log probabilities, and mean |z - m| under p."""
    rows, vocab = z.shape
    out = {"logprob": np.full(rows, -np.inf), "rank": np.full(rows, -1), "entropy": np.zeros(rows),
           "ids": np.full((rows, top), -1), "lp": np.full((rows, top), -np.inf), "far": np.zeros(rows)}
    for r in range(rows):
        x = np.where(np.isnan(z[r]), -np.inf, z[r])
        m = x.max()
        order = np.argsort(-x, kind="stable")
        if np.isinf(m) and m > 0:
            lp = np.where(x == np.inf, -np.log((x == np.inf).sum()), -np.inf)
            out["entropy"][r] = np.log((x == np.inf).sum())
        elif m == -np.inf:
            lp = x
        else:
            d = x - m
            w = np.exp(d)
            s = w.sum()
            lp = d - np.log(s)
            d0 = np.where(w > 0, d, 0)
            out["far"][r] = -(w * d0).sum() / s
            out["entropy"][r] = np.log(s) + out["far"][r]
        listed = [i for i in order[:top] if x[i] > -np.inf]
        out["ids"][r, :len(listed)] = listed
        out["lp"][r, :len(listed)] = lp[listed]
        if tokens is not None and 0 <= tokens[r] < vocab:
            out["logprob"][r] = lp[tokens[r]]
            out["rank"][r] = int(np.nonzero(order == tokens[r])[0][0])
    return out


def run(moe, logits, tokens, top):
    t = torch()
    rows = logits.shape[0]
    f32, i32 = dict(device="cuda"), dict(device="cuda", dtype=t.int32)
    o = dict(logprob=t.full((rows,), 9.0, **f32), rank=t.full((rows,), 77, **i32), entropy=t.full((rows,), 9.0, **f32))
    if top:
        o |= dict(top_ids=t.full((rows, top), 77, **i32), top_logprobs=t.full((rows, top), 9.0, **f32))
    moe.token_logprobs(logits, t.tensor(tokens, **i32), **o)
    return {k: v.cpu().numpy().astype(np.float64 if v.dtype == t.float32 else np.int64) for k, v in o.items()}


def check(moe, logits, tokens, top):
    got, want = run(moe, logits, tokens, top), expected(ref.host(logits), tokens, top)
    vocab = logits.shape[1]
    assert np.array_equal(got["rank"], want["rank"])
    if top:
        assert np.array_equal(got["top_ids"], want["ids"])
    # log S: a thread adds up to vocab / 512 terms one after the other and rescales them where its maximum grows, lanes,
    # warps and CTAs add 12 more (3 roundings each); a term errs by 2^-22 (the exponential) and by 2^-23 |z - m| (its
    # argument), the latter by its mean under p.  Entropy's second sum has the same terms times |z - m|.
    unit = 2.0 ** -24 * (2 * vocab / 512 + 48 + 2 * want["far"])

    def near(a, b, tol):
        inf = np.isinf(b)
        assert np.array_equal(a[inf], b[inf])
        a, b, tol = a[~inf], b[~inf], np.broadcast_to(tol, inf.shape)[~inf]
        assert np.all(np.abs(a - b) <= tol + 2.0 ** -23 * np.abs(b)), np.abs(a - b).max()

    near(got["logprob"], want["logprob"], unit)
    near(got["entropy"], want["entropy"], unit * (2 + want["far"]))
    if top:
        near(got["top_logprobs"], want["lp"], unit[:, None])


def rows_of(rng, rows, vocab, dtype):
    t = torch()
    x = rng.standard_normal((rows, vocab)) * 2.5
    for _ in range(8):
        x[np.arange(rows), rng.integers(0, vocab, rows)] += rng.random(rows) * 10
    return t.from_numpy(x.astype(np.float32)).cuda().to(t.float32 if dtype == "f32" else t.bfloat16)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab,top", [(1, 1, 1), (1, 1, 0), (3, 5, 8), (2, 33, 32), (1, 100003, 5), (8, 4099, 20), (70, 1000, 32),
                                            (200, 16387, 1), (40, 50000, 20), (700, 2049, 3), (1, 262144, 32), (160, 163840, 20)])
def test_rows(moe, dtype, rows, vocab, top):
    rng = np.random.default_rng(rows + vocab)
    x = rows_of(rng, rows, vocab, dtype)
    tokens = rng.integers(0, vocab, rows)
    tokens[::5] = ref.host(x).argmax(1)[::5]
    if rows > 3:
        tokens[1], tokens[2], tokens[3] = -1, vocab, vocab - 1
    check(moe, x, tokens, top)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [300, 5000, 40001])
def test_awkward_rows(moe, dtype, vocab):
    """Constant, sorted, masked, infinite and NaN rows, ties at the cut, far maxima, -0 against 0."""
    t = torch()
    rng = np.random.default_rng(vocab)
    x = rng.standard_normal((18, vocab)).astype(np.float32)
    x[0] = 0.25
    x[1] = np.arange(vocab) * 0.001                    # every logit is the best so far
    x[2] = -np.arange(vocab) * 0.001
    x[3] = -np.inf
    x[4] = np.nan
    x[5, :] = -np.inf
    x[5, vocab // 2] = 3                               # all but one masked
    x[6, :] = np.finfo(np.float32).min                 # masked by the type's lowest value
    x[6, [1, vocab - 1]] = 1, 2
    x[7, [3, vocab - 2]] = np.inf
    x[8, rng.integers(0, vocab, vocab // 3)] = np.nan
    x[9] = rng.integers(-2, 3, vocab)                  # many ties
    x[10, vocab // 3] = 1000
    x[11] *= 1e30
    x[12] = np.where(np.arange(vocab) % 2, -0.0, 0.0)
    x[13] = np.where(np.arange(vocab) < vocab - 20, -np.inf, x[13])
    x[14] = np.abs(x[14]) * -1e-40
    x[15] = np.inf
    x[16] = 88.0 + 5 * x[16]
    x[17, 0] = -np.inf
    logits = t.from_numpy(x).cuda().to(t.float32 if dtype == "f32" else t.bfloat16)
    tokens = rng.integers(0, vocab, 18)
    tokens[[5, 6, 7, 12, 13, 17]] = vocab // 2, 1, 3, vocab // 2, 7, 0
    for top in (1, 20, 32):
        check(moe, logits, tokens, top)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_misaligned_strided_rows(moe, dtype):
    """Rows that begin at any element; what lies outside them is not looked at."""
    t = torch()
    rng = np.random.default_rng(3)
    wide = rows_of(rng, 9, 3011, dtype)
    wide[:, :3], wide[:, 3 + 3001:] = float("inf"), float("inf")
    x = wide[:, 3:3 + 3001]
    check(moe, x, rng.integers(0, 3001, 9), 10)
    check(moe, x.flip(0)[:4].contiguous()[1:], rng.integers(0, 3001, 3), 10)


def test_outputs_one_by_one_and_repeat(moe):
    """Each output alone gives what all together give, again and again, on another stream and in a graph."""
    t = torch()
    rng = np.random.default_rng(8)
    x = rows_of(rng, 33, 20011, "bf16")
    tokens = t.tensor(rng.integers(0, 20011, 33), dtype=t.int32, device="cuda")
    all_ = run(moe, x, tokens.tolist(), 7)
    f32, i32 = dict(device="cuda"), dict(device="cuda", dtype=t.int32)
    entropy = t.empty(33, **f32)
    moe.token_logprobs(x, entropy=entropy)
    assert np.array_equal(ref.host(entropy), all_["entropy"])
    rank = t.empty(33, **i32)
    moe.token_logprobs(x, tokens, rank=rank)
    assert np.array_equal(rank.cpu().numpy(), all_["rank"])
    ids, lp, logprob = t.empty(33, 7, **i32), t.empty(33, 7, **f32), t.empty(33, **f32)
    moe.token_logprobs(x, top_ids=ids, top_logprobs=lp)
    assert np.array_equal(ids.cpu().numpy(), all_["top_ids"]) and np.array_equal(ref.host(lp), all_["top_logprobs"])
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    graph = t.cuda.CUDAGraph()
    with t.cuda.stream(side):
        with t.cuda.graph(graph, stream=side):
            moe.token_logprobs(x, tokens, logprob)
    t.cuda.current_stream().wait_stream(side)
    graph.replay()
    t.cuda.synchronize()
    assert np.array_equal(ref.host(logprob), all_["logprob"])
    x.copy_(rows_of(rng, 33, 20011, "bf16"))
    graph.replay()
    t.cuda.synchronize()
    assert np.array_equal(ref.host(logprob), run(moe, x, tokens.tolist(), 0)["logprob"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("token_at", [0, 7, 900, 2999])
def test_signed_zeros_are_equal(moe, dtype, token_at):
    """0 and -0 tie, whichever of them the token's is: the index decides."""
    t = torch()
    vocab = 3001
    x = np.full((4, vocab), -1.0, dtype=np.float32)
    x[0, ::3], x[1, ::3] = 0.0, -0.0
    x[2], x[3] = np.where(np.arange(vocab) % 2, -0.0, 0.0), np.where(np.arange(vocab) % 2, 0.0, -0.0)
    x[0, token_at], x[1, token_at] = -0.0, 0.0
    logits = t.from_numpy(x).cuda().to(t.float32 if dtype == "f32" else t.bfloat16)
    check(moe, logits, np.full(4, token_at), 20)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [37, 999, 2048, 2049, 9001, 16384])
def test_awkward_rows_among_many(moe, dtype, vocab):
    """Batches whose rows are short take smaller groups of threads: the same rows there, in turn."""
    t = torch()
    rng = np.random.default_rng(vocab)
    rows = 330
    x = rng.standard_normal((rows, vocab)).astype(np.float32)
    at = np.arange(vocab)
    for r in range(0, rows, 11):
        x[r] = 0.25
        x[r + 1] = at * 0.001
        x[r + 2] = at * -0.001
        x[r + 3] = -np.inf
        x[r + 4] = np.where(at == (r * 17) % vocab, 3, -np.inf)
        x[r + 5] = np.finfo(np.float32).min
        x[r + 5, r % vocab] = 1
        x[r + 6, [r % vocab, vocab - 1]] = np.inf
        x[r + 7, rng.integers(0, vocab, vocab // 3)] = np.nan
        x[r + 8] = rng.integers(-2, 3, vocab)
        x[r + 9] *= 1e30
    logits = t.from_numpy(x).cuda().to(t.float32 if dtype == "f32" else t.bfloat16)
    tokens = rng.integers(0, vocab, rows)
    tokens[5::22] = np.arange(5, rows, 22) % vocab
    for top in (1, 32):
        check(moe, logits, tokens, top)
