"""moe_token_logprobs on rows whose probability lies on few tokens, against its definition in 64 bits: results of either
sign's side of 0 and errors that a reference far from the maximum would leave."""
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


def score(moe, logits, tokens, top):
    t = torch()
    rows = logits.shape[0]
    o = dict(logprob=t.full((rows,), 9.0, device="cuda"), rank=t.full((rows,), 77, dtype=t.int32, device="cuda"),
             entropy=t.full((rows,), 9.0, device="cuda"))
    if top:
        o |= dict(top_ids=t.full((rows, top), 77, dtype=t.int32, device="cuda"),
                  top_logprobs=t.full((rows, top), 9.0, device="cuda"))
    moe.token_logprobs(logits, tokens, **o)
    return o


def exact(logits, tokens, top):
    """In 64 bits, with the mean distance to the maximum and the probability of all that is below it."""
    t = torch()
    z = logits.double()
    d = z - z.max(1, keepdim=True).values
    w = d.exp()
    below = t.where(d < 0, w, 0).sum(1)
    s = w.sum(1)
    # log S = log(number of maxima) + log1p(below / that): below itself is what a sum next to 1 would lose.
    n = (d == 0).sum(1)
    log_s = n.double().log() + (below / n).log1p()
    far = -(w * d).sum(1) / s
    at = tokens.long()[:, None]
    o = dict(logprob=d.gather(1, at)[:, 0] - log_s, entropy=log_s + far, far=far, below=below / s, d=d.gather(1, at)[:, 0])
    if top:
        order = d.sort(dim=1, descending=True, stable=True)
        o |= dict(top_ids=order.indices[:, :top], top_logprobs=order.values[:, :top] - log_s[:, None], top_d=order.values[:, :top])
    return o


def check(moe, logits, tokens, top):
    """The error of log S, relative of S: the exponential of a weight errs by 2^-22, and so do factors by which sums move
    to a larger reference (three at most: of a thread's, a warp's and a CTA's sums, each on probability below the maximum);
    an argument, by 2^-24 of its size in base 2 and 2^-26 for the constant, 2^-23 |z - m| together; additions of a lane
    (its share of the row is 1 / 256 at least, in eights) and of 18 joins by 2^-24 each, but never by more than what they
    add, which is at most `below` next to the maximum.  A logit's own log probability adds its argument's error and one
    rounding each of two differences and a product.  Entropy's second sum has the same terms times |z - m|, taken from a
    reference up to 3 below the maximum where no maximum stands that much above the others."""
    t = torch()
    got, want = score(moe, logits, tokens, top), exact(logits, tokens, top)
    vocab = logits.shape[1]
    far, below = want["far"], want["below"]
    adds = 2.0 ** -24 * (vocab / 256 + 8 + 18)
    s = 2.0 ** -22 * (1 + 3 * below) + 2.0 ** -23 * far + t.minimum(t.full_like(below, adds), 2 * below)
    own = 2.0 ** -22

    def near(a, b, tol):
        a = a.double()
        assert t.all((a - b).abs() <= tol), float(((a - b).abs() - tol).max())

    near(got["logprob"], want["logprob"], s + own * (0.5 + want["d"].abs()) * (want["d"] < 0) + 2.0 ** -23 * want["logprob"].abs())
    peaked = (logits.double().sort(1, descending=True).values[:, :2].diff(dim=1)[:, 0] < -3) if vocab > 1 else below == 0
    near(got["entropy"], want["entropy"],
         s + (2.0 ** -22 + adds + 2.0 ** -23 * far) * t.where(peaked, far, far + 3) + 2.0 ** -23 * want["entropy"])
    assert t.all(got["logprob"] <= 0) and t.all(got["entropy"] >= 0)
    if top:
        assert t.equal(got["top_ids"].long(), want["top_ids"]) and t.all(got["top_logprobs"] <= 0)
        near(got["top_logprobs"], want["top_logprobs"], s[:, None] + own * (0.5 + want["top_d"].abs()) * (want["top_d"] < 0) +
             2.0 ** -23 * want["top_logprobs"].abs())
    return got, want


SIZES = [(3, 300), (330, 300), (330, 1000), (3, 5000), (330, 9001), (5, 40001), (310, 40001), (2, 163840), (306, 163840)]


def background(rows, vocab, seed, dtype):
    """Logits in [-3, 0]."""
    t = torch()
    x = t.rand(rows, vocab, generator=t.Generator("cuda").manual_seed(seed), device="cuda") * -3
    return x.to(t.float32 if dtype == "f32" else t.bfloat16)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", SIZES)
@pytest.mark.parametrize("top", [0, 20])
def test_one_token_above_the_rest(moe, dtype, rows, vocab, top):
    """One token 1.5 to 60 above the others, anywhere in the row.  From 28 on nothing but 2^-21 is left to err."""
    t = torch()
    x = background(rows, vocab, vocab + rows, dtype)
    rng = np.random.default_rng(rows * vocab)
    at = t.from_numpy(rng.integers(0, vocab, rows)).cuda()
    at[::3] = t.from_numpy(rng.integers(vocab * 9 // 10, vocab, len(range(0, rows, 3)))).cuda()  # behind the first tile, in long rows
    up = t.tensor([39.0, 28.0, 33.0, 25.0, 39.875, 15.0, 10.0, 30.0, 3.0, 8.0, 41.0, 1.5, 60.0, 2.0], device="cuda")
    up = up[t.arange(rows, device="cuda") % len(up)]
    for shift in (0.0, 17.0, -200.0):
        z = x.float() + shift
        z[t.arange(rows), at] = up + shift
        z = z.to(x.dtype)
        got, want = check(moe, z, at.int(), top)
        sure = up >= 28
        for k in ("logprob", "entropy"):
            assert t.all((got[k].double() - want[k]).abs()[sure] <= 2.0 ** -21)
        assert t.all(got["rank"][up >= 1.5] == 0)
        other = (at + 1) % vocab  # unlikely tokens
        check(moe, z, other.int(), top)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(3, 5000), (330, 9001), (2, 163840), (306, 163840)])
def test_rows_that_rise(moe, dtype, rows, vocab):
    """The first tile at 0 and the rest near 39; steps of 1.9 and of 5 up to 39; one long rise; two equal maxima 30 above."""
    t = torch()
    i = t.arange(vocab, device="cuda").float() / vocab
    x = background(rows, vocab, 3 * vocab, dtype).float()
    kinds = [t.where(i * vocab < 8192 if vocab > 8192 else i < 0.1, 0.0, 39.0), (i * 20).floor() * 1.9, (i * 8).floor() * 5, 39 * i]
    for r in range(rows):
        x[r] = x[r] * 0.2 + kinds[r % 5] if r % 5 < 4 else x[r]
    at = t.from_numpy(np.random.default_rng(vocab).integers(0, vocab, rows)).cuda()
    pair = t.from_numpy(np.arange(4, rows, 5)).cuda()
    x[pair, at[pair]] = 30.0
    x[pair, vocab - 1 - at[pair]] = 30.0
    z = x.to(t.float32 if dtype == "f32" else t.bfloat16)
    check(moe, z, at.int(), 0)
    check(moe, z, at.int(), 5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_and_infinite_rows_keep_to_their_side_of_zero(moe, dtype):
    """Rows masked with -inf, or with the type's lowest value, but for one to three tokens."""
    t = torch()
    dt = t.float32 if dtype == "f32" else t.bfloat16
    for vocab in (1000, 40001):
        x = t.full((12, vocab), float("-inf"), device="cuda", dtype=dt)
        x[6:] = t.finfo(dt).min
        rng = np.random.default_rng(vocab)
        at = t.zeros(12, dtype=t.int32, device="cuda")
        for r in range(12):
            n = r % 3 + 1
            pick = np.sort(rng.choice(vocab, n, replace=False))
            x[r, t.from_numpy(pick).cuda()] = t.tensor(rng.standard_normal(n) * 30, device="cuda").to(dt)
            at[r] = int(x[r].float().argmax())
        o = score(moe, x, at, 3)
        z = x.double()
        lp = t.log_softmax(z, 1)
        p = lp.exp()
        h = -t.where(p > 0, p * lp, 0).sum(1)
        assert t.all(o["logprob"] <= 0) and t.all(o["entropy"] >= 0) and t.all(o["top_logprobs"] <= 0)
        # One to three terms: their exponentials, arguments of up to 2^-23 60 under their probability, and few additions.
        assert t.all((o["logprob"].double() - lp.gather(1, at.long()[:, None])[:, 0]).abs() <= 2.0 ** -19)
        assert t.all((o["entropy"].double() - h).abs() <= 2.0 ** -18)
