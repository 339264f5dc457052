"""moe_prefix_attention against its definition in 64 bits."""
import numpy as np
import pytest

from serve_ref import Paged, attend, bf16, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch().cuda.is_available():
        pytest.skip("no CUDA device")
    import mxfp4_routed_expert_moe_gb300 as m
    return m


class Case:
    def __init__(self, moe, seed, q_lens, lens, prefix, page, hq, hk, dim, single=False, head_major=False, amp=1.0,
                 max_q=None, capacity=0):
        t = torch()
        rng = np.random.default_rng(seed)
        self.moe, self.q_lens, self.lens, self.prefix, self.hq, self.hk, self.dim = moe, q_lens, lens, prefix, hq, hk, dim
        pg = self.pg = Paged(rng, lens, prefix, page, hk, dim, head_major=head_major, capacity=capacity)
        self.kp, kp = bf16(rng.standard_normal((prefix, hk, dim)))
        self.vp, vp = bf16(rng.standard_normal((prefix, hk, dim)))
        if prefix:
            pg.fill(pg.prefix_table, prefix, self.kp, self.vp)
        self.keys, self.values = [], []
        for b, n in enumerate(lens):
            k, kd = bf16(rng.standard_normal((n, hk, dim)))
            v, vd = bf16(rng.standard_normal((n, hk, dim)))
            if n:
                pg.fill(pg.table[b], n, k, v)
            self.keys.append(np.concatenate([kp, kd]))
            self.values.append(np.concatenate([vp, vd]))
        self.n = sum(q_lens)
        # Rows of a wider projection.
        wide, _ = bf16(rng.standard_normal((self.n, hq * dim + 64)) * amp)
        self.q = wide[:, : hq * dim].view(self.n, hq, dim)
        self.qd = self.q.double().cpu().numpy()
        start = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        self.batch = moe.KVBatch(t.tensor(lens, dtype=t.int32, device="cuda"), t.from_numpy(pg.table).cuda(),
                                 tokens=self.n, q_start=None if single else t.from_numpy(start).cuda(),
                                 max_q=max_q or max(q_lens), prefix_len=prefix,
                                 prefix_table=t.from_numpy(pg.prefix_table).cuda() if prefix else None)
        self.cache = moe.KVCache(pg.k, pg.v)
        self.ws = t.full((moe.attention_workspace_bytes(self.cache, self.batch, hq),), 0xFF, dtype=t.uint8, device="cuda")

    def run(self, scale=None, stream=None):
        t = torch()
        out = t.full((self.n, self.hq, self.dim), 9.0, dtype=t.bfloat16, device="cuda")
        lse = t.full((self.n, self.hq), 9.0, device="cuda")
        status = t.zeros(1, dtype=t.int32, device="cuda")
        self.moe.prefix_attention(self.cache, self.batch, self.q, out, self.ws, scale=scale, lse=lse, status=status,
                                  stream=stream)
        t.cuda.synchronize()
        assert int(status.item()) == 0
        return out, lse

    def check(self, scale=None):
        out, lse = self.run(scale)
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        scale = self.dim ** -0.5 if scale is None else scale
        grp = self.hq // self.hk
        n0 = 0
        for b, ql in enumerate(self.q_lens):
            vis = [self.prefix + max(0, self.lens[b] - ql + 1 + i) for i in range(ql)]
            for h in range(self.hq):
                ref, rl, weight, mag = attend(self.qd[n0:n0 + ql, h], self.keys[b][:, h // grp], self.values[b][:, h // grp],
                                              vis, scale)
                # A score's error: the fp32 sum of dim products, then the product with scale log2 e; the
                # approximate 2^x adds 2^-22 relative.  Each weight enters the second product rounded to
                # bf16 (2^-8 relative at most), and so does the result.
                e = (self.dim + 4) * 2.0 ** -24 * scale * mag + 2.0 ** -20
                tol = 1.01 * 2.0 ** -8 * (weight + np.abs(ref)) + 2 * e[:, None] * weight + 1e-30
                err = np.abs(out[n0:n0 + ql, h] - ref)
                assert np.all(err <= tol), (b, h, (err / tol).max())
                empty = np.isinf(rl)
                got = lse[n0:n0 + ql, h]
                assert np.array_equal(np.isneginf(got), empty)
                assert np.all(np.abs(got[~empty] - rl[~empty]) <= e[~empty] + 2.0 ** -21 * (1 + np.abs(rl[~empty])))
            n0 += ql


# q_lens, own lengths, prefix, page, q heads, kv heads, dim, one-token form, head-major cache
CASES = {
    "one": ([1], [1], 0, 16, 1, 1, 64, True, False),
    "one_prefix_only": ([1, 1], [0, 0], 17, 16, 4, 2, 128, True, False),
    "empty_rows": ([1, 1, 1], [0, 5, 0], 0, 64, 14, 2, 128, True, False),
    "lengths": ([1] * 9, [1, 15, 16, 17, 63, 64, 65, 127, 300], 0, 16, 7, 1, 128, True, True),
    "prefix_and_own": ([1] * 3, [1, 64, 200], 130, 64, 56, 8, 128, True, False),
    "mha": ([1] * 4, [33, 5, 128, 70], 50, 32, 6, 6, 64, True, False),
    "group16": ([1] * 2, [1000, 130], 65, 128, 32, 2, 64, True, True),
    "group20": ([1] * 2, [100, 30], 31, 16, 20, 1, 128, True, False),
    "verify_8": ([8], [501], 0, 64, 56, 8, 128, False, False),
    "verify_ragged": ([8, 0, 1, 3], [8, 9, 40, 70], 20, 16, 14, 2, 128, False, False),
    "more_new_than_kept": ([4, 2], [2, 0], 0, 16, 4, 2, 64, False, False),
    "rows_64": ([8, 4], [130, 70], 0, 32, 16, 2, 64, False, False),
    "rows_33": ([33, 1], [33, 65], 70, 16, 2, 2, 128, False, True),
    "rows_many": ([70, 0, 129, 3], [70, 3, 300, 200], 150, 32, 8, 2, 128, False, False),
    "rows_many_64": ([200, 57], [333, 57], 1, 64, 6, 2, 64, False, False),
    "prefix_rows_100": ([1] * 100, [7] * 100, 300, 64, 2, 2, 128, True, False),
    "prefix_rows_300": ([1] * 150, list(range(150)), 257, 128, 4, 2, 64, True, False),
    "prefix_rows_520": ([2] * 65, [9] * 65, 700, 32, 8, 2, 128, False, True),
    "long_own": ([1], [9001], 0, 64, 8, 1, 128, True, False),
}


# Tables with room for many more tokens go to the kernels that split long sequences, narrow ones to the one for
# small problems.
LONG = 40000


@pytest.mark.parametrize("capacity", [0, LONG])
@pytest.mark.parametrize("name", CASES)
def test_attention(moe, name, capacity):
    q_lens, lens, prefix, page, hq, hk, dim, single, hm = CASES[name]
    c = Case(moe, sorted(CASES).index(name), q_lens, lens, prefix, page, hq, hk, dim, single=single, head_major=hm,
             capacity=capacity)
    c.check()


def test_large_scores_and_scale(moe):
    """Peaked rows (scores of tens) and another scale; one token takes nearly all the weight."""
    for rows, capacity in ((1, 0), (1, LONG), (40, LONG)):
        c = Case(moe, 5, [rows] * 2, [400, 90], 100, 32, 4, 2, 128, amp=8.0, capacity=capacity)
        c.check()
        c.check(scale=0.3)


def test_repeats_and_streams(moe):
    """The same bits from run to run, on another stream, and in a graph; a smaller max_q does not matter."""
    t = torch()
    for kw in (dict(q_lens=[1] * 40, lens=list(range(3, 43)), prefix=1000, capacity=LONG),
               dict(q_lens=[50, 3], lens=[77, 500], prefix=333, capacity=LONG),
               dict(q_lens=[2, 3], lens=[77, 500], prefix=333)):
        c = Case(moe, 11, page=32, hq=8, hk=2, dim=128, **kw)
        out, lse = c.run()
        side = t.cuda.Stream()
        side.wait_stream(t.cuda.current_stream())
        again, lse2 = c.run(stream=side)
        assert t.equal(out, again) and t.equal(lse, lse2)
        g = t.cuda.CUDAGraph()
        o3 = t.empty_like(out)
        with t.cuda.graph(g):
            moe.prefix_attention(c.cache, c.batch, c.q, o3, c.ws)
        for _ in range(2):
            o3.fill_(3)
            g.replay()
        t.cuda.synchronize()
        assert t.equal(o3, out)


def test_lengths_are_read_on_the_device(moe):
    """A captured call follows kv_len: the same graph after the sequences grew."""
    t = torch()
    for capacity in (0, LONG):
        check_follows_lengths(moe, Case(moe, 2, [1] * 3, [100, 64, 30], 40, 16, 8, 2, 64, single=True, capacity=capacity))


def check_follows_lengths(moe, c):
    t = torch()
    full = t.tensor(c.lens, dtype=t.int32, device="cuda")
    c.batch.kv_len.copy_(full - 25)
    out = t.empty(3, 8, 64, dtype=t.bfloat16, device="cuda")
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        moe.prefix_attention(c.cache, c.batch, c.q, out, c.ws)
    c.batch.kv_len.copy_(full)
    g.replay()
    t.cuda.synchronize()
    assert t.equal(out, c.run()[0])
    c.check()


def test_bad_entries_are_reported(moe):
    """A page id outside the cache, a length past the table, more new tokens than max_q: reported, never
    followed; the other sequences' results stand."""
    t = torch()
    for rows, capacity in ((1, 0), (1, LONG), (40, LONG)):
        for what in ("page", "length", "max_q"):
            c = Case(moe, 4, [rows] * 3, [50, 90, 70], 0, 16, 4, 2, 128, capacity=capacity)
            good, _ = c.run()
            if what == "page":
                c.batch.table[1, 2] = 1 << 20
            elif what == "length":
                c.batch.kv_len[1] = 16 * c.batch.table.shape[1] + 1
            else:
                c.batch.q_start.copy_(t.tensor([0, rows, 2 * rows + 1, 3 * rows], dtype=t.int32))
            out = t.empty_like(good)
            status = t.zeros(1, dtype=t.int32, device="cuda")
            moe.prefix_attention(c.cache, c.batch, c.q, out, c.ws, status=status)
            t.cuda.synchronize()
            assert int(status.item()) == moe.MOE_ERR_DEVICE_CHECK, what
            assert t.equal(out[:rows], good[:rows])
            if what != "max_q":
                assert t.equal(out[2 * rows:], good[2 * rows:])


def test_waits_give_up_and_next_call_is_correct(moe):
    """With a limit of one cycle a real wait that does not find its phase complete gives up and is reported, and
    the next call is right.  The Tensor Memory kernel always has such a wait (for its own scores); a warp's
    units may have landed before it asks, so the other kernels may also finish, and then correctly."""
    t = torch()
    for must, kw in ((False, dict(q_lens=[1] * 4, lens=[6000, 200, 100, 5], prefix=0, capacity=LONG)),
                     (True, dict(q_lens=[50, 90], lens=[300, 200], prefix=500, capacity=LONG)),
                     (False, dict(q_lens=[1] * 60, lens=[600] * 60, prefix=100))):
        c = Case(moe, 6, page=64, hq=8, hk=2, dim=128, **kw)
        good, _ = c.run()
        out = t.empty_like(good)
        status = t.zeros(1, dtype=t.int32, device="cuda")
        try:
            moe.set_wait_limit(1)
            moe.prefix_attention(c.cache, c.batch, c.q, out, c.ws, status=status)
            t.cuda.synchronize()
        finally:
            moe.set_wait_limit(0)
        if must or int(status.item()) != 0:
            assert int(status.item()) == moe.MOE_ERR_TIMEOUT
        else:
            assert t.equal(out, good)
        c.check()


@pytest.mark.parametrize("dim,hk,prefix", [(128, 64, 3205), (64, 128, 3207)])
def test_prefix_longer_than_the_cache_on_the_chip(moe, dim, hk, prefix):
    """A prefix of more than 100 MB, two row tiles a key head: segments that begin inside their range."""
    c = Case(moe, 21, q_lens=[140, 3], lens=[150, 20], prefix=prefix, page=64, hq=2 * hk, hk=hk, dim=dim, capacity=LONG)
    c.check()
    a, la = c.run()
    b, lb = c.run()
    assert torch().equal(a, b) and torch().equal(la, lb)


def test_broken_starts_are_reported(moe):
    """q_start that falls (sequences would overlap, and their tiles be more than the workspace holds), or that
    leaves rows to no sequence: reported."""
    t = torch()
    for rows, capacity in ((1, 0), (1, LONG), (40, LONG), (300, LONG)):
        c = Case(moe, 6, [rows] * 8, [rows + 50] * 8, 33, 16, 4, 2, 64, capacity=capacity, max_q=8 * rows)
        good, lse = c.run()
        keep = c.batch.q_start.clone()
        for bad in ([0, 8 * rows] * 4 + [8 * rows], [0] * 8 + [7 * rows], [1] + [8 * rows] * 8):
            c.batch.q_start.copy_(t.tensor(bad, dtype=t.int32))
            out = t.empty_like(good)
            status = t.zeros(1, dtype=t.int32, device="cuda")
            moe.prefix_attention(c.cache, c.batch, c.q, out, c.ws, status=status)
            t.cuda.synchronize()
            assert int(status.item()) == moe.MOE_ERR_DEVICE_CHECK, bad
        c.batch.q_start.copy_(keep)
        again, lse2 = c.run()
        assert t.equal(good, again) and t.equal(lse, lse2)


@pytest.mark.parametrize("capacity", [0, LONG])
@pytest.mark.parametrize("hq,hk", [(3, 3), (14, 2), (56, 8)])
@pytest.mark.parametrize("q_lens,lens,prefix", [([2], [9], 32768), ([1, 1], [3, 40], 200), ([1], [0], 77), ([2, 0, 1], [5, 9, 1], 513)])
def test_max_q_far_above_the_new_tokens(moe, q_lens, lens, prefix, hq, hk, capacity):
    """max_q is an upper bound that a server may keep for all its steps: past the batch's new tokens, which are what
    the call knows without reading q_start, it changes no bit."""
    kw = dict(seed=31, q_lens=q_lens, lens=lens, prefix=prefix, page=64, hq=hq, hk=hk, dim=128, capacity=capacity)
    tight = Case(moe, max_q=sum(q_lens), **kw)
    out, lse = tight.run()
    if prefix < 1000:
        tight.check()
    for max_q in (8, 64, 5000):
        c = Case(moe, max_q=max_q, **kw)
        assert c.ws.numel() == tight.ws.numel()
        got, got_lse = c.run()
        assert torch().equal(got, out) and torch().equal(got_lse, lse)


def test_max_q_above_one_without_starts(moe):
    """Without q_start every sequence has one new token, whatever max_q says."""
    kw = dict(seed=32, q_lens=[1] * 2, lens=[70, 9], prefix=300, page=32, hq=14, hk=2, dim=64, single=True, capacity=LONG)
    c = Case(moe, max_q=8, **kw)
    c.check()
    got, want = c.run(), Case(moe, **kw).run()
    assert torch().equal(got[0], want[0]) and torch().equal(got[1], want[1])


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("capacity", [0, LONG])
def test_short_parts_in_turn_through_the_same_buffers(moe, dim, capacity):
    """Parts that end inside a unit, where the rows past the end are cleared, followed at once by others that refill
    the same buffers: the prefix's last unit before the own part's, and many short sequences in turn."""
    t = torch()
    for q_lens, lens, prefix in (([1] * 2, [200, 37], 233), ([1] * 700, [1 + (7 * i) % 50 for i in range(700)], 0),
                                 ([2] * 300, [2 + (11 * i) % 90 for i in range(300)], 17)):
        c = Case(moe, 41, q_lens, lens, prefix, 16, 6, 3, dim, capacity=capacity)
        c.check()
        out, lse = c.run()
        for _ in range(20):
            again, lse2 = c.run()
            assert t.equal(out, again) and t.equal(lse, lse2)


UNSEEN = {  # q_lens, own lengths, prefix, page, q heads, kv heads, dim, capacity
    "tile": ([8, 3], [40, 3], 50, 16, 14, 2, 128, 0),
    "tile_64": ([5, 16], [70, 30], 0, 16, 4, 4, 64, 0),
    "warps": ([2, 1, 2], [90, 33, 64], 20, 32, 14, 2, 128, LONG),
    "warps_64": ([16, 7], [64, 100], 0, 16, 3, 3, 64, LONG),
    "half": ([40], [333], 70, 64, 6, 2, 128, LONG),
    "both_halves": ([70, 0, 129], [70, 3, 300], 150, 32, 8, 2, 128, LONG),
    "many_tokens_a_tile": ([300, 40], [431, 40], 1, 128, 2, 2, 64, LONG),
}


@pytest.mark.parametrize("name", UNSEEN)
def test_values_that_a_row_does_not_see_do_not_reach_it(moe, name):
    """Infinities and NaN in the values of a new token reach the rows that see it, and no earlier one."""
    q_lens, lens, prefix, page, hq, hk, dim, capacity = UNSEEN[name]
    c = Case(moe, 51, q_lens, lens, prefix, page, hq, hk, dim, capacity=capacity)
    for b, ql in enumerate(q_lens):
        for n, i in enumerate({ql - 1, ql // 2, ql // 3 + 1}):
            j = lens[b] - ql + i
            if not 0 < i < ql or j < 0:
                continue
            for h in range(hk):
                for d, x in ((0, np.inf), (dim - 1, np.nan), ((17 + 5 * n + h) % dim, -np.inf), (40 + n, np.inf)):
                    c.pg.v[int(c.pg.table[b, j // page]), j % page, h, d] = float(x)
                    c.values[b][prefix + j, h, d] = x
    out, lse = c.run()
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    scale, grp, n0, seen = dim ** -0.5, hq // hk, 0, 0
    for b, ql in enumerate(q_lens):
        vis = [prefix + max(0, lens[b] - ql + 1 + i) for i in range(ql)]
        for h in range(hq):
            with np.errstate(invalid="ignore"):
                ref, rl, weight, mag = attend(c.qd[n0:n0 + ql, h], c.keys[b][:, h // grp], c.values[b][:, h // grp], vis, scale)
            got = out[n0:n0 + ql, h]
            fin = np.isfinite(ref)
            seen += (~fin).sum()
            assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(got[np.isinf(ref)], ref[np.isinf(ref)]), (b, h)
            # The tolerances of Case.check.
            e = (dim + 4) * 2.0 ** -24 * scale * mag + 2.0 ** -20
            tol = (1.01 * 2.0 ** -8 * (weight + np.abs(ref)) + 2 * e[:, None] * weight + 1e-30)[fin]
            assert np.all(np.abs(got[fin] - ref[fin]) <= tol), (b, h)
            assert np.all(np.abs(lse[n0:n0 + ql, h] - rl) <= e + 2.0 ** -21 * (1 + np.abs(rl)))
        n0 += ql
    assert seen > 0


@pytest.mark.parametrize("name", UNSEEN)
def test_keys_that_a_row_does_not_see_do_not_reach_it(moe, name):
    """The same of the keys: the last new token's are NaN; its own row is NaN, the others are as they were."""
    t = torch()
    q_lens, lens, prefix, page, hq, hk, dim, capacity = UNSEEN[name]
    c = Case(moe, 52, q_lens, lens, prefix, page, hq, hk, dim, capacity=capacity)
    good, glse = c.run()
    for b, n in enumerate(lens):
        if q_lens[b]:
            c.pg.k[int(c.pg.table[b, (n - 1) // page]), (n - 1) % page] = float("nan")
    out, lse = c.run()
    last = [int(x) - 1 for x in np.cumsum(q_lens) if x]
    rest = [i for i in range(c.n) if i not in last]
    assert t.equal(out[rest], good[rest]) and t.equal(lse[rest], glse[rest])
    assert out[last].isnan().all() and lse[last].isnan().all()
