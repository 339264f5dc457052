"""moe_kv_append against its definition in 64 bits."""
import numpy as np
import pytest

from serve_ref import Paged, rotate, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch().cuda.is_available():
        pytest.skip("no CUDA device")
    import mxfp4_routed_expert_moe_gb300 as m
    return m


# dtype, q_lens, own lengths, prefix, page, q heads, kv heads, dim, rot, interleaved, head-major cache, one-token form
CASES = [
    ("bf16", [1] * 8, [1, 64, 65, 16, 17, 128, 100, 63], 2048, 64, 56, 8, 128, 128, False, False, True),
    ("bf16", [1], [1], 0, 16, 1, 1, 64, 64, False, False, True),
    ("f32", [3, 0, 17, 1, 40], [3, 9, 20, 33, 40], 33, 16, 14, 2, 64, 32, True, True, False),
    ("f32", [5, 2], [70, 2], 1, 32, 5, 5, 128, 128, True, False, False),
    ("bf16", [33, 1, 0, 0, 90], [300, 1, 0, 5, 90], 7, 128, 8, 8, 128, 64, False, True, False),
    ("bf16", [2] * 700, [5] * 700, 3, 16, 4, 1, 64, 16, False, False, False),
    ("f32", [9], [11], 100000, 16, 2, 1, 64, 64, False, False, False),
    ("bf16", [4, 4], [4, 9], 0, 64, 3, 1, 128, 0, False, False, False),
]


@pytest.mark.parametrize("c", range(len(CASES)))
@pytest.mark.parametrize("with_q", [True, False])
def test_append(moe, c, with_q):
    t = torch()
    dtype, q_lens, lens, prefix, page, hq, hk, dim, rot, inter, hm, single = CASES[c]
    rng = np.random.default_rng(100 + c)
    pg = Paged(rng, lens, prefix, page, hk, dim, head_major=hm)
    n = sum(q_lens)
    dt = t.float32 if dtype == "f32" else t.bfloat16
    # One projection's rows: q, k and v are strided views of it.
    qkv = t.from_numpy(rng.standard_normal((n, (hq + 2 * hk) * dim), dtype=np.float32)).cuda().to(dt)
    q, k, v = (x.view(n, -1, dim) for x in qkv.split((hq * dim, hk * dim, hk * dim), 1))
    rope = moe.rope_table(prefix + max(lens), rot) if rot else None
    q_out = t.full((n, hq, dim), 7.0, dtype=t.bfloat16, device="cuda")
    status = t.zeros(1, dtype=t.int32, device="cuda")
    start = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    kv_len = t.tensor(lens, dtype=t.int32, device="cuda")
    batch = moe.KVBatch(kv_len, t.from_numpy(pg.table).cuda(), tokens=n,
                        q_start=None if single else t.from_numpy(start).cuda(), max_q=max(q_lens), prefix_len=prefix,
                        prefix_table=t.from_numpy(pg.prefix_table).cuda() if prefix else None)
    before_k, before_v = pg.k.clone(), pg.v.clone()
    moe.kv_append(moe.KVCache(pg.k, pg.v), batch, k, v, q=q if with_q else None, q_out=q_out if with_q else None,
                  rope=rope, rot_dim=rot, interleaved=inter, status=status)
    assert int(status.item()) == 0
    qd, kd, vd = (x.double().cpu().numpy() for x in (q, k, v))
    rd = rope.double().cpu().numpy() if rot else None
    seq = np.repeat(np.arange(len(lens)), q_lens)
    own = np.concatenate([np.arange(a - b, a) for a, b in zip(lens, q_lens)]) if n else np.zeros(0, int)
    want_k, want_q = rotate(kd, prefix + own, rd, rot, inter), rotate(qd, prefix + own, rd, rot, inter)

    def check(got, want, x):
        # fp32 products and sums (3 roundings of at most |a| + |b|, here <= 2 max|x|), then one rounding to
        # bf16's 8 significand bits.
        err = np.abs(got.double().cpu().numpy() - want)
        mag = np.abs(x).max(-1, keepdims=True)
        assert np.all(err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * mag + 1e-38), err.max()

    pages = t.from_numpy(pg.table[seq, own // page].astype(np.int64)).cuda()
    at = t.from_numpy(own % page).cuda()
    check(pg.k[pages, at], want_k, kd)
    assert t.equal(pg.v[pages, at], v.bfloat16())  # converted only: the same rounding
    if with_q:
        check(q_out, want_q, qd)
    else:
        assert t.all(q_out == 7)
    # Nothing else changed.
    before_k[pages, at] = 0
    before_v[pages, at] = 0
    pg.k[pages, at] = 0
    pg.v[pages, at] = 0
    assert t.equal(pg.k.contiguous().view(t.int16), before_k.contiguous().view(t.int16))
    assert t.equal(pg.v.contiguous().view(t.int16), before_v.contiguous().view(t.int16))


def test_append_in_place_on_another_stream(moe):
    """q_out may be q itself, and the work follows the given stream."""
    t = torch()
    rng = np.random.default_rng(7)
    pg = Paged(rng, [40, 3], 0, 16, 2, 128)
    n = 5
    qkv = t.from_numpy(rng.standard_normal((n, 12 * 128), dtype=np.float32)).cuda().bfloat16()
    q, k, v = (x.view(n, -1, 128) for x in qkv.split((8 * 128, 256, 256), 1))
    rope = moe.rope_table(64, 128)
    batch = moe.KVBatch(t.tensor([40, 3], dtype=t.int32, device="cuda"), t.from_numpy(pg.table).cuda(), tokens=n,
                        q_start=t.tensor([0, 2, 5], dtype=t.int32, device="cuda"), max_q=3)
    ref = t.empty(n, 8, 128, dtype=t.bfloat16, device="cuda")
    moe.kv_append(moe.KVCache(pg.k, pg.v), batch, k, v, q=q, q_out=ref, rope=rope, rot_dim=128)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    moe.kv_append(moe.KVCache(pg.k, pg.v), batch, k, v, q=q, q_out=q, rope=rope, rot_dim=128, stream=side)
    t.cuda.current_stream().wait_stream(side)
    assert t.equal(q, ref)


def test_append_reports_bad_entries_and_skips_them(moe):
    """A page id outside the cache, a position past the rope table, a length past the table row and a new
    token before the start of its sequence: each is reported, its token skipped, the others written."""
    t = torch()
    for what in ("page", "rope", "length", "before"):
        rng = np.random.default_rng(3)
        pg = Paged(rng, [5, 20, 7], 0, 16, 1, 64)
        lens, table, rows = [5, 20, 7], pg.table.copy(), 64
        if what == "page":
            table[1, 1] = pg.pages
        elif what == "rope":
            rows = 19  # position 19 of sequence 1
        elif what == "length":
            lens[1] = 2 * 16 + 1
        else:
            lens[1] = 0
        k = t.ones(3, 1, 64, dtype=t.bfloat16, device="cuda")
        status = t.zeros(1, dtype=t.int32, device="cuda")
        batch = moe.KVBatch(t.tensor(lens, dtype=t.int32, device="cuda"), t.from_numpy(table).cuda())
        moe.kv_append(moe.KVCache(pg.k, pg.v), batch, k, k, rope=moe.rope_table(rows, 64), rot_dim=64, status=status)
        assert int(status.item()) == moe.MOE_ERR_DEVICE_CHECK, what
        assert t.all(pg.v[int(table[0, 0]), 4] == 1) and t.all(pg.v[int(table[2, 0]), 6] == 1)
        assert int((pg.v == 1).sum()) == 2 * 64, what
