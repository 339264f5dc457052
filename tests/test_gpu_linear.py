"""moe_mx_linear against the product in 64 bits."""
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


def product(xv, wv):
    """Sum and sum of magnitudes."""
    return xv @ wv.T, np.abs(xv) @ np.abs(wv).T


def bound(kind, K, mag, y, out):
    """Error of a sum.  Products of the element types are exact; an MMA of 32 (E4M3) or 64 (E2M1) products and its
    accumulator err by at most 18 units of 2^-23 of their magnitudes (each addend aligned and cut, one rounding), and
    parts of a split sum add at most 8 roundings, the addend one; then one rounding to the output's type."""
    mmas = K // (32 if kind == "e4m3" else 64) + 1
    err = (18 * mmas + 9) * 2.0 ** -23 * mag
    return err + (2.0 ** -8 * (np.abs(y) + err) if out == "bf16" else 0) + 1e-37


CASES = [  # T, N, K, x kind, output, addend
    (1, 128, 128, "e4m3", "f32", False), (1, 128, 128, "e2m1", "f32", False), (1, 1, 128, "e2m1", "bf16", True),
    (1, 9216, 1408, "e4m3", "bf16", False), (3, 300, 256, "e2m1", "f32", True), (8, 7168, 1408, "e2m1", "bf16", True),
    (17, 129, 384, "e4m3", "f32", True), (64, 1408, 7168, "e4m3", "f32", True), (64, 1407, 7168, "e2m1", "bf16", False),
    (100, 515, 640, "e2m1", "f32", False), (128, 256, 128, "e4m3", "bf16", True), (129, 256, 512, "e4m3", "f32", False),
    (255, 777, 896, "e2m1", "f32", True), (256, 128, 16384, "e4m3", "f32", False), (257, 131, 256, "e2m1", "bf16", True),
    (700, 1000, 384, "e4m3", "bf16", False), (1021, 4099, 128, "e2m1", "f32", False), (513, 513, 1152, "e4m3", "f32", True),
    (2047, 700, 640, "e4m3", "bf16", True), (2048, 2560, 256, "e2m1", "bf16", False), (1500, 3333, 896, "e2m1", "f32", True),
    (4100, 1300, 128, "e4m3", "f32", False),
]


@pytest.mark.parametrize("T,N,K,kind,out,addend", CASES)
def test_linear(moe, T, N, K, kind, out, addend):
    t = torch()
    rng = np.random.default_rng(T + N + K)
    xc, xs = ref.random_mx(rng, T, K, kind)
    wc, ws = ref.random_mx(rng, N, K, "e2m1")
    x, w = ref.matrix(moe, xc, xs, kind), ref.matrix(moe, wc, ws, "e2m1")
    y, mag = product(ref.values(xc, xs, kind), ref.values(wc, ws, "e2m1"))
    dt = t.float32 if out == "f32" else t.bfloat16
    got = t.full((T, N), float("nan"), dtype=dt, device="cuda")
    add = None
    if addend:
        add = t.from_numpy(rng.standard_normal((T, N)).astype(np.float32) * 30).cuda().to(dt)
        y, mag = y + ref.host(add), mag + np.abs(ref.host(add))
    status = t.zeros(1, dtype=t.int32, device="cuda")
    moe.mx_linear(x, w, got, add=add, status=status)
    assert int(status.item()) == 0
    g = ref.host(got)
    assert np.all(np.abs(g - y) <= bound(kind, K, mag, y, out))
    # The same again, in place, and bit for bit.
    if addend:
        again = add.clone()
        moe.mx_linear(x, w, again, add=again)
    else:
        again = t.empty_like(got)
        moe.mx_linear(x, w, again)
    assert t.equal(again, got)


@pytest.mark.parametrize("T,N,K,kind", [(1, 300, 7168, "e2m1"), (40, 300, 7168, "e2m1"), (300, 513, 16384, "e2m1"),
                                        (2100, 1025, 7168, "e2m1"), (33, 129, 1408, "e4m3"), (2100, 1025, 1408, "e4m3")])
def test_sums_that_fit_are_exact(moe, T, N, K, kind):
    """Whole numbers of units: with equal scales the products are multiples of 2^-2 below 36 (E2M1) or, of E4M3 codes
    below 16 in whole steps, multiples of 2^-2 below 96, so that every partial sum is a multiple of 2^-2 below
    16384 x 36 < 2^20 or 1408 x 96 < 2^18: fp32 holds each, and aligning addends to 22 bits below the largest loses
    nothing."""
    t = torch()
    rng = np.random.default_rng(K + T)
    xc, xs = ref.random_mx(rng, T, K, kind, scales=np.full((T, K // 32), 127, dtype=np.uint8))
    if kind == "e4m3":  # 0, 0.5, ... 15.5 by their codes
        xc = ref.nearest(rng.integers(0, 32, (T, K)) / 2.0, kind).astype(np.uint8)
        whole = ref.GRID[kind][xc] * 2 == np.rint(ref.GRID[kind][xc] * 2)
        xc[~whole] = 0
        xc |= rng.integers(0, 2, (T, K)).astype(np.uint8) << 7
    wc, ws = ref.random_mx(rng, N, K, "e2m1", scales=np.full((N, K // 32), 125, dtype=np.uint8))
    got = t.empty(T, N, device="cuda")
    moe.mx_linear(ref.matrix(moe, xc, xs, kind), ref.matrix(moe, wc, ws, "e2m1"), got)
    assert np.array_equal(ref.host(got), ref.values(xc, xs, kind) @ ref.values(wc, ws, "e2m1").T)


@pytest.mark.parametrize("kind", ["e2m1", "e4m3"])
@pytest.mark.parametrize("T,N,K", [(2, 130, 256), (70, 257, 384), (1100, 1400, 384)])
def test_each_scale_reaches_its_block(moe, kind, T, N, K):
    """One-hot rows: x[t] picks column k_t of w, so that out[t][n] = x[t][k] w[n][k] with wide-spread scales."""
    t = torch()
    rng = np.random.default_rng(T * 3 + N)
    xc, xs = ref.random_mx(rng, T, K, kind, spread=20)
    pick = rng.integers(0, K, T)
    keep = np.zeros((T, K), dtype=bool)
    keep[np.arange(T), pick] = True
    xc[~keep] = 0
    wc, ws = ref.random_mx(rng, N, K, "e2m1", spread=20)
    got = t.empty(T, N, device="cuda")
    moe.mx_linear(ref.matrix(moe, xc, xs, kind, pad=1), ref.matrix(moe, wc, ws, "e2m1", pad=2), got)
    xv, wv = ref.values(xc, xs, kind), ref.values(wc, ws, "e2m1")
    assert np.array_equal(ref.host(got), xv[np.arange(T), pick][:, None] * wv[:, pick].T)


@pytest.mark.parametrize("kind", ["e2m1", "e4m3"])
@pytest.mark.parametrize("T,N,K", [(3, 200, 512), (300, 400, 256), (1100, 1400, 384)])
def test_nan_scales_and_codes(moe, kind, T, N, K):
    """A NaN in a row of x or w reaches that row's or column's results and no others, a zero against it included."""
    t = torch()
    rng = np.random.default_rng(T)
    xc, xs = ref.random_mx(rng, T, K, kind)
    wc, ws = ref.random_mx(rng, N, K, "e2m1")
    xs[1, K // 32 - 1] = 255
    ws[5, 0] = 255
    ws[N - 1, 3] = 255
    xc[2, :] = 0
    if kind == "e4m3":
        xc[0, 40] = 0x7F
    got = t.empty(T, N, device="cuda")
    moe.mx_linear(ref.matrix(moe, xc, xs, kind), ref.matrix(moe, wc, ws, "e2m1"), got)
    want = np.zeros((T, N), dtype=bool)
    want[1] = True
    want[:, [5, N - 1]] = True
    if kind == "e4m3":
        want[0] = True
    assert np.array_equal(np.isnan(ref.host(got)), want)


def test_extreme_scales(moe):
    """Scales 0 (2^-127) and 254 (2^127) whose product is in range; sums past fp32's range are infinite."""
    t = torch()
    for kind in ("e2m1", "e4m3"):
        one = {"e2m1": 2, "e4m3": 56}[kind]
        xc, wc = np.full((2, 128), one, dtype=np.uint8), np.full((4, 128), 2, dtype=np.uint8)
        xs, ws = np.full((2, 4), 0, dtype=np.uint8), np.full((4, 4), 254, dtype=np.uint8)
        xs[1] = 254
        got = t.empty(2, 4, device="cuda")
        moe.mx_linear(ref.matrix(moe, xc, xs, kind), ref.matrix(moe, wc, ws, "e2m1"), got)
        assert t.all(got[0] == 128) and t.all(got[1] == float("inf")), kind


@pytest.mark.parametrize("T,N", [(5, 200), (1030, 1290)])
def test_strided_output_graph_and_stream(moe, T, N):
    """out and add inside wider tensors with odd strides, on another stream, captured and replayed."""
    t = torch()
    rng = np.random.default_rng(9)
    K = 384
    xc, xs = ref.random_mx(rng, T, K, "e4m3")
    wc, ws = ref.random_mx(rng, N, K, "e2m1")
    x, w = ref.matrix(moe, xc, xs, "e4m3", pad=1), ref.matrix(moe, wc, ws, "e2m1")
    plain = t.empty(T, N, device="cuda")
    moe.mx_linear(x, w, plain)
    wide = t.full((T, N + 3), 2.0, device="cuda")
    add = t.randn(T, N + 5, device="cuda")
    out = wide[:, 1:1 + N]
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    graph = t.cuda.CUDAGraph()
    with t.cuda.stream(side):
        moe.mx_linear(x, w, out, add=add[:, 2:2 + N])
        with t.cuda.graph(graph, stream=side):
            moe.mx_linear(x, w, out, add=add[:, 2:2 + N])
    t.cuda.current_stream().wait_stream(side)
    assert t.equal(out, plain + add[:, 2:2 + N])
    assert t.all(wide[:, 0] == 2) and t.all(wide[:, 1 + N:] == 2)
    add.neg_()
    graph.replay()
    t.cuda.synchronize()
    assert t.equal(out, plain + add[:, 2:2 + N])


def test_rows_do_not_depend_on_others(moe):
    """A row's result among few and many others of the same tile shape: bit for bit."""
    t = torch()
    rng = np.random.default_rng(4)
    K, N = 1408, 640
    xc, xs = ref.random_mx(rng, 16, K, "e4m3")
    wc, ws = ref.random_mx(rng, N, K, "e2m1")
    w = ref.matrix(moe, wc, ws, "e2m1")
    all_rows = t.empty(16, N, device="cuda")
    moe.mx_linear(ref.matrix(moe, xc, xs, "e4m3"), w, all_rows)
    for r in (0, 7, 15):
        one = t.empty(1, N, device="cuda")
        moe.mx_linear(ref.matrix(moe, xc[r:r + 1], xs[r:r + 1], "e4m3"), w, one)
        assert t.equal(one[0], all_rows[r])


def test_a_wait_that_runs_out_is_reported(moe):
    """With a limit of one cycle for waits the call ends and says so; the next call is as ever."""
    t = torch()
    rng = np.random.default_rng(6)
    for T, N, K in ((4, 512, 7168), (1024, 2048, 1024)):
        xc, xs = ref.random_mx(rng, T, K, "e4m3")
        wc, ws = ref.random_mx(rng, N, K, "e2m1")
        x, w = ref.matrix(moe, xc, xs, "e4m3"), ref.matrix(moe, wc, ws, "e2m1")
        good, out = t.empty(T, N, device="cuda"), t.empty(T, N, device="cuda")
        moe.mx_linear(x, w, good)
        status = t.zeros(1, dtype=t.int32, device="cuda")
        moe.set_wait_limit(1)
        try:
            moe.mx_linear(x, w, out, status=status)
            t.cuda.synchronize()
        finally:
            moe.set_wait_limit(0)
        assert int(status.item()) == moe.MOE_ERR_TIMEOUT
        status.zero_()
        moe.mx_linear(x, w, out, status=status)
        assert int(status.item()) == 0 and t.equal(out, good)


@pytest.mark.parametrize("T,N,K,kind", [(65536, 130, 128, "e2m1"), (65536, 257, 256, "e4m3"), (3, 262144, 128, "e4m3"), (300, 262144, 128, "e2m1"),
                                        (1, 1, 16384, "e4m3"), (2000, 1, 256, "e2m1"), (9000, 3, 128, "e4m3"),
                                        (30, 45001, 2048, "e4m3"), (1, 60000, 2176, "e4m3"), (7, 30000, 384, "e2m1"), (100, 9300, 384, "e4m3"),
                                        (64, 19332, 256, "e4m3")])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_largest_and_thinnest(moe, T, N, K, kind, out):
    """The largest counts of rows and results, and single columns, with one addend for all rows; rows at both ends and in
    between are compared."""
    t = torch()
    rng = np.random.default_rng(T + N)
    xc, xs = ref.random_mx(rng, T, K, kind)
    wc, ws = ref.random_mx(rng, N, K, "e2m1")
    dt = t.float32 if out == "f32" else t.bfloat16
    bias = t.from_numpy(rng.standard_normal((1, N)).astype(np.float32) * 30).cuda().to(dt)
    got = t.full((T, N), float("nan"), dtype=dt, device="cuda")
    moe.mx_linear(ref.matrix(moe, xc, xs, kind), ref.matrix(moe, wc, ws, "e2m1"), got, add=bias.expand(T, N))
    assert not got.isnan().any()
    r = np.unique(np.r_[np.arange(min(T, 70)), rng.integers(0, T, 60), np.arange(max(T - 70, 0), T)])
    c = np.unique(np.r_[np.arange(min(N, 300)), rng.integers(0, N, 60), np.arange(max(N - 300, 0), N)])
    y, mag = product(ref.values(xc[r], xs[r], kind), ref.values(wc[c], ws[c], "e2m1"))
    b = ref.host(bias)[:, c]
    y, mag = y + b, mag + np.abs(b)
    assert np.all(np.abs(ref.host(got[r][:, c]) - y) <= bound(kind, K, mag, y, out))


def test_calls_at_once_on_two_streams(moe):
    """Products of both forms side by side on two streams, many times, one of them captured: the same bits."""
    t = torch()
    rng = np.random.default_rng(12)
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    jobs = []
    for T, N, K, kind in ((3, 7168, 2048, "e4m3"), (1100, 2600, 512, "e2m1"), (40, 1300, 7168, "e4m3"), (500, 7168, 256, "e4m3")):
        xc, xs = ref.random_mx(rng, T, K, kind)
        wc, ws = ref.random_mx(rng, N, K, "e2m1")
        x, w = ref.matrix(moe, xc, xs, kind), ref.matrix(moe, wc, ws, "e2m1")
        want = t.empty(T, N, device="cuda")
        moe.mx_linear(x, w, want)
        jobs.append((x, w, want, [t.zeros_like(want) for _ in streams]))
    status = t.zeros(1, dtype=t.int32, device="cuda")
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph, stream=streams[0]):
        for x, w, _, outs in jobs:
            moe.mx_linear(x, w, outs[0], status=status)
    t.cuda.synchronize()
    for _ in range(20):
        with t.cuda.stream(streams[0]):
            graph.replay()
        for x, w, _, outs in reversed(jobs):
            moe.mx_linear(x, w, outs[1], status=status, stream=streams[1])
    t.cuda.synchronize()
    assert int(status.item()) == 0
    for _, _, want, outs in jobs:
        assert all(t.equal(o, want) for o in outs)
