"""moe_mx_quantize, moe_mx_dequantize and moe_rms_norm against their definitions in 64 bits."""
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


def dtype_of(name):
    return {"f32": torch().float32, "bf16": torch().bfloat16}[name]


def awkward(rng, rows, cols):
    """Values of many sizes, with whole blocks of zeros, of ties, of subnormal and of the largest numbers."""
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-20, 20, (rows, cols // 32)).repeat(32, 1))
    blocks = x.reshape(rows, -1, 32)
    special = [np.zeros(32), np.full(32, -0.0), np.linspace(-7, 7, 32), np.arange(-16, 16) / 4.0, np.arange(32) * 14.5 + 1,
               np.full(32, 3.0e38), np.full(32, 1e-40), np.r_[1e-39, np.zeros(31)], np.r_[448.0, np.full(31, 2.0 ** -9)],
               np.r_[7.99, np.full(31, 0.25)], np.r_[480.0, np.full(31, 464.0)], np.full(32, -6.0)]
    flat = blocks.reshape(-1, 32)
    for i, b in enumerate(special):
        if i < len(flat):
            flat[(i * 7) % len(flat)] = b
    return flat.reshape(rows, cols)


@pytest.mark.parametrize("kind", ["e2m1", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 7168), (3, 96), (61, 1408), (300, 128), (7, 16384)])
def test_quantize_gives_the_defined_bytes(moe, kind, dtype, rows, cols):
    t = torch()
    rng = np.random.default_rng(rows * cols)
    x = t.from_numpy(awkward(rng, rows, cols).astype(np.float32)).cuda().to(dtype_of(dtype))
    out = moe.MXMatrix.empty(rows, cols, kind)
    out.q.fill_(0x55), out.s.fill_(0x55)
    moe.mx_quantize(x, out)
    code, s = ref.quantize(ref.host(x), kind)
    assert np.array_equal(out.s.cpu().numpy(), s)
    assert np.array_equal(out.q.cpu().numpy(), ref.pack(code, kind))
    # And back: fp32 holds every value that is in its range, bf16 rounds it once.
    want = ref.values(code, s, kind)
    for back in ("f32", "bf16"):
        y = t.empty(rows, cols, dtype=dtype_of(back), device="cuda")
        moe.mx_dequantize(out, y)
        exact = t.from_numpy(want).cuda().float().to(dtype_of(back))
        assert t.equal(y, exact)


@pytest.mark.parametrize("kind", ["e2m1", "e4m3"])
def test_blocks_with_infinities_or_nan_read_as_nan(moe, kind):
    t = torch()
    x = t.randn(4, 128, device="cuda")
    x[0, 5], x[1, 40], x[2, 96], x[3, 127] = float("inf"), float("-inf"), float("nan"), float("inf")
    out = moe.MXMatrix.empty(4, 128, kind)
    moe.mx_quantize(x, out)
    bad = t.zeros(4, 4, dtype=t.bool, device="cuda")
    bad[0, 0] = bad[1, 1] = bad[2, 3] = bad[3, 3] = True
    assert t.equal(out.s == 255, bad)
    y = t.empty(4, 128, device="cuda")
    moe.mx_dequantize(out, y)
    assert t.equal(y.isnan(), bad.repeat_interleave(32, 1))


def test_every_code_and_scale_dequantizes(moe):
    t = torch()
    for kind, n in (("e2m1", 16), ("e4m3", 256)):
        code = np.tile(np.arange(n, dtype=np.uint8), (256, 32 // n if n < 32 else 1))
        s = np.repeat(np.arange(256, dtype=np.uint8)[:, None], code.shape[1] // 32, 1)
        y = t.empty(code.shape, device="cuda")
        moe.mx_dequantize(ref.matrix(moe, code, s, kind), y)
        with np.errstate(over="ignore"):
            want = t.from_numpy(ref.values(code, s, kind)).cuda().float()  # 2^127 and more: infinity
        assert t.equal(y.nan_to_num(nan=7.5), want.nan_to_num(nan=7.5))


def test_strided_rows_and_another_stream(moe):
    """Rows of a wider tensor, an MX matrix inside a larger one; what lies between rows stays as it was."""
    t = torch()
    rng = np.random.default_rng(5)
    wide = t.from_numpy(rng.standard_normal((9, 256 + 64), dtype=np.float32)).cuda().bfloat16()
    x = wide[:, 32:32 + 256]
    q = t.full((9, 256 + 32), 0x77, dtype=t.uint8, device="cuda")
    s = t.full((9, 8 + 3), 0x77, dtype=t.uint8, device="cuda")
    out = moe.MXMatrix(q[:, :256], s[:, :8], "e4m3")
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    moe.mx_quantize(x, out, stream=side)
    t.cuda.current_stream().wait_stream(side)
    code, sc = ref.quantize(ref.host(x), "e4m3")
    assert np.array_equal(out.q.cpu().numpy(), code) and np.array_equal(out.s.cpu().numpy(), sc)
    assert t.all(q[:, 256:] == 0x77) and t.all(s[:, 8:] == 0x77)
    y = t.full((9, 256 + 8), 5.0, device="cuda")
    moe.mx_dequantize(out, y[:, :256])
    assert np.array_equal(ref.host(y[:, :256]), ref.values(code, sc, "e4m3")) and t.all(y[:, 256:] == 5)


# ------------------------------------------------------------------------------------------- norm --

# fp32 arithmetic of the norm, relative to |y|: at most 26 roundings in the sum of squares (8 to 16 of a thread, 10
# of the lanes and warps), halved by the root: 13; mean and eps: 2; the reciprocal root: 2 units = 4; h: 1 in it and 1
# in the mean; two products: 2.  23 x 2^-24, rounded up to a power of two:
FP32 = 2.0 ** -19
STEP = {"f32": 0.0, "bf16": 2.0 ** -8}  # then one rounding to the output's type (fp32's is in the above)

NORMS = [  # rows, cols, x, residual, weight, output
    (1, 7168, "bf16", "f32", True, "e4m3"), (1, 8, "f32", None, False, "f32"), (3, 1408, "f32", "bf16", True, "bf16"),
    (61, 7168, "bf16", "bf16", True, "bf16"), (5, 16384, "f32", "f32", True, "e2m1"), (2, 8200, "bf16", "f32", True, "f32"),
    (130, 64, "bf16", None, True, "e4m3"), (700, 32, "f32", "f32", False, "e2m1"), (9, 264, "bf16", None, False, "bf16"),
    (17, 4096, "f32", None, True, "e4m3"), (33, 12288, "bf16", "bf16", True, "e4m3"),
]


@pytest.mark.parametrize("rows,cols,xt,rt,weighted,out", NORMS)
@pytest.mark.parametrize("in_place", [False, True])
def test_norm(moe, rows, cols, xt, rt, weighted, out, in_place):
    t = torch()
    rng = np.random.default_rng(rows + cols)
    x = t.from_numpy((rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal(cols))).astype(np.float32)).cuda().to(dtype_of(xt))
    w = t.from_numpy(rng.standard_normal(cols).astype(np.float32)).cuda() if weighted else None
    if rows > 2:
        x[1] = 0  # a row of zeros (with its residual): zeros, not NaN
        x[2] *= 1e-12
    res = None
    if rt:
        res = t.from_numpy((rng.standard_normal((rows, cols)) * 3).astype(np.float32)).cuda().to(dtype_of(rt))
        if rows > 2:
            res[1] = 0
    h = ref.host(x) + (ref.host(res) if rt else 0)
    eps = 1e-6
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * (ref.host(w) if weighted else 1)
    mx = out in ("e2m1", "e4m3")
    got = moe.MXMatrix.empty(rows, cols, out) if mx else t.empty(rows, cols, dtype=dtype_of(out), device="cuda")
    ro = (res if in_place else t.empty_like(res)) if rt else None
    moe.rms_norm(x, got, weight=w, residual=res, residual_out=ro, eps=eps)
    if rt:
        assert np.all(np.abs(ref.host(ro) - h) <= (2.0 ** -24 if rt == "f32" else 2.0 ** -8 + 2.0 ** -24) * np.abs(h) + 1e-40)
    # The sum x + residual errs by 2^-24 of itself, a value near 0 by cancellation included: relative to h.
    if not mx:
        assert np.all(np.abs(ref.host(got) - y) <= (FP32 + STEP[out]) * np.abs(y) + 1e-38)
        return
    code, s = ref.unpack(got.q.cpu().numpy(), out), got.s.cpu().numpy()
    check_mx(code, s, y, out)


def check_mx(code, s, y, kind, slack=FP32):
    """Codes and scales of values that may differ from y by `slack` of themselves: the scale is that of the block's
    largest magnitude, or of one `slack` away; each element within half a step of it, or at the largest value."""
    blocks = np.abs(y).reshape(*s.shape, 32)
    for sign in (1 - slack, 1 + slack):
        m = blocks.max(-1) * sign
        e = np.where(m == 0, -127, np.maximum(np.frexp(np.where(m == 0, 1.0, m))[1] - 1 - ref.EMAX[kind], -127)) + 127
        good = e == s if sign < 1 else good | (e == s)
    assert good.all()
    scale = np.repeat(np.ldexp(1.0, s.astype(np.int64) - 127), 32, 1)
    a = np.abs(y) / scale
    least, mant = (0, 1) if kind == "e2m1" else (-6, 3)
    half = np.exp2(np.maximum(np.floor(np.log2(np.maximum(a * (1 + slack), 1e-300))), least) - mant) / 2
    allowed = np.maximum(half, a - ref.GRID[kind][-1]) + slack * a
    assert np.all(np.abs(ref.values(code, s, kind) - y) <= allowed * scale)


def test_norm_of_extreme_rows(moe):
    """Squares past fp32's range, infinities and NaN; other rows are as ever."""
    t = torch()
    x = t.randn(6, 1024, generator=t.Generator("cuda").manual_seed(1), device="cuda")
    x[0] *= 1e25
    x[1] *= 3e37
    x[2, 7] = float("inf")
    x[3, 9] = float("nan")
    out = t.empty_like(x)
    moe.rms_norm(x, out)
    h = ref.host(x)
    rows = [0, 1, 4, 5]
    y = h[rows] / np.sqrt((h[rows] ** 2).mean(1, keepdims=True) + 1e-6)
    assert np.all(np.abs(ref.host(out)[rows] - y) <= FP32 * np.abs(y))
    assert out[2, 7].isnan() and t.all(out[2, :7] == 0) and t.all(out[2, 8:] == 0) and out[3].isnan().all()
    mx = moe.MXMatrix.empty(6, 1024, "e4m3")
    moe.rms_norm(x, mx)
    assert t.all(mx.s[3] == 255) and mx.s[2, 0] == 255 and t.all(mx.s[2, 1:] == 0) and t.all(mx.s[rows] != 255)


def test_norm_strides_graph_and_repeat(moe):
    """Rows of a wider tensor; a captured call follows its inputs' values and gives the same bits."""
    t = torch()
    g = t.Generator("cuda").manual_seed(2)
    wide = t.randn(13, 512 + 64, generator=g, device="cuda")
    x, res = wide[:, :512], t.randn(13, 512, generator=g, device="cuda")
    w, out, ro = t.rand(512, generator=g, device="cuda"), t.full((13, 520), 4.0, device="cuda"), t.empty(13, 512, device="cuda")
    moe.rms_norm(x, out[:, :512], weight=w, residual=res, residual_out=ro)
    first = out.clone()
    assert t.all(out[:, 512:] == 4)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    graph = t.cuda.CUDAGraph()
    with t.cuda.stream(side):
        with t.cuda.graph(graph, stream=side):
            moe.rms_norm(x, out[:, :512], weight=w, residual=res, residual_out=ro)
    t.cuda.current_stream().wait_stream(side)
    keep = wide.clone()
    wide.mul_(2)
    graph.replay()
    t.cuda.synchronize()
    assert not t.equal(out, first)
    wide.copy_(keep)
    graph.replay()
    t.cuda.synchronize()
    assert t.equal(out, first)


@pytest.mark.parametrize("kind", ["e2m1", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_strided_matrices(moe, kind, dtype):
    """Enough values for several a thread, in rows with gaps on either side."""
    t = torch()
    rows, cols = 2600, 7168
    wide = t.randn(rows, cols + 64, generator=t.Generator("cuda").manual_seed(5), device="cuda").to(dtype_of(dtype))
    per = cols if kind == "e4m3" else cols // 2
    q = t.full((rows, per + 32), 0x77, dtype=t.uint8, device="cuda")
    s = t.full((rows, cols // 32 + 1), 0x77, dtype=t.uint8, device="cuda")
    out = moe.MXMatrix(q[:, :per], s[:, :cols // 32], kind)
    moe.mx_quantize(wide[:, 32:32 + cols], out)
    whole = moe.MXMatrix.empty(rows, cols, kind)
    moe.mx_quantize(wide[:, 32:32 + cols].contiguous(), whole)
    assert t.equal(out.q, whole.q) and t.equal(out.s, whole.s)
    assert t.all(q[:, per:] == 0x77) and t.all(s[:, cols // 32:] == 0x77)
    some = [0, 1, 777, rows - 1]
    code, sc = ref.quantize(ref.host(wide[some, 32:32 + cols]), kind)
    assert np.array_equal(out.q[some].cpu().numpy(), ref.pack(code, kind)) and np.array_equal(out.s[some].cpu().numpy(), sc)
    y, back = t.empty(rows, cols, device="cuda"), t.full((rows, cols + 8), 5.0, device="cuda")
    moe.mx_dequantize(whole, y)
    moe.mx_dequantize(out, back[:, :cols])
    assert t.equal(back[:, :cols], y) and t.all(back[:, cols:] == 5)
    assert np.array_equal(ref.host(y[some]), ref.values(code, sc, kind))


def test_more_than_2_to_34_values(moe):
    """Offsets past 32 bits: the ends of a matrix of 64 GiB of fp32, to MXFP4 and back over itself."""
    t = torch()
    t.cuda.empty_cache()
    if t.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GiB")
    rows, cols, n = (1 << 20) + 32, 16384, 32
    x = t.empty(rows, cols, device="cuda")
    g = t.Generator("cuda").manual_seed(3)
    ends = [slice(0, n), slice(rows - n, rows)]
    for e in ends:
        x[e] = t.randn(n, cols, generator=g, device="cuda")
    want = [ref.quantize(ref.host(x[e]), "e2m1") for e in ends]
    out = moe.MXMatrix.empty(rows, cols)
    moe.mx_quantize(x, out)
    for e, (code, s) in zip(ends, want):
        assert np.array_equal(out.q[e].cpu().numpy(), ref.pack(code, "e2m1")) and np.array_equal(out.s[e].cpu().numpy(), s)
    for e in ends:
        x[e] = 0
    moe.mx_dequantize(out, x)
    for e, (code, s) in zip(ends, want):
        assert np.array_equal(ref.host(x[e]), ref.values(code, s, "e2m1"))
    del x, out
    t.cuda.empty_cache()


@pytest.mark.parametrize("cols", [64, 256, 512, 768])
def test_norm_of_extreme_narrow_rows(moe, cols):
    """Rows that a warp takes: what one holds does not reach its neighbours."""
    t = torch()
    x = t.randn(21, cols, generator=t.Generator("cuda").manual_seed(cols), device="cuda")
    x[1] *= 1e25
    x[2] *= 3e37
    x[4, 7] = float("inf")
    x[5, 9] = float("nan")
    x[8] = 0
    x[20] *= 1e-30
    out = t.empty_like(x)
    moe.rms_norm(x, out)
    h = ref.host(x)
    rows = [r for r in range(21) if r not in (4, 5)]
    y = h[rows] / np.sqrt((h[rows] ** 2).mean(1, keepdims=True) + 1e-6)
    assert np.all(np.abs(ref.host(out)[rows] - y) <= FP32 * np.abs(y) + 1e-38)
    assert out[4, 7].isnan() and t.all(out[4, :7] == 0) and t.all(out[4, 8:] == 0) and out[5].isnan().all()
    mx = moe.MXMatrix.empty(21, cols, "e4m3")
    moe.rms_norm(x, mx)
    assert t.all(mx.s[5] == 255) and mx.s[4, 0] == 255 and t.all(mx.s[4, 1:] == 0) and t.all(mx.s[rows] != 255)


@pytest.mark.parametrize("cols", [7, 40, 100, 1000])
def test_norm_of_many_rows(moe, cols):
    """More rows than CTAs at once, a broadcast x, the residual's place taken by the result."""
    t = torch()
    cols *= 8
    g = t.Generator("cuda").manual_seed(cols)
    x, res = t.randn(1, cols, generator=g, device="cuda").bfloat16(), t.randn(5003, cols, generator=g, device="cuda")
    h = ref.host(x) + ref.host(res)
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + 1e-5)
    ro = t.empty_like(res)
    moe.rms_norm(x.expand(5003, cols), res, residual=res, residual_out=ro, eps=1e-5)
    assert np.all(np.abs(ref.host(ro) - h) <= 2.0 ** -24 * np.abs(h))
    # h, the sum, errs by 2^-24 of itself.
    assert np.all(np.abs(ref.host(res) - y) <= FP32 * np.abs(y))


def test_norm_of_the_most_rows(moe):
    """2^31 - 1 rows, 32 GiB of bf16, in place: its ends."""
    t = torch()
    t.cuda.empty_cache()
    if t.cuda.mem_get_info()[0] < 50 << 30:
        pytest.skip("needs 50 GiB")
    rows, n = (1 << 31) - 1, 1000
    x = t.empty(rows, 8, dtype=t.bfloat16, device="cuda")
    g = t.Generator("cuda").manual_seed(6)
    ends = [slice(0, n), slice(rows - n, rows)]
    for e in ends:
        x[e] = t.randn(n, 8, generator=g, device="cuda").bfloat16()
    h = [ref.host(x[e]) for e in ends]
    moe.rms_norm(x, x)
    for e, v in zip(ends, h):
        y = v / np.sqrt((v * v).mean(1, keepdims=True) + 1e-6)
        assert np.all(np.abs(ref.host(x[e]) - y) <= (FP32 + STEP["bf16"]) * np.abs(y))
    del x
    t.cuda.empty_cache()
