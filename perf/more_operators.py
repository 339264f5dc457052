"""Timed cases of the dense half of a serving step around the routed MoE layer: a residual sum with its
root-mean-square norm, microscaled (MX) rounding of activations and weights, the product of MX matrices, and log
probabilities of given tokens with entropy and the best alternatives.

``run`` computes an operator in plain torch operations in 32 bits, or, where ``own`` is set, through this
package's entry points.  Sizes follow the package's own workloads (hidden size 7168, intermediate size 1408, 56
query and 8 key heads of 128; 1, 64 and 4096 tokens) or are generic.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32                              # elements that share a scale
TOP = {"e2m1": 2, "e4m3": 8}            # exponent of the largest power of two of an element type
MOST = {"e2m1": 6.0, "e4m3": 448.0}     # its largest value
MANT = {"e2m1": 1, "e4m3": 3}           # its mantissa bits
LEAST = {"e2m1": 0, "e4m3": -6}         # exponent of its smallest normal value


# ------------------------------------------------------------------------------------------- cases --

def listed():
    return [
        # Activations of a small batch before an MX product: latency.
        dict(name="quantize_61", op="quantize", dtype="bf16", rows=61, cols=7168, kind="e4m3"),
        # A projection's weights brought to MXFP4 when a checkpoint is loaded, and looked at.
        dict(name="quantize_weights", op="quantize", dtype="bf16", rows=9216, cols=7168, kind="e2m1"),
        # One token's residual and norm, codes for the next projection: latency.
        dict(name="norm_1", op="norm", dtype="bf16", rows=1, cols=7168, res="f32", out="e4m3"),
        # A mid-sized batch with narrow rows, bf16 residual.
        dict(name="norm_509", op="norm", dtype="f32", rows=509, cols=1408, res="bf16", out="bf16"),
        # A prefill's rows.
        dict(name="norm_4096", op="norm", dtype="bf16", rows=4096, cols=7168, res="f32", out="e4m3"),
        # One token through the query, key and value projection.
        dict(name="linear_1", op="linear", rows=1, outs=9216, cols=7168, kind="e4m3", out="bf16", add="none"),
        # A serving batch through the attention's output projection, added into the fp32 residual.
        dict(name="linear_64", op="linear", rows=64, outs=7168, cols=7168, kind="e4m3", out="f32", add="f32"),
        # Ragged sizes, 4 bits on both sides.
        dict(name="linear_1021", op="linear", rows=1021, outs=4099, cols=1408, kind="e2m1", out="bf16", add="none"),
        # A prefill through the query, key and value projection, activations in 8 and in 4 bits.
        dict(name="linear_4096", op="linear", rows=4096, outs=9216, cols=7168, kind="e4m3", out="bf16", add="none"),
        dict(name="linear_4096_fp4", op="linear", rows=4096, outs=9216, cols=7168, kind="e2m1", out="bf16", add="none"),
        # The token just drawn, with five alternatives: latency.
        dict(name="score_1", op="score", dtype="f32", rows=1, vocab=100003, top=5),
        # A prompt's tokens under the model, with twenty alternatives each.
        dict(name="score_512", op="score", dtype="bf16", rows=512, vocab=163840, top=20),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ones' ranges, no dearer than the largest of its operator."""
    op = rng.choice(("quantize", "norm", "linear", "linear", "score"))
    if op == "quantize":
        cols = 32 * _log(rng, 1, 512)
        rows = min(_log(rng, 1, 60000), max(1, 9216 * 7168 // cols))
        return dict(op=op, dtype=rng.choice(("f32", "bf16")), rows=rows, cols=cols, kind=rng.choice(("e2m1", "e4m3")))
    if op == "norm":
        cols = 32 * _log(rng, 2, 512)
        rows = min(_log(rng, 1, 20000), max(1, 4096 * 7168 // cols))
        return dict(op=op, dtype=rng.choice(("f32", "bf16")), rows=rows, cols=cols, res=rng.choice(("f32", "bf16", "none")),
                    out=rng.choice(("f32", "bf16", "e4m3", "e4m3")))
    if op == "linear":
        rows, outs, cols = _log(rng, 1, 4096), _log(rng, 32, 16384), 128 * _log(rng, 1, 128)
        while rows * outs * cols > 4096 * 9216 * 7168 or outs * cols > 16384 * 7168:
            outs = outs // 2 + 1
        out = rng.choice(("bf16", "bf16", "f32"))
        return dict(op=op, rows=rows, outs=outs, cols=cols, kind=rng.choice(("e4m3", "e2m1")), out=out,
                    add=rng.choice(("none", out)))
    vocab = _log(rng, 1000, 200000)
    return dict(op=op, dtype=rng.choice(("f32", "bf16")), rows=max(1, min(_log(rng, 1, 4096), 256 * 163840 // vocab)),
                vocab=vocab, top=rng.choice((0, 1, 5, 20, rng.randint(2, 32))))


def _size(dtype):
    return {"f32": 4.0, "bf16": 2.0, "none": 0.0, "e4m3": 1 + 1 / BLOCK, "e2m1": 0.5 + 1 / BLOCK}[dtype]


def work(case):
    c = case
    if c["op"] == "quantize":  # the values that the codes stand for are looked at in bf16
        n = c["rows"] * c["cols"]
        return {"bytes": n * (_size(c["dtype"]) + 2), "flops": 4.0 * n}
    if c["op"] == "norm":
        n = c["rows"] * c["cols"]
        out = 2.0 if c["out"] == "e4m3" else _size(c["out"])  # codes: as above
        return {"bytes": n * (_size(c["dtype"]) + 2 * _size(c["res"]) + out) + 4 * c["cols"], "flops": 6.0 * n}
    if c["op"] == "linear":
        t, n, k = c["rows"], c["outs"], c["cols"]
        return {"bytes": t * k * _size(c["kind"]) + n * k * _size("e2m1") + t * n * (_size(c["out"]) + _size(c["add"])),
                "flops": 2.0 * t * n * k}
    n = c["rows"] * c["vocab"]
    return {"bytes": n * _size(c["dtype"]) + c["rows"] * (16 + 8 * c["top"]), "flops": 6.0 * n}


# ------------------------------------------------------------------------------------------ inputs --

def _type(name):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": dict(case)}

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=DEV).to(dtype)

    if c["op"] == "score":
        # Scores with a wide body and a few strong tokens, as a trained head gives; the text's own token is
        # usually a likely one.
        rows, vocab = c["rows"], c["vocab"]
        x = normal(rows, vocab) * 2.5
        hot = torch.randint(0, vocab, (rows, 8), generator=g, device=DEV)
        x.scatter_add_(1, hot, torch.rand(rows, 8, generator=g, device=DEV) * 10)
        s["logits"] = x.to(_type(c["dtype"]))
        any_token = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
        s["tokens"] = torch.where(torch.rand(rows, generator=g, device=DEV) < 0.7, hot[:, 0], any_token).to(torch.int32)
        f32, i32 = dict(device=DEV), dict(device=DEV, dtype=torch.int32)
        s["logprob"], s["entropy"], s["rank"] = torch.empty(rows, **f32), torch.empty(rows, **f32), torch.empty(rows, **i32)
        s["top_ids"] = torch.empty(rows, c["top"], **i32) if c["top"] else None
        s["top_logprobs"] = torch.empty(rows, c["top"], **f32) if c["top"] else None
        return s
    rows, cols = c["rows"], c["cols"]
    if c["op"] == "linear":
        s["xq"], s["xs"] = _codes(normal(rows, cols), c["kind"])            # normalised activations
        s["wq"], s["ws"] = _codes(normal(c["outs"], cols) * cols ** -0.5, "e2m1")
        s["add"] = normal(rows, c["outs"], dtype=_type(c["add"])) if c["add"] != "none" else None
        s["out"] = torch.empty(rows, c["outs"], device=DEV, dtype=_type(c["out"]))
        if own:
            import mxfp4_routed_expert_moe_gb300 as moe
            s["x"] = moe.MXMatrix(s["xq"], s["xs"], c["kind"])
            s["w"] = moe.MXMatrix(s["wq"], s["ws"], "e2m1")
        return s
    # Activations differ in size by channel, with some channels far above the others.
    channel = torch.exp(normal(cols) * 0.5)
    channel[torch.rand(cols, generator=g, device=DEV) < 0.003] *= 30
    s["x"] = (normal(rows, cols) * channel * (0.02 if c["op"] == "quantize" else 1.0)).to(_type(c["dtype"]))
    if c["op"] == "norm":
        s["weight"] = 1 + 0.2 * normal(cols)
        s["res"] = (normal(rows, cols) * channel * 3).to(_type(c["res"])) if c["res"] != "none" else None
        s["res_out"] = torch.empty_like(s["res"]) if c["res"] != "none" else None
        if c["out"] != "e4m3":
            s["y"] = torch.empty(rows, cols, device=DEV, dtype=_type(c["out"]))
    kind = c["kind"] if c["op"] == "quantize" else c["out"] if c["out"] == "e4m3" else None
    if kind:
        s["values"] = torch.empty(rows, cols, device=DEV, dtype=torch.bfloat16)
        if own:
            import mxfp4_routed_expert_moe_gb300 as moe
            s["codes"] = moe.MXMatrix.empty(rows, cols, kind, device=DEV)
    return s


# ------------------------------------------------------------------------------------------- passes --

def run(state):
    op = state["case"]["op"]
    if own:
        return {"quantize": _own_quantize, "norm": _own_norm, "linear": _own_linear, "score": _own_score}[op](state)
    return {"quantize": _plain_quantize, "norm": _plain_norm, "linear": _plain_linear, "score": _plain_score}[op](state)


def _own_quantize(s):
    import mxfp4_routed_expert_moe_gb300 as moe
    moe.mx_quantize(s["x"], s["codes"])
    moe.mx_dequantize(s["codes"], s["values"])
    return {"values": s["values"]}


def _own_norm(s):
    import mxfp4_routed_expert_moe_gb300 as moe
    c = s["case"]
    codes = c["out"] == "e4m3"
    moe.rms_norm(s["x"], s["codes"] if codes else s["y"], weight=s["weight"], residual=s["res"], residual_out=s["res_out"],
                 eps=1e-6)
    if codes:
        moe.mx_dequantize(s["codes"], s["values"])
    return {"y": s["values"] if codes else s["y"], "residual": s["res_out"]}


def _own_linear(s):
    import mxfp4_routed_expert_moe_gb300 as moe
    moe.mx_linear(s["x"], s["w"], s["out"], add=s["add"])
    return {"out": s["out"]}


def _own_score(s):
    import mxfp4_routed_expert_moe_gb300 as moe
    moe.token_logprobs(s["logits"], s["tokens"], s["logprob"], rank=s["rank"], entropy=s["entropy"], top_ids=s["top_ids"],
                       top_logprobs=s["top_logprobs"])
    return _scores(s)


def _scores(s):
    return {n: s[n] for n in ("logprob", "rank", "entropy", "top_ids", "top_logprobs")}


def _by_power(x, n):
    """x * 2^n for whole n in -252 .. 254, by two factors made of their bits: exact, which a power function need not be."""
    half = torch.div(n, 2, rounding_mode="floor")
    a, b = (((h + 127).to(torch.int32) << 23).view(torch.float32) for h in (half, n - half))
    return x * a * b


def _rounded(x, kind):
    """fp32 values [rows][cols] on the grid of their block's scale: (elements on the type's own grid, exponents
    [rows][blocks]).  The scale is the power of two that puts the largest magnitude on the type's top binade;
    elements are rounded to nearest, ties to even, and saturate."""
    b = x.view(x.shape[0], -1, BLOCK)
    most = b.abs().amax(-1)
    e = torch.frexp(most)[1] - 1 - TOP[kind]
    e = torch.where(most > 0, e.clamp(-127, 127), -127)
    v = _by_power(b, -e[..., None])
    step = (torch.frexp(v)[1] - 1).clamp(min=LEAST[kind]) - MANT[kind]
    v = _by_power(torch.round(_by_power(v, -step)), step).clamp(-MOST[kind], MOST[kind])
    return v, e


def _codes(x, kind):
    """Codes and scales of fp32 values: uint8 [rows][cols] or, two to a byte, [rows][cols / 2]; uint8 [rows][blocks]."""
    v, e = _rounded(x, kind)
    v = v.view(x.shape)
    if kind == "e4m3":
        return v.to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=x.device)
    c = torch.bucketize(v.abs(), grid).to(torch.uint8) + torch.where(v < 0, 8, 0).to(torch.uint8)
    return c[:, 0::2] + 16 * c[:, 1::2], (e + 127).to(torch.uint8)


def _values(q, scale, kind):
    """What codes and scales stand for, fp32 [rows][cols]."""
    if kind == "e4m3":
        v = q.view(torch.float8_e4m3fn).float()
    else:
        grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=q.device)
        v = torch.stack((grid[(q & 15).long()], grid[(q >> 4).long()]), -1)
    v = v.view(q.shape[0], -1, BLOCK)
    return _by_power(v, (scale.int() - 127)[..., None]).view(q.shape[0], -1)


def _plain_quantize(s):
    v, e = _rounded(s["x"].float(), s["case"]["kind"])
    s["values"].copy_(_by_power(v, e[..., None]).view(s["values"].shape))
    return {"values": s["values"]}


def _plain_norm(s):
    c = s["case"]
    h = s["x"].float()
    if s["res"] is not None:
        h = h + s["res"].float()
        s["res_out"].copy_(h)
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * s["weight"]
    if c["out"] == "e4m3":
        v, e = _rounded(y, "e4m3")
        s["values"].copy_(_by_power(v, e[..., None]).view(y.shape))
        return {"y": s["values"], "residual": s["res_out"]}
    s["y"].copy_(y)
    return {"y": s["y"], "residual": s["res_out"]}


def _plain_linear(s):
    x = _values(s["xq"], s["xs"], s["case"]["kind"])
    y = torch.matmul(x, _values(s["wq"], s["ws"], "e2m1").T)
    s["out"].copy_(y if s["add"] is None else y + s["add"].float())
    return {"out": s["out"]}


def _plain_score(s):
    x = s["logits"].float()
    n = s["case"]["top"]
    m = x.amax(1, keepdim=True)
    d = x - m
    w = torch.exp(d)
    total = w.sum(1)
    lse = torch.log(total)
    token = s["tokens"].long()[:, None]
    own_score = x.gather(1, token)
    s["logprob"].copy_(d.gather(1, token)[:, 0] - lse)
    s["entropy"].copy_(lse - (w * d).sum(1) / total)
    index = torch.arange(x.shape[1], device=DEV)[None]
    s["rank"].copy_(((x > own_score) | ((x == own_score) & (index < token))).sum(1))
    if n:
        best, order = torch.sort(x, dim=1, descending=True, stable=True)
        s["top_ids"].copy_(order[:, :n])
        s["top_logprobs"].copy_(best[:, :n] - m - lse[:, None])
    return _scores(s)


# --------------------------------------------------------------------------- the definition, 64 bits --

def exact(case, seed):
    s = prepare(case, seed)
    return {"quantize": _exact_quantize, "norm": _exact_norm, "linear": _exact_linear, "score": _exact_score}[case["op"]](case, s)


def _grid(kind):
    """All magnitudes of an element type, ascending, from its codes' bits."""
    m = MANT[kind]
    bias = 1 - LEAST[kind]
    codes = range(8) if kind == "e2m1" else range(127)  # E4M3's last code is NaN
    at = [(c >> m, (c & ((1 << m) - 1)) / (1 << m)) for c in codes]
    return torch.tensor([f * 2.0 ** (1 - bias) if e == 0 else (1 + f) * 2.0 ** (e - bias) for e, f in at], device=DEV,
                        dtype=torch.float64)


def _two_to(n):
    """2^n in 64 bits from its bits, whole n."""
    return ((n + 1023).long() << 52).view(torch.float64)


def _exact_mx(x, kind):
    """x in 64 bits on its blocks' grids: the nearer of the two neighbours among the type's magnitudes."""
    b = x.view(x.shape[0], -1, BLOCK)
    most = b.abs().amax(-1, keepdim=True)
    e = torch.where(most > 0, torch.floor(torch.log2(torch.where(most > 0, most, 1.0))), 0.0)
    e += (_two_to(e + 1) <= most).double() - (_two_to(e) > most).double()  # a logarithm next to a whole number
    scale = torch.where(most > 0, _two_to((e - TOP[kind]).clamp(-127, 127)), 1.0)
    a = b.abs() / scale
    grid = _grid(kind)
    hi = torch.searchsorted(grid, a).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    pick = torch.where(a >= grid[-1], len(grid) - 1, pick)
    return (torch.copysign(grid[pick], b) * scale).view(x.shape)


def _exact_quantize(c, s):
    return {"values": torch.cat([_exact_mx(x.double(), c["kind"]) for x in s["x"].split(2048)])}


def _exact_norm(c, s):
    y, res = [], []
    for i in range(0, c["rows"], 1024):
        h = s["x"][i:i + 1024].double()
        if s["res"] is not None:
            h = h + s["res"][i:i + 1024].double()
            res.append(h)
        v = h * s["weight"].double() / torch.sqrt((h * h).sum(1, keepdim=True) / c["cols"] + 1e-6)
        y.append(_exact_mx(v, "e4m3") if c["out"] == "e4m3" else v)
    return {"y": torch.cat(y), "residual": torch.cat(res) if res else None}


def _exact_linear(c, s):
    if work(c)["flops"] > 2e12:
        return None

    def values(q, scale, kind):
        grid = _grid(kind)
        grid = torch.cat((grid, torch.zeros(1, device=DEV, dtype=grid.dtype))) if kind == "e4m3" else grid
        grid = torch.cat((grid, -grid))
        if kind == "e2m1":
            v = torch.empty(q.shape[0], 2 * q.shape[1], device=DEV, dtype=torch.float64)
            v[:, 0::2], v[:, 1::2] = grid[(q % 16).int()], grid[torch.div(q, 16, rounding_mode="floor").int()]
        else:
            v = grid[q.int()]
        return v * torch.repeat_interleave(_two_to(scale.int() - 127), BLOCK, 1)

    x, w = values(s["xq"], s["xs"], c["kind"]), values(s["wq"], s["ws"], "e2m1")
    y = torch.einsum("tk,nk->tn", x, w)
    return {"out": y if s["add"] is None else y + s["add"].double()}


def _exact_score(c, s):
    out = {n: [] for n in ("logprob", "entropy", "top_logprobs")}
    for i in range(0, c["rows"], 64):
        x = s["logits"][i:i + 64].double()
        logp = torch.log_softmax(x, 1)
        out["logprob"].append(logp.gather(1, s["tokens"][i:i + 64].long()[:, None])[:, 0])
        out["entropy"].append(-(torch.exp(logp) * logp).sum(1))
        if c["top"]:
            out["top_logprobs"].append(torch.topk(logp, c["top"], dim=1).values)
    return {n: torch.cat(v) if v else None for n, v in out.items()} | {"rank": None, "top_ids": None}
