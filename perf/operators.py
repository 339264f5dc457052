"""Timed cases of the serving operators that surround the routed MoE layer in a decode step: appending
rotated keys and values to a paged cache, attention of a batch that shares a long prefix over that cache,
and sampling from logits with given uniform numbers.

``run`` computes an operator in plain torch operations in 32 bits, or, where ``own`` is set, through this
package's entry points.  Sizes follow the package's own workloads (hidden size 7168 as 56 heads of 128;
1, 8, 64, 256 and 4096 tokens) or are generic.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
FIX = 2.0 ** 31  # fixed-point unit of the sampling weights


# ------------------------------------------------------------------------------------------- cases --

def listed():
    return [
        # A speculative step's 8 tokens, one per sequence: the launch's latency is all there is.
        dict(name="append_8", op="append", dtype="bf16", batch=8, q=1, ragged=False, own=777, prefix=2048, page=64,
             q_heads=56, kv_heads=8, dim=128, rot=128, inter=False),
        # fp32 projections of a mid-sized chunk, half of each head rotated in neighbouring pairs.
        dict(name="append_f32_512", op="append", dtype="f32", batch=7, q=143, ragged=True, own=301, prefix=0, page=16,
             q_heads=32, kv_heads=8, dim=64, rot=32, inter=True),
        # The prompts of a large prefill.
        dict(name="append_16384", op="append", dtype="bf16", batch=16, q=1024, ragged=False, own=1500, prefix=4096,
             page=64, q_heads=56, kv_heads=8, dim=128, rot=128, inter=False),
        # One sequence, one token, a short context: latency.
        dict(name="attend_1", op="attend", batch=1, q=1, ragged=False, own=201, prefix=512, page=64, q_heads=56,
             kv_heads=8, dim=128),
        # Speculative verification: 8 tokens of one sequence over its own long context, causal among themselves.
        dict(name="attend_verify_8", op="attend", batch=1, q=8, ragged=False, own=16001, prefix=0, page=64, q_heads=56,
             kv_heads=8, dim=128),
        # A serving batch behind one system prompt, ragged contexts of its own.
        dict(name="attend_64", op="attend", batch=64, q=1, ragged=False, own=2047, prefix=8192, page=64, q_heads=56,
             kv_heads=8, dim=128),
        # No shared part: long ragged contexts, small pages, 16 query heads to a key head, short heads.
        dict(name="attend_own_24", op="attend", batch=24, q=1, ragged=False, own=32771, prefix=0, page=16, q_heads=64,
             kv_heads=4, dim=64),
        # A wide batch over a long shared document.
        dict(name="attend_256", op="attend", batch=256, q=1, ragged=False, own=509, prefix=32768, page=128, q_heads=56,
             kv_heads=8, dim=128),
        # Prompts behind a shared prefix: many new tokens a sequence, ragged, causal.
        dict(name="attend_prompt", op="attend", batch=9, q=301, ragged=True, own=700, prefix=4001, page=32, q_heads=32,
             kv_heads=8, dim=128),
        # One token's logits: latency.
        dict(name="sample_1", op="sample", dtype="f32", rows=1, vocab=100003, mode="mixed", probs=False),
        # A serving batch's logits in bf16, every filter in use.
        dict(name="sample_64", op="sample", dtype="bf16", rows=64, vocab=163840, mode="mixed", probs=False),
        # A large batch whose filtered distribution is wanted too (the target of a speculative test).
        dict(name="sample_512", op="sample", dtype="f32", rows=512, vocab=128000, mode="mixed", probs=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ones' ranges, no dearer than the largest of its operator."""
    op = rng.choice(("append", "attend", "attend", "sample"))
    if op == "sample":
        vocab = _log(rng, 1000, 200000)
        return dict(op=op, dtype=rng.choice(("f32", "bf16")), rows=max(1, min(_log(rng, 1, 512), 512 * 128000 // vocab)),
                    vocab=vocab, mode=rng.choice(("mixed", "mixed", "plain", "topk", "topp")), probs=rng.random() < 0.3)
    kv_heads = rng.choice((1, 2, 4, 8, 16))
    group = rng.choice((1, 2, 4, 5, 7, 8, 16))
    while kv_heads * group > 64:
        group = rng.choice((1, 2, 4))
    dim = rng.choice((64, 128))
    page = rng.choice((16, 32, 64, 128))
    if op == "append":
        n = _log(rng, 1, 16384)
        batch = min(n, _log(rng, 1, 256))
        q = max(1, n // batch)
        rot = rng.choice((dim, dim // 2, 32, 0))
        return dict(op=op, dtype=rng.choice(("f32", "bf16", "bf16")), batch=batch, q=q, ragged=q > 1 and rng.random() < 0.5,
                    own=q + _log(rng, 1, 1500), prefix=rng.choice((0, _log(rng, 1, 8192))), page=page,
                    q_heads=min(56, kv_heads * group) // kv_heads * kv_heads, kv_heads=min(kv_heads, 8), dim=dim, rot=rot,
                    inter=rng.random() < 0.3) if kv_heads <= 8 else draw(rng)
    batch = _log(rng, 1, 256)
    q = rng.choice((1, 1, 1, _log(rng, 2, 16), _log(rng, 17, 300)))
    case = dict(op=op, batch=batch, q=q, ragged=q > 1 and rng.random() < 0.6, own=q + _log(rng, 1, 32768),
                prefix=rng.choice((0, _log(rng, 1, 32768), _log(rng, 1, 32768))), page=page, q_heads=kv_heads * group,
                kv_heads=kv_heads, dim=dim)
    # Within the largest listed case: its operations, the bytes of its cache, and the plain form's score matrices.
    top, mem = work(_largest()), 3 << 30
    while True:
        w = work(case)
        lq = max(_q_lens(case))
        scores = 4 * case["q_heads"] * (sum(_q_lens(case)) * case["prefix"] + case["batch"] * lq * case["own"])
        pad = 8 * case["batch"] * case["own"] * case["kv_heads"] * dim
        if w["flops"] <= top["flops"] and w["bytes"] <= 1.45 * top["bytes"] and scores <= mem and pad <= mem:
            return case
        if case["batch"] > 8:
            case["batch"] //= 2
        elif case["q"] > 1:
            case["q"] = max(1, case["q"] // 2)
            case["ragged"] = case["ragged"] and case["q"] > 1
        else:
            case["own"] = 1 + case["own"] // 2
            case["prefix"] //= 2


def _largest():
    return next(c for c in listed() if c["name"] == "attend_256")


def _q_lens(c):
    """New tokens of each sequence: all alike, or spread over 0 .. q."""
    if not c["ragged"]:
        return [c["q"]] * c["batch"]
    n = [(c["q"] * ((i * 377 + 233) % 610)) // 609 for i in range(c["batch"])]
    n[0] = c["q"]
    return n


def _own_lens(c):
    """Tokens of each sequence's own part of the cache, the new ones among them: spread up to own."""
    spare = c["own"] - c["q"]
    lens = [n + (spare * ((i * 610 + 377) % 987)) // 986 for i, n in enumerate(_q_lens(c))]
    lens[0] = _q_lens(c)[0] + spare
    return lens


def work(case):
    c = case
    if c["op"] == "sample":
        e = 4 if c["dtype"] == "f32" else 2
        n = c["rows"] * c["vocab"]
        return {"bytes": n * e + (4 * n if c["probs"] else 0) + c["rows"] * 32, "flops": 4.0 * n}
    q_lens, lens = _q_lens(c), _own_lens(c)
    n = sum(q_lens)
    if c["op"] == "append":
        e = 4 if c["dtype"] == "f32" else 2
        vals = n * c["dim"] * (c["q_heads"] + 2 * c["kv_heads"])
        return {"bytes": vals * (e + 2) + n * (c["rot"] * 4 + 4), "flops": 3.0 * n * c["rot"] * (c["q_heads"] + c["kv_heads"])}
    seen = n * c["prefix"] + sum(q * (l - q) + q * (q + 1) // 2 for q, l in zip(q_lens, lens))
    kv = 4 * c["kv_heads"] * c["dim"] * (c["prefix"] + sum(l for q, l in zip(q_lens, lens) if q))
    return {"bytes": kv + n * c["q_heads"] * (4 * c["dim"] + 4), "flops": 4.0 * c["dim"] * c["q_heads"] * seen}


# ------------------------------------------------------------------------------------------ inputs --

def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": dict(case)}
    if c["op"] == "sample":
        rows, vocab = c["rows"], c["vocab"]
        # Scores with a wide body and a few strong tokens, as a trained head gives.
        x = torch.randn(rows, vocab, generator=g, device=DEV) * 2.5
        hot = torch.randint(0, vocab, (rows, 8), generator=g, device=DEV)
        x.scatter_add_(1, hot, torch.rand(rows, 8, generator=g, device=DEV) * 10)
        s["logits"] = x if c["dtype"] == "f32" else x.bfloat16()
        r = torch.rand(6, rows, generator=g, device=DEV)
        mixed = c["mode"] == "mixed"
        s["u"] = torch.rand(rows, generator=g, device=DEV)
        s["temperature"] = 0.3 + r[0] * 1.2
        if mixed:
            s["temperature"][r[1] < 0.1] = 0.0  # greedy rows
        off = torch.zeros_like(r[2])
        k = (torch.exp(r[2] * math.log(min(vocab, 4000)))).to(torch.int32)
        s["top_k"] = torch.where(r[3] < 0.3, torch.zeros_like(k), k) if mixed else k if c["mode"] == "topk" else None
        s["top_p"] = torch.where(r[4] < 0.2, off + 1, 0.5 + 0.5 * r[4]) if mixed or c["mode"] == "topp" else None
        s["min_p"] = torch.where(r[5] < 0.5, off, r[5] * 0.1) if mixed else None
        s["out"] = torch.empty(rows, dtype=torch.int32, device=DEV)
        s["kept"] = torch.empty(rows, dtype=torch.int32, device=DEV)
        s["logprob"] = torch.empty(rows, device=DEV)
        s["probs"] = torch.empty(rows, vocab, device=DEV) if c["probs"] else None
        return s
    q_lens, lens, page = _q_lens(c), _own_lens(c), c["page"]
    n, hq, hk, d = sum(q_lens), c["q_heads"], c["kv_heads"], c["dim"]
    np_prefix, width = -(-c["prefix"] // page), max(1, -(-max(lens) // page))
    own_pages = [-(-l // page) for l in lens]
    pages = np_prefix + sum(own_pages) + 3
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    s["prefix_table"] = perm[:np_prefix].contiguous()
    at = np.concatenate([[0], np.cumsum(own_pages)])[:-1] + np_prefix
    cell = np.minimum(at[:, None] + np.arange(width)[None, :], pages - 1)
    s["table"] = perm[torch.from_numpy(cell).to(DEV)].contiguous()
    s["kv_len"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["q_start"] = torch.from_numpy(np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)).to(DEV)
    s["tokens"], s["max_q"] = n, max(q_lens)
    shape = (pages, page, hk, d)
    s["k_cache"] = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    s["v_cache"] = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    if c["op"] == "append":
        t = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
        qkv = torch.randn(n, (hq + 2 * hk) * d, generator=g, device=DEV, dtype=t)  # one projection's rows
        s["q"], s["k"], s["v"] = (x.view(n, -1, d) for x in qkv.split((hq * d, hk * d, hk * d), 1))
        inv = 10000.0 ** (-torch.arange(0, max(c["rot"], 2), 2, device=DEV, dtype=torch.float64) / max(c["rot"], 2))
        a = torch.arange(c["prefix"] + max(lens), device=DEV, dtype=torch.float64)[:, None] * inv
        s["rope"] = torch.cat((a.cos(), a.sin()), 1).float()
        s["q_out"] = torch.empty(n, hq, d, device=DEV, dtype=torch.bfloat16)
    else:
        # Normalised queries of a trained model reach further than the keys: some scores stand out.
        s["q"] = torch.randn(n, hq, d, generator=g, device=DEV, dtype=torch.bfloat16) * 1.5
        s["out"] = torch.empty(n, hq, d, device=DEV, dtype=torch.bfloat16)
        s["lse"] = torch.empty(n, hq, device=DEV)
    if own:
        import mxfp4_routed_expert_moe_gb300 as moe
        s["cache"] = moe.KVCache(s["k_cache"], s["v_cache"])
        s["batch"] = moe.KVBatch(s["kv_len"], s["table"], tokens=n, q_start=s["q_start"], max_q=s["max_q"],
                                 prefix_table=s["prefix_table"], prefix_len=c["prefix"])
        if c["op"] == "attend":
            s["ws"] = torch.empty(moe.attention_workspace_bytes(s["cache"], s["batch"], hq), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------------------------------- passes --

def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "attend": _own_attend, "sample": _own_sample}[op](state)
    return {"append": _plain_append, "attend": _plain_attend, "sample": _plain_sample}[op](state)


def _own_append(s):
    import mxfp4_routed_expert_moe_gb300 as moe
    c = s["case"]
    moe.kv_append(s["cache"], s["batch"], s["k"], s["v"], q=s["q"], q_out=s["q_out"],
                  rope=s["rope"] if c["rot"] else None, rot_dim=c["rot"], interleaved=c["inter"])
    return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}


def _own_attend(s):
    import mxfp4_routed_expert_moe_gb300 as moe
    moe.prefix_attention(s["cache"], s["batch"], s["q"], s["out"], s["ws"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_sample(s):
    import mxfp4_routed_expert_moe_gb300 as moe
    moe.sample(s["logits"], s["u"], s["out"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
               min_p=s["min_p"], logprob=s["logprob"], kept=s["kept"], probs=s["probs"])
    return {"token": s["out"], "kept": s["kept"], "logprob": s["logprob"]} | ({"probs": s["probs"]} if s["probs"] is not None else {})


def _places(s):
    """Of each new token: its sequence, and its index in that sequence's own part of the cache."""
    tok = torch.arange(s["tokens"], device=DEV, dtype=torch.int32)
    seq = torch.searchsorted(s["q_start"], tok, right=True) - 1
    end = s["q_start"][1:]
    return seq, (s["kv_len"][seq] - (end[seq] - tok)).long()


def _rotated(x, cos, sin, rot, inter):
    """x [n][heads][d] with its first rot values rotated by the angles of its row."""
    if rot == 0:
        return x
    r, rest = x[..., :rot], x[..., rot:]
    a, b = (r[..., 0::2], r[..., 1::2]) if inter else (r[..., : rot // 2], r[..., rot // 2:])
    p, q = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((p, q), -1).flatten(-2) if inter else torch.cat((p, q), -1)
    return torch.cat((r, rest), -1)


def _plain_append(s):
    c = s["case"]
    rot, page = c["rot"], c["page"]
    seq, j = _places(s)
    angles = s["rope"][c["prefix"] + j]
    cos, sin = (x[:, None] for x in angles.chunk(2, 1))
    where = s["table"][seq, j // page].long(), j % page
    s["k_cache"][where] = _rotated(s["k"].float(), cos, sin, rot, c["inter"]).bfloat16()
    s["v_cache"][where] = s["v"].bfloat16()
    s["q_out"].copy_(_rotated(s["q"].float(), cos, sin, rot, c["inter"]))
    return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}


def _plain_attend(s):
    c = s["case"]
    hq, hk, d = c["q_heads"], c["kv_heads"], c["dim"]
    n, b, page, maxq = s["tokens"], c["batch"], c["page"], s["max_q"]
    grp = hq // hk
    seq, j = _places(s)
    q = s["q"].float().view(n, hk, grp, d) / math.sqrt(d)
    # The shared part: every row against every key.
    kp = s["k_cache"][s["prefix_table"].long()].float().view(-1, hk, d)[: c["prefix"]]
    vp = s["v_cache"][s["prefix_table"].long()].float().view(-1, hk, d)[: c["prefix"]]
    sp = torch.matmul(q.permute(1, 0, 2, 3).reshape(hk, n * grp, d), kp.permute(1, 2, 0))
    # Each sequence's own part, padded to the longest.
    row = torch.arange(n, device=DEV, dtype=torch.int32) - s["q_start"][seq]
    qb = torch.zeros(b, maxq, hk, grp, d, device=DEV)
    qb[seq, row] = q
    ko = s["k_cache"][s["table"].long()].float().view(b, -1, hk, d)
    vo = s["v_cache"][s["table"].long()].float().view(b, -1, hk, d)
    so = torch.matmul(qb.permute(0, 2, 1, 3, 4).reshape(b, hk, maxq * grp, d), ko.permute(0, 2, 3, 1))
    so = so.view(b, hk, maxq, grp, -1)
    seen = torch.full((b, maxq), -1, device=DEV, dtype=torch.long)
    seen[seq, row] = j
    so.masked_fill_(torch.arange(so.shape[-1], device=DEV) > seen[:, None, :, None, None], -math.inf)
    # One softmax over both parts.
    mo = so.amax(-1)[seq, :, row]                       # [n][hk][grp]
    top = torch.maximum(mo, sp.amax(-1).view(hk, n, grp).transpose(0, 1)) if c["prefix"] else mo
    full = torch.zeros(b, maxq, hk, grp, device=DEV)
    full[seq, row] = top
    po = so.sub_(full.transpose(1, 2)[..., None]).exp_()
    pp = sp.sub_(top.transpose(0, 1).reshape(hk, n * grp, 1)).exp_()
    total = po.sum(-1)[seq, :, row] + pp.sum(-1).view(hk, n, grp).transpose(0, 1)
    out = torch.matmul(po.view(b, hk, maxq * grp, -1), vo.transpose(1, 2)).view(b, hk, maxq, grp, d)[seq, :, row]
    out = out + torch.matmul(pp, vp.transpose(0, 1)).view(hk, n, grp, d).transpose(0, 1)
    s["out"].copy_((out / total[..., None]).view(n, hq, d))
    s["lse"].copy_((top + total.log()).view(n, hq))
    return {"out": s["out"], "lse": s["lse"]}


def _plain_sample(s):
    x = s["logits"].float()
    rows, vocab = x.shape
    t = s["temperature"]
    greedy = t == 0
    z = x * torch.where(greedy, torch.ones_like(t), 1.0 / t)[:, None]
    w = torch.exp(z - z.amax(1, keepdim=True))
    fixed = torch.round(w * FIX).long()
    z_sorted, order = torch.sort(z, dim=1, descending=True, stable=True)
    ws, fs = w.gather(1, order), fixed.gather(1, order)
    rank = torch.arange(vocab, device=DEV)[None]
    keep = (fs > 0) & (~greedy[:, None] | (rank == 0))
    if s["top_k"] is not None:
        k = s["top_k"][:, None]
        keep &= (rank < k) | (k <= 0)
    if s["top_p"] is not None:
        fs_k = torch.where(keep, fs, 0)
        before = torch.cumsum(fs_k, 1) - fs_k
        p = s["top_p"].double()[:, None]
        keep &= (before.double() < p * fs_k.sum(1, keepdim=True).double()) | (rank == 0) | (p >= 1)
    if s["min_p"] is not None:
        keep &= ws >= s["min_p"][:, None]
    mask = torch.zeros_like(keep).scatter_(1, order, keep)
    kept = torch.where(mask, fixed, 0)
    total = kept.sum(1)
    target = torch.minimum((s["u"].double() * total.double()).long(), total - 1)
    token = (torch.cumsum(kept, 1) <= target[:, None]).sum(1)
    probs = kept.float() / total.float()[:, None]
    s["out"].copy_(token)
    s["kept"].copy_(mask.sum(1))
    s["logprob"].copy_(probs.gather(1, token[:, None])[:, 0].log())
    if s["probs"] is not None:
        s["probs"].copy_(probs)
    return {"token": s["out"], "kept": s["kept"], "logprob": s["logprob"]} | ({"probs": s["probs"]} if s["probs"] is not None else {})


# --------------------------------------------------------------------------- the definition, 64 bits --

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "sample": _exact_sample}[case["op"]](case, s)


def _exact_append(c, s):
    k, v, q = s["k_cache"].double(), s["v_cache"].double(), s["q"].double()
    rot, start = c["rot"], s["q_start"].tolist()

    def turn(x, pos):  # as complex numbers
        if rot == 0 or x.shape[0] == 0:
            return x
        a = s["rope"][pos].double()
        e = torch.complex(a[:, : rot // 2], a[:, rot // 2:])[:, None]
        r = x[..., :rot]
        z = torch.view_as_complex(r.reshape(*r.shape[:-1], rot // 2, 2).contiguous()) if c["inter"] else torch.complex(
            r[..., : rot // 2].contiguous(), r[..., rot // 2:].contiguous())
        z = z * e
        r = torch.view_as_real(z).flatten(-2) if c["inter"] else torch.cat((z.real, z.imag), -1)
        return torch.cat((r, x[..., rot:]), -1)

    for b, length in enumerate(s["kv_len"].tolist()):
        lo, hi = start[b], start[b + 1]
        j = torch.arange(length - (hi - lo), length, device=DEV)
        pages, at = s["table"][b].long()[j // c["page"]], j % c["page"]
        k[pages, at] = turn(s["k"][lo:hi].double(), c["prefix"] + j)
        v[pages, at] = s["v"][lo:hi].double()
        q[lo:hi] = turn(s["q"][lo:hi].double(), c["prefix"] + j)
    return {"q": q, "k": k, "v": v}


def _exact_attend(c, s):
    hq, hk, d, page = c["q_heads"], c["kv_heads"], c["dim"], c["page"]
    if work(c)["flops"] > 4e11:
        return None
    out = torch.zeros(s["tokens"], hq, d, device=DEV, dtype=torch.float64)
    lse = torch.zeros(s["tokens"], hq, device=DEV, dtype=torch.float64)
    start, lens = s["q_start"].tolist(), s["kv_len"].tolist()
    pre = s["prefix_table"].long()
    for h in range(hk):
        kp = s["k_cache"][pre, :, h].double().reshape(-1, d)[: c["prefix"]]
        vp = s["v_cache"][pre, :, h].double().reshape(-1, d)[: c["prefix"]]
        heads = slice(h * hq // hk, (h + 1) * hq // hk)
        # The scores of the shared part for all rows at once, in slices that fit.
        for b, length in enumerate(lens):
            lo, hi = start[b], start[b + 1]
            if hi == lo:
                continue
            own_pages = s["table"][b].long()[: -(-length // page)]
            k = torch.cat((kp, s["k_cache"][own_pages, :, h].double().reshape(-1, d)[:length]))
            v = torch.cat((vp, s["v_cache"][own_pages, :, h].double().reshape(-1, d)[:length]))
            x = torch.einsum("qgd,kd->gqk", s["q"][lo:hi, heads].double(), k) * d ** -0.5
            last = c["prefix"] + length - (hi - lo) + torch.arange(hi - lo, device=DEV)
            x = torch.where(torch.arange(len(k), device=DEV)[None, None] <= last[None, :, None], x, -math.inf)
            out[lo:hi, heads] = torch.einsum("gqk,kd->qgd", torch.softmax(x, -1), v)
            lse[lo:hi, heads] = torch.logsumexp(x, -1).T
    return {"out": out, "lse": lse}


def _exact_sample(c, s):
    """Row by row on the host in 64 bits; the weights' fixed-point unit is part of the definition."""
    rows = c["rows"]
    value = lambda name, i, off: off if s[name] is None else s[name][i].item()  # noqa: E731
    logprob = np.zeros(rows)
    probs = np.zeros((rows, c["vocab"])) if c["probs"] else None
    logits, u = s["logits"].double().cpu().numpy(), s["u"].double().cpu().numpy()
    for i in range(rows):
        t = float(s["temperature"][i])
        x = logits[i]
        if t == 0:
            kept = np.array([np.argmax(x)])
            f = np.ones(1)
        else:
            # The scaled scores are 32-bit numbers by definition: ties and ranks are among those.
            z = (x.astype(np.float32) * np.float32(1.0 / np.float32(t))).astype(np.float64)
            k, p, least = value("top_k", i, 0), value("top_p", i, 1.0), value("min_p", i, 0.0)
            order = np.argsort(-z, kind="stable")[: k if k > 0 else None]
            w = np.exp(z[order] - z[order[0]])
            f = np.rint(w * FIX)
            n = len(f)
            if p < 1:
                n = max(1, int(np.searchsorted(np.cumsum(f) - f, p * f.sum(), side="left")))
            n = min(n, int((w >= least).sum()), int((f > 0).sum()))
            by_index = np.argsort(order[:n])
            kept, f = order[:n][by_index], f[:n][by_index]
        j = int(np.searchsorted(np.cumsum(f), np.floor(u[i] * f.sum()), side="right"))
        logprob[i] = np.log(f[min(j, len(f) - 1)] / f.sum())
        if probs is not None:
            probs[i, kept] = f / f.sum()
    return {"token": None, "kept": None, "logprob": torch.from_numpy(logprob)} | ({"probs": torch.from_numpy(probs)} if probs is not None else {})
