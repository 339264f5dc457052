"""Plain 64-bit forms of the operators of moe_serve.h, in numpy, and the inputs of their tests."""
from __future__ import annotations

import math

import numpy as np


def torch():
    import torch as _t
    return _t


def bf16(x):
    """numpy array -> (bf16 cuda tensor, its values in fp64)."""
    t = torch()
    b = t.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to("cuda").bfloat16()
    return b, b.double().cpu().numpy()


class Paged:
    """A cache with pages handed out in a random order, NaN in every row that no token owns."""

    def __init__(self, rng, lens, prefix, page, heads, dim, head_major=False, spare=2, capacity=0):
        t = torch()
        self.page, self.heads, self.dim, self.prefix, self.lens = page, heads, dim, prefix, list(lens)
        npre = -(-prefix // page)
        own = [-(-n // page) for n in lens]
        self.pages = npre + sum(own) + spare
        order = rng.permutation(self.pages).astype(np.int32)
        self.prefix_table = order[:npre].copy()
        width = max(1, max(own), -(-capacity // page))  # a table may have room for more
        self.table = np.full((len(lens), width), -7, dtype=np.int32)  # entries past a length are never read
        at = npre
        for b, n in enumerate(own):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (self.pages, heads, page, dim) if head_major else (self.pages, page, heads, dim)
        self.k_all = t.full(shape, float("nan"), dtype=t.bfloat16, device="cuda")
        self.v_all = t.full(shape, float("nan"), dtype=t.bfloat16, device="cuda")
        self.k, self.v = (x.transpose(1, 2) if head_major else x for x in (self.k_all, self.v_all))

    def fill(self, table, n, k, v):
        """Put n tokens' bf16 keys and values [n][heads][dim] into the pages of `table`."""
        t = torch()
        j = np.arange(n)
        pages, at = t.from_numpy(table[j // self.page].astype(np.int64)).cuda(), t.from_numpy(j % self.page).cuda()
        self.k[pages, at] = k
        self.v[pages, at] = v


def rotate(x, pos, rope, rot, inter):
    """x [n][heads][dim] fp64, rope rows fp64."""
    y = x.copy()
    if rot == 0:
        return y
    c, s = rope[pos, : rot // 2][:, None], rope[pos, rot // 2:][:, None]
    i = np.arange(rot // 2)
    ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


def attend(q, k, v, visible, scale):
    """q [rows][dim] against k, v [n][dim]; row i sees the first visible[i] tokens.  Returns out, lse, the
    softmax-weighted |v| and the largest sum |q_d k_jd| of a seen token (for error bounds)."""
    rows, dim = q.shape
    out, lse = np.zeros((rows, dim)), np.full(rows, -np.inf)
    weight, mag = np.zeros((rows, dim)), np.zeros(rows)
    for i in range(rows):
        n = visible[i]
        if n <= 0:
            continue
        x = scale * (k[:n] @ q[i])
        m = x.max()
        p = np.exp(x - m)
        l = p.sum()
        out[i], weight[i] = p @ v[:n] / l, p @ np.abs(v[:n]) / l
        lse[i] = m + math.log(l)
        mag[i] = (np.abs(k[:n]) @ np.abs(q[i])).max()
    return out, lse, weight, mag


def sample_row(z, w, u, top_k=0, top_p=1.0, min_p=0.0):
    """One row by the definition: z fp32 scaled scores (no NaN), w = exp(z - max) in fp32.  Returns the
    token, the number kept, and the kept integer weights by index."""
    fixed = np.rint(w.astype(np.float64) * 2.0 ** 31).astype(np.int64)
    order = np.lexsort((np.arange(len(z)), -z.astype(np.float64)))
    order = order[fixed[order] > 0]
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1.0:
        f = fixed[order]
        before = np.cumsum(f) - f
        keep = before.astype(np.float64) < float(np.float32(top_p)) * float(f.sum())
        keep[0] = True
        order = order[keep]
    if min_p > 0.0:
        order = order[w[order] >= min(np.float32(min_p), np.float32(1))]
    kept = np.zeros(len(z), dtype=np.int64)
    kept[order] = fixed[order]
    total = int(kept.sum())
    target = min(int(math.floor(float(np.float32(u)) * float(total))), total - 1)
    token = int(np.searchsorted(np.cumsum(kept), target, side="right"))
    return token, len(order), kept
