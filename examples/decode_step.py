"""A decode loop on random weights: several continuations of one prompt.

Every layer is: projection -> kv_append (rotary positions, paged cache) -> prefix_attention (the prompt is
stored once and shared by all sequences) -> projection -> moe forward (routed MXFP4 experts, added into the
residual).  The last layer's output gives logits, and sample draws a token per sequence from given uniform
numbers.  The dense projections are plain torch products.

    python examples/decode_step.py [--sequences 8] [--prompt 300] [--steps 16] [--private] [--mx]

``--private`` gives every sequence its own copy of the prompt instead: the same computation from a larger cache,
in other tiles (rounding may part the drawn tokens after some steps).

``--mx`` has the dense half in microscaled formats, too: projections and head in MXFP4, their inputs in MXFP8.
rms_norm writes the codes that mx_linear reads, the output projection adds into the fp32 residual, and the
prompt's tokens are scored with token_logprobs.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp4_routed_expert_moe_gb300 as moe  # noqa: E402


class Layer:
    """Weights of one layer and its part of the cache."""

    def __init__(self, m: "Model", gen):
        def normal(*shape):
            return (torch.randn(*shape, generator=gen, device="cuda") * shape[-1] ** -0.5).bfloat16()

        self.qkv = m.weights(normal((m.q_heads + 2 * m.kv_heads) * m.dim, m.hidden))
        self.out = m.weights(normal(m.hidden, m.q_heads * m.dim))
        self.router = torch.randn(m.experts, m.hidden, generator=gen, device="cuda") * m.hidden ** -0.5
        # Random MXFP4 experts: any codes, scales around 2^-7.
        self.table = moe.ExpertTable(m.experts, m.hidden, m.inter)
        self.table.blob.random_(0, 256, generator=gen)
        for e in range(m.experts):
            for j in (1, 3, 5):
                self.table.tensor(e, j).random_(118, 121, generator=gen)
        shape = (m.pages, m.page_size, m.kv_heads, m.dim)
        self.cache = moe.KVCache(torch.zeros(shape, dtype=torch.bfloat16, device="cuda"),
                                 torch.zeros(shape, dtype=torch.bfloat16, device="cuda"))


class Model:
    def __init__(self, layers=2, hidden=512, q_heads=8, kv_heads=2, dim=64, experts=16, top_k=2, inter=256, vocab=4099,
                 pages=512, page_size=16, positions=4096, seed=0, mx=False):
        self.mx = mx
        self.hidden, self.q_heads, self.kv_heads, self.dim = hidden, q_heads, kv_heads, dim
        self.experts, self.top_k, self.inter, self.pages, self.page_size = experts, top_k, inter, pages, page_size
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.embedding = torch.randn(vocab, hidden, generator=gen, device="cuda")
        self.head = self.weights((torch.randn(vocab, hidden, generator=gen, device="cuda") * 3 * hidden ** -0.5).bfloat16())
        self.rope = moe.rope_table(positions, dim)
        self.layers = [Layer(self, gen) for _ in range(layers)]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")  # sticky: one look at the end

    def weights(self, w):
        """bf16 weights as the model keeps them."""
        if not self.mx:
            return w
        q = moe.MXMatrix.empty(*w.shape, "e2m1")
        moe.mx_quantize(w, q)
        return q

    def norm(self, h, out=None):
        """The norm of the residual: bf16, or the MXFP8 codes for a product."""
        if out is None:
            return torch.nn.functional.rms_norm(h, (self.hidden,)).bfloat16()
        moe.rms_norm(h, out)
        return out

    def forward_mx(self, tokens, batch: moe.KVBatch):
        """:meth:`forward` with the dense half in microscaled formats."""
        n = tokens.shape[0]
        h = self.embedding[tokens].float().contiguous()  # the residual, fp32
        bf16 = dict(dtype=torch.bfloat16, device="cuda")
        widths = (self.q_heads * self.dim, self.kv_heads * self.dim, self.kv_heads * self.dim)
        x8, a8 = moe.MXMatrix.empty(n, self.hidden, "e4m3"), moe.MXMatrix.empty(n, widths[0], "e4m3")
        qkv, x = torch.empty(n, sum(widths), **bf16), torch.empty(n, self.hidden, **bf16)
        attn = torch.empty(n, self.q_heads, self.dim, **bf16)
        ws = torch.empty(moe.attention_workspace_bytes(self.layers[0].cache, batch, self.q_heads), dtype=torch.uint8, device="cuda")
        shape = moe.shape(n, self.hidden, self.experts, self.inter, self.top_k)
        moe_ws = torch.empty(moe.workspace_bytes(n, self.hidden, self.experts, self.inter, self.top_k), dtype=torch.uint8,
                             device="cuda")
        for layer in self.layers:
            moe.mx_linear(self.norm(h, x8), layer.qkv, qkv, status=self.status)
            q, k, v = (t.view(n, -1, self.dim) for t in qkv.split(widths, 1))
            moe.kv_append(layer.cache, batch, k, v, q=q, q_out=q, rope=self.rope, rot_dim=self.dim, status=self.status)
            moe.prefix_attention(layer.cache, batch, q, attn, ws, status=self.status)
            moe.mx_quantize(attn.view(n, -1), a8)
            moe.mx_linear(a8, layer.out, h, add=h, status=self.status)
            moe.forward(shape, self.norm(h, x), layer.router, None, layer.table.desc, None, h, True, moe_ws)
        logits = torch.empty(n, self.embedding.shape[0], device="cuda")
        moe.mx_linear(self.norm(h, x8), self.head, logits, status=self.status)
        return logits

    def forward(self, tokens, batch: moe.KVBatch):
        """Logits [tokens][vocab] of new tokens, whose keys and values join the cache."""
        if self.mx:
            return self.forward_mx(tokens, batch)
        n = tokens.shape[0]
        h = self.embedding[tokens].float().contiguous()  # the residual, fp32
        attn = torch.empty(n, self.q_heads, self.dim, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(moe.attention_workspace_bytes(self.layers[0].cache, batch, self.q_heads), dtype=torch.uint8, device="cuda")
        shape = moe.shape(n, self.hidden, self.experts, self.inter, self.top_k)
        moe_ws = torch.empty(moe.workspace_bytes(n, self.hidden, self.experts, self.inter, self.top_k), dtype=torch.uint8,
                             device="cuda")
        for layer in self.layers:
            x = torch.nn.functional.rms_norm(h, (self.hidden,)).bfloat16()
            q, k, v = (x @ layer.qkv.T).split((self.q_heads * self.dim, self.kv_heads * self.dim, self.kv_heads * self.dim), 1)
            q, k, v = (t.view(n, -1, self.dim) for t in (q, k, v))
            moe.kv_append(layer.cache, batch, k, v, q=q, q_out=q, rope=self.rope, rot_dim=self.dim, status=self.status)
            moe.prefix_attention(layer.cache, batch, q, attn, ws, status=self.status)
            h += (attn.view(n, -1) @ layer.out.T).float()
            x = torch.nn.functional.rms_norm(h, (self.hidden,)).bfloat16()
            moe.forward(shape, x, layer.router, None, layer.table.desc, None, h, True, moe_ws)
        return torch.nn.functional.rms_norm(h, (self.hidden,)).bfloat16() @ self.head.T


def score(model: Model, text, top=0, pages=None):
    """Of a text's tokens but the first: log probability, rank and the distribution's entropy, and with ``top`` the
    best alternatives' ids and log probabilities.  The text's keys and values are written to ``pages`` (ids; the cache's
    first pages without), whatever those held: between decode steps, pages that no sequence uses."""
    n, size = text.shape[0], model.page_size
    need = -(-n // size)
    pages = list(range(need)) if pages is None else [int(p) for p in pages]
    if n < 2 or n > model.rope.shape[0]:
        raise ValueError(f"a text of 2 to {model.rope.shape[0]} tokens, not {n}")
    if len(pages) < need or len(set(pages)) < len(pages) or not all(0 <= p < model.pages for p in pages):
        raise ValueError(f"a text of {n} tokens takes {need} different pages of {model.pages}, not {pages}")
    i32, f32 = dict(dtype=torch.int32, device="cuda"), dict(device="cuda")
    table = torch.tensor([pages[:need]], **i32)
    batch = moe.KVBatch(torch.full((1,), n, **i32), table, tokens=n, max_q=n, q_start=torch.tensor([0, n], **i32))
    logits = model.forward(text, batch)[:-1]
    out = dict(logprob=torch.empty(n - 1, **f32), rank=torch.empty(n - 1, **i32), entropy=torch.empty(n - 1, **f32))
    if top:
        out |= dict(top_ids=torch.empty(n - 1, top, **i32), top_logprobs=torch.empty(n - 1, top, **f32))
    moe.token_logprobs(logits, text[1:].to(torch.int32), **out)
    return out


def generate(model: Model, prompt, sequences: int, steps: int, private=False, seed=1):
    """Tokens [sequences][steps] and the first step's logits: continuations of one prompt, drawn with
    temperature 0.8, top-k 50, top-p 0.95."""
    size = model.page_size
    n = prompt.shape[0]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    prompt_pages = -(-n // size)
    own = n if private else 0
    width = -(-(own + steps) // size)
    first = 0 if private else prompt_pages
    table = torch.arange(first, first + sequences * width, **i32).view(sequences, width)
    prefix = torch.arange(prompt_pages, **i32)
    # The prompt once (or, with private copies, once per sequence): all its tokens are new.
    copies = sequences if private else 1
    batch = moe.KVBatch(torch.full((copies,), n, **i32), table if private else prefix[None], tokens=copies * n, max_q=n,
                        q_start=torch.arange(copies + 1, **i32) * n)
    logits = model.forward(prompt.repeat(copies), batch).view(copies, n, -1)[:, -1].expand(sequences, -1).contiguous()
    start = logits.float().clone()
    kv_len = torch.full((sequences,), own, **i32)
    batch = moe.KVBatch(kv_len, table, **({} if private else dict(prefix_table=prefix, prefix_len=n)))
    f32 = dict(device="cuda")
    temperature, top_p = torch.full((sequences,), 0.8, **f32), torch.full((sequences,), 0.95, **f32)
    top_k = torch.full((sequences,), 50, **i32)
    tokens = torch.empty(sequences, **i32)
    logprob = torch.empty(sequences, **f32)
    out, total = [], torch.zeros(sequences, **f32)
    for step in range(steps):
        u = torch.rand(sequences, generator=gen, device="cuda")
        moe.sample(logits, u, tokens, temperature=temperature, top_k=top_k, top_p=top_p, logprob=logprob)
        out.append(tokens.clone())
        total += logprob
        if step + 1 < steps:
            kv_len += 1  # in place: the batch's lengths are read on the device
            logits = model.forward(tokens, batch)
    if int(model.status.item()) != moe.MOE_OK:
        raise moe.MoeError(int(model.status.item()), "decode step")
    return torch.stack(out, 1), start, total


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--sequences", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--private", action="store_true")
    ap.add_argument("--mx", action="store_true")
    a = ap.parse_args()
    model = Model(mx=a.mx)
    prompt = torch.randint(0, model.embedding.shape[0], (a.prompt,), generator=torch.Generator().manual_seed(2)).cuda()
    if a.mx:
        s = score(model, prompt)
        print(f"prompt: {s['logprob'].sum().item():.3f}, median rank {s['rank'].median().item()}, mean entropy {s['entropy'].mean().item():.3f}")
    tokens, _, total = generate(model, prompt, a.sequences, a.steps, a.private)
    for t, lp in zip(tokens.tolist(), total.tolist()):
        print(f"{lp:9.3f}  {' '.join(map(str, t))}")


if __name__ == "__main__":
    main()
