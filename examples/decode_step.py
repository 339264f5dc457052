"""A decode loop on random weights: several continuations of one prompt.

Every layer is: projection -> kv_append (rotary positions, paged cache) -> prefix_attention (the prompt is
stored once and shared by all sequences) -> projection -> moe forward (routed MXFP4 experts, added into the
residual).  The last layer's output gives logits, and sample draws a token per sequence from given uniform
numbers.  The dense projections are plain torch products.

    python examples/decode_step.py [--sequences 8] [--prompt 300] [--steps 16] [--private]

``--private`` gives every sequence its own copy of the prompt instead: the same computation from a larger cache,
in other tiles (rounding may part the drawn tokens after some steps).
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

        self.qkv = normal((m.q_heads + 2 * m.kv_heads) * m.dim, m.hidden)
        self.out = normal(m.hidden, m.q_heads * m.dim)
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
                 pages=512, page_size=16, positions=4096, seed=0):
        self.hidden, self.q_heads, self.kv_heads, self.dim = hidden, q_heads, kv_heads, dim
        self.experts, self.top_k, self.inter, self.pages, self.page_size = experts, top_k, inter, pages, page_size
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.embedding = torch.randn(vocab, hidden, generator=gen, device="cuda")
        self.head = (torch.randn(vocab, hidden, generator=gen, device="cuda") * 3 * hidden ** -0.5).bfloat16()
        self.rope = moe.rope_table(positions, dim)
        self.layers = [Layer(self, gen) for _ in range(layers)]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")  # sticky: one look at the end

    def forward(self, tokens, batch: moe.KVBatch):
        """Logits [tokens][vocab] of new tokens, whose keys and values join the cache."""
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
    a = ap.parse_args()
    model = Model()
    prompt = torch.randint(0, model.embedding.shape[0], (a.prompt,), generator=torch.Generator().manual_seed(2)).cuda()
    tokens, _, total = generate(model, prompt, a.sequences, a.steps, a.private)
    for t, lp in zip(tokens.tolist(), total.tolist()):
        print(f"{lp:9.3f}  {' '.join(map(str, t))}")


if __name__ == "__main__":
    main()
