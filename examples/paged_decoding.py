"""Decoding over a paged key-value cache: the operators of a decode step, together.

A small transformer with random weights (bf16; projections by gemm_bounded).
One cache holds the keys and values of all layers: (2 * layers planes, pages,
slots, heads, depth).  Per step and row:

    pages_reserve          a page for rows whose last one is full
    qk_norm_rope_append    norm and rotation; keys and values into the pages
    paged_attention        the new token against its cached ones

and between steps pages_fork (several continuations of one prompt), pages_free
(rows that ended) and pages_compact (the pool packed).  Tables, lengths and
counts stay on the device throughout.

    python examples/paged_decoding.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import scatter_tile_gather_amd as stg  # noqa: E402


class Decoder:
    def __init__(self, rows=8, layers=2, heads=2, group=4, depth=64, vocab=512, pages=96, slots=16, width=24, seed=0,
                 device="cuda:0"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.heads, self.q_heads, self.depth, self.slots, self.device = heads, heads * group, depth, slots, device
        self.dim = self.q_heads * depth
        qkv = (self.q_heads + 2 * heads) * depth

        def weight(*shape):
            return (torch.randn(shape, generator=g, device=device) * shape[0] ** -0.5).to(torch.bfloat16)

        self.embed = weight(vocab, self.dim) * vocab ** 0.5
        self.layers = [dict(qkv=weight(self.dim, qkv), out=weight(self.dim, self.dim),
                            qn=1 + 0.1 * torch.randn(depth, generator=g, device=device),
                            kn=1 + 0.1 * torch.randn(depth, generator=g, device=device)) for _ in range(layers)]
        self.unembed = weight(self.dim, vocab)
        freq, self.gain = stg.rope_frequencies(depth, scaling="yarn", factor=4.0)
        self.freq = torch.from_numpy(freq).to(device)
        i32 = dict(dtype=torch.int32, device=device)
        self.cache = torch.zeros((2 * layers, pages, slots, heads, depth), dtype=torch.bfloat16, device=device)
        self.planes = self.cache.view(2 * layers, pages, slots * heads * depth)
        self.table = torch.full((rows, width), -1, **i32)
        self.lens = torch.zeros(rows, **i32)
        self.refs = torch.zeros(pages, **i32)
        self.short = torch.zeros(1, **i32)  # pages that were missing at the last reserve or fork

    def step(self, tokens, active):
        """One token for every active row (int32 0 / 1 per row); returns the logits."""
        stg.pages_reserve(self.table, self.lens, active, self.refs, self.slots, shortfall=self.short)
        rows = torch.where(active > 0, torch.arange(len(active), dtype=torch.int32, device=self.device), -1)
        after = self.lens + active
        x = self.embed[tokens.long()]
        for i, w in enumerate(self.layers):
            qkv = stg.gemm_bounded(x, w["qkv"]).view(len(tokens), -1, self.depth)
            q, k, v = qkv.split([self.q_heads, self.heads, self.heads], 1)
            kc, vc = self.cache[2 * i], self.cache[2 * i + 1]
            q = stg.qk_norm_rope_append(q, k, v, self.lens, self.freq, kc, vc, self.table, rows=rows, q_weight=w["qn"],
                                        k_weight=w["kn"], rope_scale=self.gain)
            y = stg.paged_attention(q, kc, vc, self.table, after)
            x = x + stg.gemm_bounded(y.view(len(tokens), self.dim), w["out"])
        self.lens.copy_(after)
        return stg.gemm_bounded(x, self.unembed, out_dtype=torch.float32)

    def fork(self, parents, children):
        stg.pages_free(self.table, self.lens, self.refs, children)
        stg.pages_fork(self.planes, self.table, self.lens, self.refs, self.slots, parents, children,
                       shortfall=self.short)

    def free(self, rows):
        stg.pages_free(self.table, self.lens, self.refs, rows)

    def compact(self):
        return stg.pages_compact(self.planes, self.table, self.refs)


def main():
    d = Decoder()
    i32 = dict(dtype=torch.int32, device=d.device)
    rows = len(d.lens)
    g = torch.Generator(device=d.device).manual_seed(1)
    prompts = torch.randint(0, 512, (2, 37), generator=g, **i32)
    # two prompts of different lengths, token by token, in rows 0 and 4
    for t in range(37):
        tokens, active = torch.zeros(rows, **i32), torch.zeros(rows, **i32)
        for row, prompt, n in ((0, prompts[0], 37), (4, prompts[1], 22)):
            tokens[row], active[row] = prompt[t], int(t < n)
        logits = d.step(tokens, active)
    # three more continuations of the first prompt
    d.fork(torch.tensor([0, 0, 0], **i32), torch.tensor([1, 2, 3], **i32))
    alive = torch.tensor([1, 1, 1, 1, 1, 0, 0, 0], **i32)
    tokens = torch.randint(0, 512, (rows,), generator=g, **i32)
    for _ in range(20):
        logits = d.step(tokens, alive)
        tokens = logits.argmax(1).to(torch.int32)
    # one of them ends, and the pool is packed
    d.free(torch.tensor([2], **i32))
    alive[2] = 0
    d.compact()
    logits = d.step(tokens, alive)
    live = int((d.refs > 0).sum())
    assert int(d.short) == 0 and bool(torch.isfinite(logits[alive > 0]).all())
    print(f"lengths {d.lens.tolist()}, {live} pages live, last of them page {int((d.refs > 0).nonzero().max())}")


if __name__ == "__main__":
    main()
