"""A serving loop of one small transformer layer on the library's kernels.

Prompts of different lengths are prefilled together, then every sequence decodes a
token at a time.  A step is the calls a server makes:

    gemm (qkv)  ->  kv_append  ->  kv_attention  ->  gemm (o)  ->  swiglu, gemm (FFN)
    ->  gemm (LM head, fp32 logits)  ->  sample

with keys and values in a paged cache of 8-bit codes.  Weights are random; run it on a
GB300 from the repository's root, after the library is built:

    python examples/serve_step.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import roofline_driven_optimisation_gb300 as g  # noqa: E402

BF16 = torch.bfloat16


class Layer:
    """One layer, an embedding and an LM head: heads query heads over kv_heads shared ones."""

    def __init__(self, heads=16, kv_heads=4, dim=64, ffn=2048, vocab=32000, positions=4096, seed=0):
        self.heads, self.kv_heads, self.dim, self.vocab = heads, kv_heads, dim, vocab
        self.width = heads * dim
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=gen, device="cuda") / rows ** 0.5).to(BF16)
        self.embedding = torch.randn(vocab, self.width, generator=gen, device="cuda").to(BF16)
        self.qkv = weight(self.width, (heads + 2 * kv_heads) * dim)
        self.o, self.gate, self.up = weight(self.width, self.width), weight(self.width, ffn), weight(self.width, ffn)
        self.down, self.head = weight(ffn, self.width), weight(self.width, vocab) * 4
        angle = torch.arange(positions, device="cuda")[:, None] * \
            10000.0 ** (-torch.arange(0, dim, 2, device="cuda") / dim)
        self.cos, self.sin = torch.cos(angle).contiguous(), torch.sin(angle).contiguous()

    def step(self, cache, tokens, base, lengths, start, max_new):
        """Logits (fp32) of every row: tokens[start[b]:start[b+1]] are sequence b's new
        ones, behind the base[b] it has in the cache."""
        x = self.embedding[tokens.long()]
        rows = x.shape[0]
        qkv = torch.empty(rows, self.qkv.shape[1], dtype=BF16, device="cuda")
        g.gemm(x, self.qkv, qkv)
        q, k, v = (t.unflatten(1, (-1, self.dim)) for t in qkv.split(
            [self.width, self.kv_heads * self.dim, self.kv_heads * self.dim], 1))
        turned = torch.empty(rows, self.heads, self.dim, dtype=BF16, device="cuda")
        g.kv_append(cache, q, k, v, self.cos, self.sin, base, turned, start=start, max_new=max_new)
        out = torch.empty_like(turned)
        g.kv_attention(cache, turned, out, lengths, start=start, max_new=max_new)
        x = x.clone()
        g.gemm(out.flatten(1), self.o, x, beta=1.0)                    # added to the residual
        hidden = torch.empty(rows, self.gate.shape[1], dtype=BF16, device="cuda")
        g.swiglu(x, self.gate, self.up, hidden)
        g.gemm(hidden, self.down, x, beta=1.0)
        logits = torch.empty(rows, self.vocab, dtype=torch.float32, device="cuda")
        g.gemm(x, self.head, logits, alpha=self.width ** -0.5)
        return logits


def new_cache(layer, lengths, page=64, spare=4):
    """Pages for sequences that may grow to `lengths` tokens, in no particular order."""
    need = [-(-n // page) for n in lengths]
    pages = sum(need) + spare
    order = torch.randperm(pages)
    table = torch.zeros(len(need), max(need), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    codes = torch.empty(2, pages, layer.kv_heads, page, layer.dim, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(2, pages, layer.kv_heads, device="cuda")
    return g.KVCache(codes[0], codes[1], scales[0], scales[1], table.cuda())


def serve(prompts, steps, layer=None, seed=1):
    """Prefill the prompts (lists of token numbers) and decode `steps` tokens of each:
    (tokens [sequences][steps], their log-probabilities)."""
    layer = layer or Layer()
    n = len(prompts)
    ints = dict(dtype=torch.int32, device="cuda")
    count = torch.tensor([len(p) for p in prompts], **ints)
    cache = new_cache(layer, [len(p) + steps for p in prompts])
    gen = torch.Generator(device="cuda").manual_seed(seed)
    u = torch.rand(steps, n, generator=gen, device="cuda")
    token = torch.empty(steps, n, **ints)
    logprob = torch.empty(steps, n, device="cuda")
    settings = dict(temperature=torch.full((n,), 0.8, device="cuda"), top_k=torch.full((n,), 50, **ints),
                    top_p=torch.full((n,), 0.95, device="cuda"), min_p=torch.full((n,), 0.02, device="cuda"))
    start = torch.zeros(n + 1, **ints)
    start[1:] = torch.cumsum(count, 0)
    rows = torch.tensor([t for p in prompts for t in p], **ints)
    logits = layer.step(cache, rows, torch.zeros(n, **ints), count, start, max(len(p) for p in prompts))
    logits = logits[start[1:].long() - 1]                              # the last row of each prompt
    length = count.clone()
    for i in range(steps):
        g.sample(logits, u[i], token[i], logprob[i], **settings)
        if i + 1 < steps:
            base = length.clone()
            length += 1
            logits = layer.step(cache, token[i], base, length, None, 1)
    return token.T, logprob.T


if __name__ == "__main__":
    torch.cuda.set_device(0)
    chosen, lp = serve([[1, 5, 9], list(range(100, 400)), [7]], steps=16)
    torch.cuda.synchronize()
    status, where = g.device_status()
    for b, (t, p) in enumerate(zip(chosen.tolist(), lp.tolist())):
        print(f"sequence {b}: tokens {t}  mean log-probability {sum(p) / len(p):.3f}")
    print(f"device status {status}")
