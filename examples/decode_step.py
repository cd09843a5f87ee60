"""A small mixture-of-experts decoder over quantized weights: the library's calls put together
as a serving loop makes them (run: python examples/decode_step.py).

Weights are random.  A prompt goes in at once (qmm_t for its projections, attention of all its
queries), then every step feeds one token per sequence: embedding, and per layer the
projections, kv_append, kv_attend and the expert layer, then lm_head and sampling.  Keys and
values live in 4 bits, in pages that sequences take from one pool.  RMS norms and residual
additions are torch's.
"""
from __future__ import annotations

import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_affine_quantized_qmv_amd as q  # noqa: E402


@dataclass
class Config:
    layers: int = 2
    hidden: int = 512
    heads: int = 8
    kv_heads: int = 2
    head_dim: int = 64
    experts: int = 8
    top_k: int = 2
    inter: int = 256
    vocab: int = 4096
    bits: int = 4
    group: int = 64
    page: int = 16
    pages: int = 256
    dtype: torch.dtype = torch.bfloat16


class Decoder:
    def __init__(self, cfg: Config, device="cuda", seed=0):
        self.cfg, self.device = cfg, torch.device(device)
        g = torch.Generator(device=self.device).manual_seed(seed)

        def weight(n, k, std=None):
            w = torch.randn(n, k, generator=g, device=self.device) * (k ** -0.5 if std is None else std)
            return q.quantize(w, cfg.group, cfg.bits, cfg.dtype)

        def experts(n, k):
            return q.ExpertWeights.stack([weight(n, k) for _ in range(cfg.experts)])

        self.table = weight(cfg.vocab, cfg.hidden, 1.0)
        self.head = weight(cfg.vocab, cfg.hidden)
        kv = cfg.kv_heads * cfg.head_dim
        self.layers = [dict(qkv=weight(cfg.heads * cfg.head_dim + 2 * kv, cfg.hidden),
                            out=weight(cfg.hidden, cfg.heads * cfg.head_dim),
                            router=weight(cfg.experts, cfg.hidden),
                            gate=experts(cfg.inter, cfg.hidden), up=experts(cfg.inter, cfg.hidden),
                            down=experts(cfg.hidden, cfg.inter),
                            cache=q.kv_cache(cfg.pages, cfg.page, cfg.kv_heads, cfg.head_dim, 32, cfg.dtype, device))
                       for _ in range(cfg.layers)]
        self.free = list(range(cfg.pages))

    def norm(self, x):
        return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)

    def moe(self, x, layer):
        """The expert layer: few rows, or the rows of a prompt."""
        call = q.moe if x.shape[0] <= 32 else q.moe_prompt
        return call(x, q.qmm_t(x, layer["router"]), layer["gate"], layer["up"], layer["down"], self.cfg.top_k)

    def logits(self, tokens, slots, table, lengths, longest):
        """Logits of the last token of each sequence.  tokens int32 [batch, n]: the n tokens that
        end each sequence, whose keys and values go to `slots` [batch, n] of the cache."""
        cfg = self.cfg
        batch, n = tokens.shape
        x = q.embedding(self.table, tokens.reshape(-1))
        split = [cfg.heads * cfg.head_dim, cfg.kv_heads * cfg.head_dim, cfg.kv_heads * cfg.head_dim]
        for layer in self.layers:
            qkv = q.qmm_t(self.norm(x), layer["qkv"])
            query, key, value = qkv.split(split, dim=-1)
            q.kv_append(layer["cache"], key.unflatten(-1, (cfg.kv_heads, cfg.head_dim)),
                        value.unflatten(-1, (cfg.kv_heads, cfg.head_dim)), slots.reshape(-1))
            mixed = q.kv_attend(query.unflatten(-1, (cfg.heads, cfg.head_dim)).unflatten(0, (batch, n)),
                                layer["cache"], table, lengths, max_length=longest)
            x = x + q.qmm_t(mixed.reshape(batch * n, -1), layer["out"])
            x = x + self.moe(self.norm(x), layer)
        last = self.norm(x.unflatten(0, (batch, n))[:, -1].contiguous())
        return q.qmm_t(last, self.head)

    def generate(self, prompt, steps, u, **sampling):
        """Continue prompt int32 [batch, n] by `steps` tokens; u [steps, batch] are the uniform
        numbers of the draws.  Returns int32 [batch, steps]."""
        cfg = self.cfg
        batch, n = prompt.shape
        blocks = -(-(n + steps) // cfg.page)
        table = torch.tensor([[self.free.pop() for _ in range(blocks)] for _ in range(batch)], dtype=torch.int32)
        slot = (table[:, :, None] * cfg.page + torch.arange(cfg.page, dtype=torch.int32)).flatten(1).to(self.device)
        pages = table.flatten().tolist()
        table = table.to(self.device)
        lengths = torch.full((batch,), n, dtype=torch.int32, device=self.device)
        tokens, first, out = prompt, 0, []
        for step in range(steps):
            longest = n + step
            logits = self.logits(tokens, slot[:, first:longest].contiguous(), table, lengths, longest)
            index, _ = q.sample(logits, u[step].contiguous(), **sampling)
            out.append(index)
            tokens, first = index[:, None], longest
            lengths = lengths + 1
        self.free += pages
        return torch.stack(out, 1)


if __name__ == "__main__":
    gen = torch.Generator(device="cuda").manual_seed(1)
    model = Decoder(Config())
    prompt = torch.randint(0, model.cfg.vocab, (4, 37), generator=gen, device="cuda", dtype=torch.int32)
    u = torch.rand(16, 4, generator=gen, device="cuda")
    for row in model.generate(prompt, 16, u, temperature=0.8, top_k=50, top_p=0.95, min_p=0.02).tolist():
        print(" ".join("%d" % t for t in row))
