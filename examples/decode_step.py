"""A decode step of a small quantised mixture-of-experts model, every layer through the library.

    python examples/decode_step.py [--layers 2] [--batch 4] [--steps 16]

Each layer is  x += Wo attention(norm(x));  x += moe(norm(x)):  the projections are GPTQ GEMMs
(``gemm``), the attention reads a paged cache that each step appends to (``paged_attention``), the
experts are packed weights behind a router (``moe_layer``), and the logits' GEMM ends in ``sample``.  The
weights are random, quantised by ``quantize_rtn``; PyTorch supplies memory, the embedding lookup, the
norms and the rotary embedding.
"""
import argparse
import dataclasses
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gptq_bit_weight_gemm_gb300 as g  # noqa: E402


@dataclasses.dataclass(frozen=True)
class Config:
    hidden: int = 512
    heads: int = 8
    kv_heads: int = 2
    dim: int = 64
    inter: int = 256
    experts: int = 8
    topk: int = 2
    vocab: int = 1024
    layers: int = 2
    bits: int = 4
    group: int = 64
    page: int = 16
    max_len: int = 256
    dtype: torch.dtype = torch.bfloat16


def quantised(cfg, K, N, gen, experts=0):
    """A random weight [K, N] (or one for each expert), quantised: (qweight, qzeros, scales)."""
    def one():
        W = torch.randn((K, N), device="cuda", generator=gen) * K ** -0.5
        return g.quantize_rtn(W, bits=cfg.bits, group=cfg.group, fmt=g.V2)
    if not experts:
        return one()
    return tuple(torch.stack(t) for t in zip(*(one() for _ in range(experts))))


def norm(x):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)


def rotate(x, pos):
    """Rotary embedding of [batch, heads, dim] at pos [batch]."""
    half = x.shape[-1] // 2
    angle = pos[:, None, None].float() * 10000.0 ** (-torch.arange(half, device=x.device) / half)
    a, b = x.float()[..., :half], x.float()[..., half:]
    return torch.cat([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], -1).to(x.dtype)


class Model:
    def __init__(self, cfg, batch, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.cfg, self.batch = cfg, batch
        self.embedding = torch.randn((cfg.vocab, cfg.hidden), device="cuda", generator=gen).to(cfg.dtype)
        self.layers = []
        for _ in range(cfg.layers):
            self.layers.append(dict(
                qkv=quantised(cfg, cfg.hidden, (cfg.heads + 2 * cfg.kv_heads) * cfg.dim, gen),
                out=quantised(cfg, cfg.heads * cfg.dim, cfg.hidden, gen),
                router=(torch.randn((cfg.experts, cfg.hidden), device="cuda", generator=gen) * cfg.hidden ** -0.5).to(cfg.dtype),
                up=quantised(cfg, cfg.hidden, 2 * cfg.inter, gen, cfg.experts),
                down=quantised(cfg, cfg.inter, cfg.hidden, gen, cfg.experts)))
        self.head = quantised(cfg, cfg.hidden, cfg.vocab, gen)
        # a cache of pages per layer; sequence b owns a row of shuffled pages
        width = -(-cfg.max_len // cfg.page)
        pages = batch * width
        self.table = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32).reshape(batch, width)
        shape = (cfg.layers, 2, pages, cfg.page, cfg.kv_heads, cfg.dim)
        self.cache = torch.zeros(shape, dtype=cfg.dtype, device="cuda")
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        # workspaces live as long as the model
        self.attention_ws = g.paged_attention_workspace(cfg.heads, cfg.kv_heads, cfg.dim)
        self.moe_ws = g.moe_workspace(batch, cfg.hidden, cfg.inter, cfg.experts, cfg.topk)

    def gemm(self, x, weight):
        return g.gemm(x, *weight, bits=self.cfg.bits, group=self.cfg.group, fmt=g.V2)

    def step(self, tokens):
        """Logits [batch, vocab] after one more token of each sequence."""
        c = self.cfg
        if int(self.lens.max()) >= c.max_len:
            raise ValueError("the cache is full: %d tokens" % c.max_len)
        self.lens += 1
        pos = self.lens - 1
        x = self.embedding[tokens.long()].float()
        for i, layer in enumerate(self.layers):
            qkv = self.gemm(norm(x).to(c.dtype), layer["qkv"]).view(self.batch, c.heads + 2 * c.kv_heads, c.dim)
            q, k, v = qkv.split([c.heads, c.kv_heads, c.kv_heads], 1)
            a = g.paged_attention(rotate(q, pos), self.cache[i, 0], self.cache[i, 1], self.table, self.lens,
                                  k_new=rotate(k, pos), v_new=v, workspace=self.attention_ws)
            x = x + self.gemm(a.view(self.batch, -1), layer["out"]).float()
            x = x + g.moe_layer(norm(x).to(c.dtype), layer["router"], layer["up"], layer["down"], topk=c.topk, bits=c.bits,
                                group=c.group, fmt=g.V2, workspace=self.moe_ws).float()
        return self.gemm(norm(x).to(c.dtype), self.head)


def generate(model, prompt, steps, *, temperature=0.8, top_k=50, top_p=0.95, min_p=0.02, seed=0):
    """`steps` tokens for each sequence after a prompt of one token each: [batch, steps] int32."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    full = lambda v, dt=torch.float32: torch.full((model.batch,), v, dtype=dt, device="cuda")  # noqa: E731
    settings = dict(temperature=full(temperature), top_k=full(top_k, torch.int32), top_p=full(top_p), min_p=full(min_p))
    tokens, out = prompt, []
    for _ in range(steps):
        logits = model.step(tokens)
        tokens, _ = g.sample(logits, torch.rand(model.batch, device="cuda", generator=gen), **settings)
        out.append(tokens)
    return torch.stack(out, 1)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args()
    model = Model(Config(layers=a.layers), a.batch)
    tokens = generate(model, torch.arange(a.batch, dtype=torch.int32, device="cuda"), a.steps)
    for row in tokens.tolist():
        print(" ".join("%4d" % t for t in row))
    status = g.device_status()
    if status:
        raise SystemExit("device status 0x%x" % status)


if __name__ == "__main__":
    main()
