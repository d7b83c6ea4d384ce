"""Prompts and decode steps of a small quantised mixture-of-experts model, every layer through the library.

    python examples/decode_step.py [--layers 2] [--batch 4] [--steps 16] [--prompt 1]

Each layer is  x += Wo attention(norm(x));  x += moe(norm(x)):  the projections are GPTQ GEMMs
(``gemm``), the norms take the residual's addition (``rms_norm``), queries and keys are turned by
``rotary``, the experts are packed weights behind a router (``moe_layer``), and the logits' GEMM ends in
``sample``.  Keys and values lie in a paged cache whose pages ``page_plan`` hands out and takes back.  A step
of one token a sequence attends through ``paged_attention``, which appends as well; a chunk of a prompt is
appended by ``rotary`` and attends through ``chunk_attention``.  The weights are random, quantised by
``quantize_rtn``; PyTorch supplies memory and the embedding lookup.
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
    """What ``rms_norm`` computes, in plain operations (for checks)."""
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)


def rotate(x, pos):
    """What ``rotary`` computes of [batch, heads, dim] at pos [batch], in plain operations (for checks)."""
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
        # a cache of pages per layer; the plan enters the pages of sequence b into row b of the table
        width = -(-cfg.max_len // cfg.page)
        pages = batch * width
        self.free = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        self.free_count = torch.full((1,), pages, dtype=torch.int32, device="cuda")
        self.table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
        shape = (cfg.layers, 2, pages, cfg.page, cfg.kv_heads, cfg.dim)
        self.cache = torch.zeros(shape, dtype=cfg.dtype, device="cuda")
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.turns, _ = g.rotary_table(cfg.dim)
        # workspaces live as long as the model
        self.attention_ws = g.paged_attention_workspace(cfg.heads, cfg.kv_heads, cfg.dim)
        self.chunk_ws = g.chunk_attention_workspace(cfg.heads, cfg.kv_heads, cfg.dim)
        self.moe_ws = g.moe_workspace(32, cfg.hidden, cfg.inter, cfg.experts, cfg.topk)

    def gemm(self, x, weight):
        return g.gemm(x, *weight, bits=self.cfg.bits, group=self.cfg.group, fmt=g.V2)

    def moe(self, x, layer):
        """The experts' layer takes 32 tokens a call."""
        c = self.cfg
        return torch.cat([g.moe_layer(part, layer["router"], layer["up"], layer["down"], topk=c.topk, bits=c.bits, group=c.group,
                                      fmt=g.V2, workspace=self.moe_ws) for part in x.split(32)])

    def plan(self, added, tokens):
        """Pages for added[b] (int32, negative: the last ones are dropped) more tokens of each sequence, `tokens` rows in all."""
        c = self.cfg
        if int((self.lens + added).max()) > c.max_len:
            raise ValueError("the cache is full: %d tokens" % c.max_len)
        return g.page_plan(self.lens, added, self.table, self.free, self.free_count, page_size=c.page, max_tokens=tokens,
                           seq_lens=self.lens)

    def layers_of(self, tokens, positions, attend):
        """The normed output of all layers for rows of tokens; attend(layer's number, q, k, v) -> the attention's rows."""
        c = self.cfg
        x = self.embedding[tokens.long()].float()          # the residual, in 32 bits
        h = g.rms_norm(x, dtype=c.dtype)
        for i, layer in enumerate(self.layers):
            qkv = self.gemm(h, layer["qkv"]).view(len(tokens), c.heads + 2 * c.kv_heads, c.dim)
            q, k, v = qkv.split([c.heads, c.kv_heads, c.kv_heads], 1)
            a = attend(i, q, k, v)
            h = g.rms_norm(self.gemm(a.view(len(tokens), -1), layer["out"]), residual=x)
            h = g.rms_norm(self.moe(h, layer), residual=x)
        return h

    def step(self, tokens):
        """Logits [batch, vocab] after one more token of each sequence."""
        _, _, positions, _ = self.plan(torch.ones_like(self.lens), self.batch)

        def attend(i, q, k, v):
            q, k = g.rotary(q, k, positions, self.turns)
            return g.paged_attention(q, self.cache[i, 0], self.cache[i, 1], self.table, self.lens, k_new=k, v_new=v,
                                     workspace=self.attention_ws)
        return self.gemm(self.layers_of(tokens, positions, attend), self.head)

    def extend(self, tokens, added):
        """Logits [batch, vocab] after added[b] more tokens of each sequence: `tokens` holds them, sequence after
        sequence.  A sequence that brings none has the logits of no token: its row is not to be used."""
        lens, cu, positions, slots = self.plan(added, len(tokens))

        def attend(i, q, k, v):
            k_cache, v_cache = self.cache[i]
            q, _ = g.rotary(q, k, positions, self.turns, v=v, k_cache=k_cache, v_cache=v_cache, slots=slots)
            return g.chunk_attention(q, k_cache, v_cache, self.table, lens, cu, workspace=self.chunk_ws)
        h = self.layers_of(tokens, positions, attend)
        return self.gemm(h[(cu[1:].long() - 1).clamp(min=0)], self.head)

    def prompt(self, prompts, chunk=64):
        """Logits [batch, vocab] after the prompts (a list of token tensors, one for each sequence, of any lengths from one),
        `chunk` tokens of each at a time."""
        logits = None
        for at in range(0, max(len(p) for p in prompts), chunk):
            parts = [p[at:at + chunk] for p in prompts]
            added = torch.tensor([len(p) for p in parts], dtype=torch.int32, device="cuda")
            new = self.extend(torch.cat(parts), added)
            logits = new if logits is None else torch.where(added[:, None] > 0, new, logits)
        return logits

    def end(self, which):
        """Ends the sequences of a truth value each: their pages go back to the list."""
        self.plan(torch.where(which, -self.lens, 0), 0)


def generate(model, prompt, steps, *, temperature=0.8, top_k=50, top_p=0.95, min_p=0.02, seed=0):
    """`steps` tokens for each sequence after its prompt: [batch, steps] int32.  prompt: a token each [batch], or a
    list of token tensors of any lengths."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    full = lambda v, dt=torch.float32: torch.full((model.batch,), v, dtype=dt, device="cuda")  # noqa: E731
    settings = dict(temperature=full(temperature), top_k=full(top_k, torch.int32), top_p=full(top_p), min_p=full(min_p))
    tokens, out = prompt, []
    for i in range(steps):
        logits = model.prompt(prompt) if i == 0 and isinstance(prompt, list) else model.step(tokens)
        tokens, _ = g.sample(logits, torch.rand(model.batch, device="cuda", generator=gen), **settings)
        out.append(tokens)
    return torch.stack(out, 1)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=1, help="tokens of the first prompt; each further one has some fewer")
    a = ap.parse_args()
    model = Model(Config(layers=a.layers), a.batch)
    prompt = torch.arange(a.batch, dtype=torch.int32, device="cuda")
    if a.prompt > 1:
        prompt = [(b + 7 * torch.arange(max(1, a.prompt - 5 * b), dtype=torch.int32, device="cuda")) % model.cfg.vocab
                  for b in range(a.batch)]
    tokens = generate(model, prompt, a.steps)
    for row in tokens.tolist():
        print(" ".join("%4d" % t for t in row))
    status = g.device_status()
    if status:
        raise SystemExit("device status 0x%x" % status)


if __name__ == "__main__":
    main()
