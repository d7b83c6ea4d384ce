"""examples/decode_step.py: the operators together, against the same model computed without the paged
cache, the packed weights or the library's attention, experts and sampler (weights dequantized by the
library, products in fp32 on activations rounded where the model rounds them)."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import gptq_bit_weight_gemm_gb300 as g  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    from gptq_bit_weight_gemm_gb300 import build as lib_build
    lib_build.build()
    import decode_step
    return decode_step


# activations of order 1 through 2 layers of bf16: 2^-8 a rounding, some 12 on the way
OFF = 12 * 2.0 ** -8


def plain_step(ex, model, history, tokens, chosen):
    """Logits by full attention over the kept keys and values `history` (per layer lists).  The experts are
    those the library chose (`chosen`, per layer): where two logits are closer than both can be off,
    either is right, and each has to be within that of the best ones."""
    c = model.cfg
    W = lambda w, K: g.dequant(*w, K=K, bits=c.bits, group=c.group, fmt=g.V2, dtype=torch.float16).float()  # noqa: E731
    r = lambda t: t.to(c.dtype).float()  # noqa: E731
    n = len(history[0][0]) + 1
    pos = torch.full((model.batch,), n - 1, device="cuda")
    x = model.embedding[tokens.long()].float()
    for i, layer in enumerate(model.layers):
        qkv = r(r(ex.norm(x)) @ W(layer["qkv"], c.hidden)).view(model.batch, -1, c.dim)
        q, k, v = qkv.split([c.heads, c.kv_heads, c.kv_heads], 1)
        history[i][0].append(r(ex.rotate(k, pos)))
        history[i][1].append(v)
        K, V = (torch.stack(h, 2).repeat_interleave(c.heads // c.kv_heads, 1) for h in history[i])
        s = torch.einsum("bhd,bhnd->bhn", r(ex.rotate(q, pos)), K) * c.dim ** -0.5
        a = r(torch.einsum("bhn,bhnd->bhd", torch.softmax(s, -1), V))
        x = x + r(a.reshape(model.batch, -1) @ W(layer["out"], c.heads * c.dim))
        xn = r(ex.norm(x))
        p = torch.softmax(xn @ layer["router"].float().T, -1)
        ids = chosen[i].long()
        best = torch.sort(p, dim=-1, descending=True)[0][:, c.topk - 1:c.topk]
        w = p.gather(1, ids)
        assert bool((torch.log(w / best) > -2 * OFF).all())
        w = w / w.sum(-1, keepdim=True)
        y = torch.zeros_like(x)
        for e in range(c.experts):
            h = xn @ W([t[e] for t in layer["up"]], c.hidden)
            h = torch.nn.functional.silu(h[:, :c.inter]) * h[:, c.inter:]
            y = y + ((ids == e) * w).sum(-1, keepdim=True) * (h @ W([t[e] for t in layer["down"]], c.inter))
        x = x + r(y)
    return r(r(ex.norm(x)) @ W(model.head, c.hidden))


@pytest.mark.parametrize("batch", [1, 5])
def test_steps_match_the_plain_model(example, batch, monkeypatch):
    model = example.Model(example.Config(), batch, seed=3)
    history = [([], []) for _ in model.layers]
    tokens = torch.arange(batch, dtype=torch.int32, device="cuda") * 7 % 1024
    chosen, layer = [], g.moe_layer

    def noting(*a, **kw):
        out, ids, _ = layer(*a, return_routing=True, **kw)
        chosen.append(ids)
        return out

    monkeypatch.setattr(g, "moe_layer", noting)
    for step in range(20):
        chosen.clear()
        logits = model.step(tokens)
        ref = plain_step(example, model, history, tokens, chosen)
        err = (logits.float() - ref).norm(dim=-1) / ref.norm(dim=-1)
        assert bool((err < OFF).all()), (step, err)
        tokens = ref.argmax(-1).to(torch.int32)
    assert g.device_status() == 0


def test_generate_is_repeatable_and_in_range(example):
    out = []
    for _ in range(2):
        model = example.Model(example.Config(), 4)
        out.append(example.generate(model, torch.arange(4, dtype=torch.int32, device="cuda"), 24))
    assert torch.equal(out[0], out[1]) and out[0].shape == (4, 24)
    assert int(out[0].min()) >= 0 and int(out[0].max()) < 1024
    assert len(set(out[0].flatten().tolist())) > 4
    assert g.device_status() == 0


def test_a_full_cache_is_refused(example):
    model = example.Model(example.Config(max_len=3, page=2), 2)
    t = torch.zeros(2, dtype=torch.int32, device="cuda")
    for _ in range(3):
        model.step(t)
    with pytest.raises(ValueError):
        model.step(t)
