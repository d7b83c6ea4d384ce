"""A prompt step's operators together, as examples/decode_step.py runs them: prompts in chunks, decode steps after
them, sequences that end and others in their place, against the same model computed without cache, packed
weights or the library's operators (weights dequantized by the library, products in fp32 on activations
rounded where the model rounds them); and their chain captured into a graph."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import gptq_bit_weight_gemm_gb300 as g  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"

# activations of order 1 through 2 layers of bf16: 2^-8 a rounding, some 12 on the way, and one more for the
# probabilities of each layer's attention
OFF = 14 * 2.0 ** -8


@pytest.fixture(scope="module")
def example():
    from gptq_bit_weight_gemm_gb300 import build as lib_build
    lib_build.build()
    import decode_step
    return decode_step


class Noting:
    """Notes the experts that the library chooses: rows of each layer in the order of its calls."""

    def __init__(self, model, monkeypatch):
        self.rows, self.model, layer = [[] for _ in model.layers], model, g.moe_layer
        routers = [x["router"].data_ptr() for x in model.layers]

        def noting(x, router, *a, **kw):
            out, ids, _ = layer(x, router, *a, return_routing=True, **kw)
            self.rows[routers.index(router.data_ptr())].extend(ids.long())
            return out
        monkeypatch.setattr(g, "moe_layer", noting)

    def take(self):
        rows, self.rows = self.rows, [[] for _ in self.rows]
        return rows


def plain(ex, model, tokens, chosen):
    """Logits after each of one sequence's tokens, the experts of each layer and token as the library chose them:
    where two logits are closer than both can be off either is right, and each has to be within that of the best."""
    c = model.cfg
    W = lambda w, K: g.dequant(*w, K=K, bits=c.bits, group=c.group, fmt=g.V2, dtype=torch.float16).float()  # noqa: E731
    r = lambda t: t.to(c.dtype).float()  # noqa: E731
    n = len(tokens)
    pos = torch.arange(n, device=DEV)
    x = model.embedding[tokens.long()].float()
    for i, layer in enumerate(model.layers):
        qkv = r(r(ex.norm(x)) @ W(layer["qkv"], c.hidden)).view(n, -1, c.dim)
        q, k, v = qkv.split([c.heads, c.kv_heads, c.kv_heads], 1)
        K, V = (t.repeat_interleave(c.heads // c.kv_heads, 1) for t in (r(ex.rotate(k, pos)), v))
        s = torch.einsum("thd,nhd->htn", r(ex.rotate(q, pos)), K) * c.dim ** -0.5
        s = s.masked_fill(pos[None] > pos[:, None], float("-inf"))
        a = r(torch.einsum("htn,nhd->thd", torch.softmax(s, -1), V))
        x = x + r(a.reshape(n, -1) @ W(layer["out"], c.heads * c.dim))
        xn = r(ex.norm(x))
        p = torch.softmax(xn @ layer["router"].float().T, -1)
        ids = torch.stack(chosen[i])
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


def run_prompts(model, prompts, chunk, note, chosen):
    """model.prompt in its chunks, the noted experts sorted by sequence."""
    logits = None
    for at in range(0, max(len(p) for p in prompts), chunk):
        parts = [p[at:at + chunk] for p in prompts]
        added = torch.tensor([len(p) for p in parts], dtype=torch.int32, device=DEV)
        new = model.extend(torch.cat(parts), added)
        logits = new if logits is None else torch.where(added[:, None] > 0, new, logits)
        for i, rows in enumerate(note.take()):
            for b, p in enumerate(parts):
                chosen[b][i].extend(rows[:len(p)])
                rows = rows[len(p):]
    return logits


def near(logits, ref):
    err = (logits.float() - ref).norm() / ref.norm()
    assert float(err) < OFF, float(err)


@pytest.mark.parametrize("chunk", [7, 64, 1000])
def test_prompts_in_chunks_then_steps(example, chunk, monkeypatch):
    model = example.Model(example.Config(), 4, seed=3)
    note = Noting(model, monkeypatch)
    gen = torch.Generator(device=DEV).manual_seed(chunk)
    prompts = [torch.randint(0, 1024, (n,), device=DEV, generator=gen, dtype=torch.int32) for n in (1, 130, 17, 64)]
    chosen = [[[] for _ in model.layers] for _ in prompts]
    logits = run_prompts(model, prompts, chunk, note, chosen)
    assert model.lens.tolist() == [len(p) for p in prompts]
    for b, p in enumerate(prompts):
        near(logits[b], plain(example, model, p, chosen[b])[-1])
    for step in range(3):       # and on, a token at a time, over the cache that the prompts left
        tokens = torch.randint(0, 1024, (4,), device=DEV, generator=gen, dtype=torch.int32)
        logits = model.step(tokens)
        for i, rows in enumerate(note.take()):
            for b in range(4):
                chosen[b][i].append(rows[b])
        prompts = [torch.cat([p, tokens[b:b + 1]]) for b, p in enumerate(prompts)]
    for b, p in enumerate(prompts):
        near(logits[b], plain(example, model, p, chosen[b])[-1])
    assert g.device_status() == 0


def test_ended_sequences_give_their_pages_to_others(example, monkeypatch):
    model = example.Model(example.Config(max_len=96, page=8), 3, seed=5)
    note = Noting(model, monkeypatch)
    gen = torch.Generator(device=DEV).manual_seed(9)
    draw = lambda n: torch.randint(0, 1024, (n,), device=DEV, generator=gen, dtype=torch.int32)  # noqa: E731
    pages = 3 * 12
    chosen = [[[] for _ in model.layers] for _ in range(3)]
    prompts = [draw(90), draw(33), draw(5)]
    run_prompts(model, prompts, 40, note, chosen)
    assert int(model.free_count) == pages - 12 - 5 - 1
    for turn in range(4):       # sequence `turn % 3` makes way for another, while the others wait
        b = turn % 3
        model.end(torch.arange(3, device=DEV) == b)
        note.take()
        chosen[b] = [[] for _ in model.layers]
        prompts[b] = draw(20 + 18 * turn)
        mine = [prompts[x] if x == b else prompts[x][:0] for x in range(3)]
        logits = run_prompts(model, mine, 50, note, chosen)
        near(logits[b], plain(example, model, prompts[b], chosen[b])[-1])
        used = torch.cat([model.table[x, :-(-len(prompts[x]) // 8)] for x in range(3)])
        rest = model.free[:int(model.free_count)]
        assert sorted(torch.cat([used, rest]).tolist()) == list(range(pages))
    logits = model.step(draw(3))
    assert bool(torch.isfinite(logits).all()) and g.device_status() == 0


def test_generate_from_prompts(example):
    out = []
    for _ in range(2):
        model = example.Model(example.Config(), 3)
        prompts = [torch.arange(n, dtype=torch.int32, device=DEV) for n in (70, 1, 12)]
        out.append(example.generate(model, prompts, 8))
    assert torch.equal(out[0], out[1]) and out[0].shape == (3, 8)
    model = example.Model(example.Config(max_len=64), 1)
    with pytest.raises(ValueError):
        model.prompt([torch.zeros(65, dtype=torch.int32, device=DEV)])
    assert g.device_status() == 0


def test_chain_captured_replayed_and_without_waits():
    # plan, norm, rotary with the append and attention in one graph, its lengths changing from replay to replay
    B, T, heads, kv, dim, page, width = 5, 64, 8, 2, 64, 16, 20
    gen = torch.Generator(device=DEV).manual_seed(4)
    turns, _ = g.rotary_table(dim)
    ws = g.chunk_attention_workspace(heads, kv, dim)

    def state():
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
        return dict(lens=i32([0] * B), added=i32([0] * B), table=i32([[-1] * width] * B), free=torch.arange(B * width, dtype=torch.int32, device=DEV),
                    count=i32([B * width]), cache=torch.full((2, B * width, page, kv, dim), float("nan"), dtype=torch.bfloat16, device=DEV),
                    x=torch.zeros((T, 512), dtype=torch.bfloat16, device=DEV), res=torch.zeros((T, 512), device=DEV),
                    qkv=torch.zeros((T, heads + 2 * kv, dim), dtype=torch.bfloat16, device=DEV),
                    out=torch.zeros((T, heads, dim), dtype=torch.bfloat16, device=DEV))

    def chain(s):
        lens, cu, pos, slots = g.page_plan(s["lens"], s["added"], s["table"], s["free"], s["count"], page_size=page, max_tokens=T, seq_lens=s["lens"])
        h = g.rms_norm(s["x"], residual=s["res"])
        q, k, v = s["qkv"].split([heads, kv, kv], 1)
        q, _ = g.rotary(q, k, pos, turns, v=v, k_cache=s["cache"][0], v_cache=s["cache"][1], slots=slots)
        g.chunk_attention(q, s["cache"][0], s["cache"][1], s["table"], lens, cu, out=s["out"], workspace=ws)
        return h

    eager, held = state(), state()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        chain(held)                                # nothing is added: nothing changes
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h_held = chain(held)
    for added in ([3, 20, 1, 0, 40], [1, 1, 1, 1, 1], [0, -15, 30, 5, -41], [60, 0, 0, 0, 4], [-64, -6, 9, 16, 16]):
        for s in (eager, held):
            gen.manual_seed(sum(added) + 7)
            s["added"].copy_(torch.tensor(added, dtype=torch.int32))
            s["x"].normal_(generator=gen), s["qkv"].normal_(generator=gen)
        h = chain(eager)
        graph.replay()
        torch.cuda.synchronize()
        rows = sum(max(0, a) for a in added)
        for name in ("lens", "table", "free", "count", "res"):
            assert torch.equal(eager[name], held[name]), name
        assert torch.equal(h, h_held) and torch.equal(eager["out"][:rows], held["out"][:rows])
        assert torch.equal(eager["cache"].view(torch.int16), held["cache"].view(torch.int16))
        assert bool(torch.isfinite(held["out"][:rows]).all())
    assert g.device_status() == 0
    # the same steps issued one after the other with nothing waited for between them
    steps = [[3, 20, 1, 0, 40], [1, 1, 1, 1, 1], [0, -15, 30, 5, -41], [60, 0, 0, 0, 4], [-64, -6, 9, 16, 16]] * 4
    alone = []
    for waits in (True, False):
        s = state()
        gen.manual_seed(99)
        s["x"].normal_(generator=gen), s["qkv"].normal_(generator=gen)
        ahead = torch.tensor(steps, dtype=torch.int32, device=DEV)
        torch.cuda.synchronize()
        outs = []
        for i in range(len(steps)):
            if i % 5 == 0 and i:
                s["added"].copy_(-s["lens"])           # everything ends, and the pages come back in another order
                chain(s)
            s["added"].copy_(ahead[i])
            chain(s)
            outs.append(s["out"].clone())
            if waits:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        alone.append((outs, s))
    for a, b, added in zip(alone[0][0], alone[1][0], steps):
        rows = sum(max(0, x) for x in added)
        assert torch.equal(a[:rows], b[:rows])
    for name in ("lens", "table", "free", "count", "res"):
        assert torch.equal(alone[0][1][name], alone[1][1][name]), name
    assert g.device_status() == 0
