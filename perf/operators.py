"""The operators of a quantised model's decode step, as measured cases.

Three operators stand next to the GPTQ GEMMs when a model answers token by token: attention of the
new token over a paged key-value cache (with the append of its key and value), the whole
mixture-of-experts layer for a few tokens on packed expert weights, and the choice of the next token
from the logits.  Each has a plain form here, in elementary torch operations and 32 bits, and the
call a user makes of the library (``own`` true).  ``exact`` computes the same from the definition
in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"


def _lib():
    import gptq_bit_weight_gemm_gb300 as g
    return g


def _generator(seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return gen


# ---------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one user, a short conversation: every microsecond is the user's waiting time
        dict(name="attn_one_short", op="attention", batch=1, heads=32, kv_heads=8, dim=128, page=16, min_len=997,
             max_len=997, window=0, dtype="bf16", layout="nhd", append=True, empty=False),
        # an ordinary serving batch with the 32 heads of a 4096-wide model without grouped heads
        dict(name="attn_batch_mha", op="attention", batch=16, heads=32, kv_heads=32, dim=128, page=16, min_len=40,
             max_len=2048, window=0, dtype="f16", layout="nhd", append=True, empty=False),
        # one long document: the only parallelism is the length of the cache
        dict(name="attn_one_long", op="attention", batch=1, heads=32, kv_heads=8, dim=128, page=64, min_len=131072,
             max_len=131072, window=0, dtype="bf16", layout="hnd", append=False, empty=False),
        # a full server: many sequences of very different lengths
        dict(name="attn_batch_large", op="attention", batch=64, heads=32, kv_heads=8, dim=128, page=32, min_len=512,
             max_len=8192, window=0, dtype="bf16", layout="nhd", append=False, empty=False),
        # odd everything: three query heads a key head, 80 wide, pages of 13, a sliding window, an empty sequence
        dict(name="attn_window_odd", op="attention", batch=24, heads=15, kv_heads=5, dim=80, page=13, min_len=1,
             max_len=5003, window=1000, dtype="f16", layout="nhd", append=False, empty=True),
        # the framework's own expert shape (8 experts, 4096 x 14336, 4-bit g128), one token
        dict(name="moe_wide_1", op="moe", tokens=1, experts=8, topk=2, hidden=4096, inter=14336, bits=4, group=128,
             fmt=2, dtype="f16", renormalize=True),
        # the same for a batch of eight: most experts hold a token or two
        dict(name="moe_wide_8", op="moe", tokens=8, experts=8, topk=2, hidden=4096, inter=14336, bits=4, group=128,
             fmt=2, dtype="f16", renormalize=True),
        # many small experts, several of them for each token
        dict(name="moe_fine_16", op="moe", tokens=16, experts=64, topk=6, hidden=2048, inter=1408, bits=4, group=128,
             fmt=1, dtype="bf16", renormalize=False),
        # odd widths, 8-bit codes in groups of 32
        dict(name="moe_odd_5", op="moe", tokens=5, experts=6, topk=3, hidden=1056, inter=672, bits=8, group=32,
             fmt=2, dtype="bf16", renormalize=True),
        # one user, fp32 logits of a 32000-word vocabulary
        dict(name="sample_one", op="sample", batch=1, vocab=32000, dtype="f32", kind="mixed"),
        # a serving batch, every request with its own settings
        dict(name="sample_batch", op="sample", batch=64, vocab=131072, dtype="bf16", kind="mixed"),
        # a large batch with an odd vocabulary, whose rows start at any two bytes
        dict(name="sample_odd_large", op="sample", batch=256, vocab=50257, dtype="f16", kind="mixed"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "moe", "moe", "sample"])
    if op == "attention":
        kv, per, dim = rng.choice([(8, 4, 128), (32, 1, 128), (8, 5, 128), (4, 8, 128), (1, 16, 128), (2, 7, 64),
                                   (12, 1, 64), (5, 3, 80), (8, 1, 96), (4, 4, 256), (2, 24, 128)])
        batch = _log_int(rng, 1, 64)
        # no more keys in all than the largest listed case has
        most = max(16, min(131072, int(1.0e9 / (batch * kv * dim * 4))))
        max_len = _log_int(rng, 16, most)
        return dict(op="attention", batch=batch, heads=kv * per, kv_heads=kv, dim=dim,
                    page=rng.choice([8, 13, 16, 16, 32, 64, 128, 256]), min_len=_log_int(rng, 1, max_len),
                    max_len=max_len, window=rng.choice([0, 0, 0, _log_int(rng, 8, 4096)]),
                    dtype=rng.choice(["f16", "bf16"]), layout=rng.choice(["nhd", "hnd"]),
                    append=rng.choice([False, False, True]), empty=rng.choice([False, True]))
    if op == "moe":
        bits = rng.choice([4, 4, 4, 8, 2, 3])
        group = {4: [128, 64, 32, -1], 8: [128, 64, 32, -1], 2: [128, 64], 3: [128]}[bits]
        step = {4: 32, 8: 32, 2: 128, 3: 128}[bits]
        group = rng.choice(group)
        step = max(step, group)
        experts = _log_int(rng, 4, 128)
        hidden = step * max(1, _log_int(rng, 512, 4096) // step)
        most = max(256, min(8192, int(1.0e9 / (experts * hidden * 3))))
        inter = step * max(1, _log_int(rng, 256, most) // step)
        return dict(op="moe", tokens=_log_int(rng, 1, 32), experts=experts, topk=rng.randint(1, min(8, experts)),
                    hidden=hidden, inter=inter, bits=bits, group=group, fmt=rng.choice([1, 2]),
                    dtype=rng.choice(["f16", "bf16"]), renormalize=rng.choice([True, False]))
    return dict(op="sample", batch=_log_int(rng, 1, 128), vocab=_log_int(rng, 1000, 256000),
                dtype=rng.choice(["f16", "bf16", "f32"]), kind=rng.choice(["mixed", "mixed", "top_p", "top_k", "plain"]))


def _lengths(c):
    """Keys of each sequence, spread over [min_len, max_len] evenly in their logarithm."""
    lens = [max(1, min(c["max_len"], int(round(math.exp(
        math.log(c["min_len"]) + (math.log(c["max_len"]) - math.log(c["min_len"])) * ((0.618034 * (i + 1)) % 1.0))))))
        for i in range(c["batch"])]
    lens[0] = c["max_len"]
    if c["empty"] and not c["append"] and c["batch"] > 1:
        lens[c["batch"] // 2] = 0
    return lens


def _live(c):
    """Keys that each sequence's new token attends to."""
    return [min(n, c["window"]) if c["window"] else n for n in _lengths(c)]


def work(c):
    if c["op"] == "attention":
        keys = sum(_live(c))
        io = 2 * c["batch"] * c["heads"] * c["dim"] * 2
        new = 2 * 2 * c["batch"] * c["kv_heads"] * c["dim"] * 2 if c["append"] else 0
        table = 4 * sum(-(-n // c["page"]) for n in _live(c)) + 4 * c["batch"]
        return {"bytes": keys * c["kv_heads"] * c["dim"] * 4 + io + new + table, "flops": 4 * keys * c["heads"] * c["dim"]}
    if c["op"] == "moe":
        T, E, k, H, I = c["tokens"], c["experts"], c["topk"], c["hidden"], c["inter"]
        active = E * (1.0 - (1.0 - k / E) ** T)   # experts that some token picks, on average over the inputs

        def packed(K, N):
            G = 1 if c["group"] == -1 else K // c["group"]
            return K * N * c["bits"] / 8 + G * N * 2 + G * N * c["bits"] / 8

        each = packed(H, 2 * I) + packed(I, H)
        return {"bytes": active * each + E * H * 2 + 2 * T * H * 2 + T * k * 8,
                "flops": 2 * T * E * H + 2 * T * k * 3 * H * I}
    size = torch.empty(0, dtype=DTYPES[c["dtype"]]).element_size()
    return {"bytes": c["batch"] * c["vocab"] * size + 28 * c["batch"], "flops": 3 * c["batch"] * c["vocab"]}


# ---------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = _generator(seed)
    return {"attention": _prepare_attention, "moe": _prepare_moe, "sample": _prepare_sample}[case["op"]](dict(case), gen)


def _prepare_attention(c, gen):
    dt, B, page = DTYPES[c["dtype"]], c["batch"], c["page"]
    lens = _lengths(c)
    width = max(1, -(-max(lens) // page))
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    # sequence b owns the next need[b] pages of the shuffled order; the rest of its row is not set (-1)
    need_t = torch.tensor(need, device=DEV)
    first = torch.cumsum(need_t, 0) - need_t
    j = torch.arange(width, device=DEV)
    table = torch.where(j[None] < need_t[:, None], order[(first[:, None] + j[None]).clamp(max=pages - 1)], -1).to(torch.int32)
    shape = (pages, page, c["kv_heads"], c["dim"]) if c["layout"] == "nhd" else (pages, c["kv_heads"], page, c["dim"])
    caches = []
    for _ in range(2):
        t = torch.empty(shape, dtype=dt, device=DEV).normal_(generator=gen)
        t = t if c["layout"] == "nhd" else t.permute(0, 2, 1, 3)
        # what no sequence has written holds anything at all
        used = torch.zeros((pages, page), dtype=torch.bool, device=DEV)
        pos = j[None, :, None] * page + torch.arange(page, device=DEV)
        live = pos < torch.tensor(lens, device=DEV)[:, None, None]
        used[table.clamp(min=0).long()[live.any(-1)]] = live[live.any(-1)]
        t[~used] = float("nan")
        caches.append(t)
    rnd = lambda h: torch.empty((B, h, c["dim"]), dtype=dt, device=DEV).normal_(generator=gen)  # noqa: E731
    s = dict(c, table=table, lens=torch.tensor(lens, dtype=torch.int32, device=DEV), k=caches[0], v=caches[1], q=rnd(c["heads"]),
             width=width, scale=c["dim"] ** -0.5)
    s["k_new"], s["v_new"] = (rnd(c["kv_heads"]), rnd(c["kv_heads"])) if c["append"] else (None, None)
    if own:   # a program keeps the workspace of its attention calls
        s["workspace"] = _lib().paged_attention_workspace(c["heads"], c["kv_heads"], c["dim"])
    return s


def _prepare_moe(c, gen):
    dt, E, H, I, bits = DTYPES[c["dtype"]], c["experts"], c["hidden"], c["inter"], c["bits"]

    def words(*shape):
        return torch.randint(-2 ** 31, 2 ** 31, shape, dtype=torch.int64, device=DEV, generator=gen).to(torch.int32)

    def weight(K, N):
        G = 1 if c["group"] == -1 else K // c["group"]
        scales = 0.12 / 2 ** bits * (0.5 + torch.rand((E, G, N), device=DEV, generator=gen))
        return words(E, K * bits // 32, N), words(E, G, N * bits // 32), scales.to(torch.float16)

    s = dict(c, up=weight(H, 2 * I), down=weight(I, H), x=torch.empty((c["tokens"], H), dtype=dt, device=DEV).normal_(generator=gen))
    s["router"] = (torch.randn((E, H), device=DEV, generator=gen) * H ** -0.5 * 2).to(dt)
    if own:
        s["workspace"] = _lib().moe_workspace(c["tokens"], H, I, E, c["topk"])
    return s


def _prepare_sample(c, gen):
    B, V = c["batch"], c["vocab"]
    # a broad body, and a few words that stand out by an exponential margin
    logits = 2.0 * torch.randn((B, V), device=DEV, generator=gen)
    few = torch.randint(0, V, (B, 24), device=DEV, generator=gen)
    logits.scatter_add_(1, few, torch.empty((B, 24), device=DEV).exponential_(generator=gen) * 4.0)
    rnd = lambda lo, hi: torch.empty(B, device=DEV).uniform_(lo, hi, generator=gen)  # noqa: E731
    i = torch.arange(B, device=DEV)
    temperature, top_k, top_p, min_p = rnd(0.4, 1.4), torch.zeros(B, dtype=torch.int32, device=DEV), rnd(1.0, 1.0), rnd(0.0, 0.0)
    if c["kind"] in ("mixed", "top_k"):
        k = torch.randint(1, 200, (B,), device=DEV, generator=gen).to(torch.int32)
        top_k = torch.where((i % 3 != 1) | (c["kind"] == "top_k"), k, 0).to(torch.int32)
    if c["kind"] in ("mixed", "top_p"):
        top_p = torch.where((i % 4 != 2) | (c["kind"] == "top_p"), rnd(0.5, 0.99), 1.0)
    if c["kind"] == "mixed":
        min_p = torch.where(i % 2 == 1, rnd(0.0, 0.1), 0.0)
        temperature = torch.where(i % 8 == 5, 0.0, temperature)   # the greedy requests of the batch
    return dict(c, logits=logits.to(DTYPES[c["dtype"]]), uniform=torch.rand(B, device=DEV, generator=gen), temperature=temperature,
                top_k=top_k, top_p=top_p, min_p=min_p)


# ---------------------------------------------------------------------------------- one pass
def run(s):
    return {"attention": _attention, "moe": _moe, "sample": _sample}[s["op"]](s)


def _attention(s):
    if own:
        out = _lib().paged_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], scale=s["scale"], window=s["window"],
                                     k_new=s["k_new"], v_new=s["v_new"], workspace=s["workspace"])
        return [out, s["k"], s["v"]] if s["append"] else [out]
    B, page, D, kv = s["batch"], s["page"], s["dim"], s["kv_heads"]
    lens, table = s["lens"].long(), s["table"].clamp(min=0).long()
    if s["append"]:
        at = lens - 1
        where = table.gather(1, (at // page)[:, None])[:, 0], at % page
        s["k"][where], s["v"][where] = s["k_new"], s["v_new"]
    L = s["width"] * page
    pos = torch.arange(L, device=DEV)
    live = pos[None] < lens[:, None]
    if s["window"]:
        live &= pos[None] >= lens[:, None] - s["window"]
    k = s["k"][table].reshape(B, L, kv, D).permute(0, 2, 3, 1).float()
    q = s["q"].float().reshape(B, kv, -1, D)
    scores = (q @ k * s["scale"]).masked_fill(~live[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == float("-inf"), 0.0, top))
    total = p.sum(-1, keepdim=True)
    v = s["v"][table].reshape(B, L, kv, D).permute(0, 2, 1, 3).float().masked_fill(~live[:, None, :, None], 0.0)
    out = (p @ v) / torch.where(total == 0, 1.0, total)
    out = out.reshape(B, s["heads"], D).to(s["q"].dtype)
    return [out, s["k"], s["v"]] if s["append"] else [out]


def _codes(words, bits, count):
    """The codes 0 .. count-1 of little-endian bit streams along dim 1 of int32 words [R, W, N] -> [R, count, N]."""
    mask = (1 << bits) - 1
    if 32 % bits == 0:
        shift = torch.arange(0, 32, bits, device=DEV, dtype=torch.int32)
        return ((words[:, :, None] >> shift[:, None]) & mask).reshape(words.shape[0], count, words.shape[2])
    bit = torch.arange(count, device=DEV) * bits
    w, sh = bit // 32, (bit % 32)[:, None]
    lo = words[:, w].long() & 0xFFFFFFFF
    hi = words[:, (w + 1).clamp(max=words.shape[1] - 1)].long() & 0xFFFFFFFF
    return (((lo | (hi << 32)) >> sh) & mask).to(torch.int32)


def _dequant(weight, pick, K, bits, fmt):
    """fp32 weights [R, K, N] of the picked experts (all of them: None)."""
    qw, qz, sc = weight if pick is None else tuple(t[pick] for t in weight)
    R, G, N = sc.shape
    z = _codes(qz.transpose(1, 2), bits, N).transpose(1, 2) + (1 if fmt == 1 else 0)
    w = _codes(qw, bits, K).reshape(R, G, K // G, N) - z[:, :, None]
    return (w * sc.float()[:, :, None]).reshape(R, K, N)


def _moe(s):
    if own:
        return list(_lib().moe_layer(s["x"], s["router"], s["up"], s["down"], topk=s["topk"], bits=s["bits"], group=s["group"],
                                     fmt=s["fmt"], renormalize=s["renormalize"], workspace=s["workspace"], return_routing=True))
    T, E, H, I, k = s["tokens"], s["experts"], s["hidden"], s["inter"], s["topk"]
    x = s["x"].float()
    logits = x @ s["router"].float().T
    p = torch.exp(logits - logits.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    weights, ids = torch.sort(p, dim=-1, descending=True, stable=True)
    weights, ids = weights[:, :k], ids[:, :k]
    if s["renormalize"]:
        weights = weights / weights.sum(-1, keepdim=True)
    if T * k < E:      # fewer choices than experts: only the chosen ones are unpacked
        pick, rows = ids.reshape(-1), x.repeat_interleave(k, 0)[:, None]
    else:              # all experts for all tokens, and the choice made by the weights
        pick, rows = None, x[None]
    gate, up = (rows @ _dequant(s["up"], pick, H, s["bits"], s["fmt"])).chunk(2, dim=-1)
    y = (gate / (1 + torch.exp(-gate)) * up) @ _dequant(s["down"], pick, I, s["bits"], s["fmt"])
    if pick is None:
        dense = torch.zeros((T, E), device=DEV).scatter_(1, ids, weights)
        out = (y * dense.T[:, :, None]).sum(0)
    else:
        out = (y.reshape(T, k, H) * weights[:, :, None]).sum(1)
    return [out.to(s["x"].dtype), ids.to(torch.int32), weights.contiguous()]


def _sample(s):
    if own:
        return list(_lib().sample(s["logits"], s["uniform"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                                  min_p=s["min_p"]))
    B, V = s["logits"].shape
    greedy = s["temperature"] == 0
    logits = s["logits"].float()
    x = (logits - logits.amax(-1, keepdim=True)) / torch.where(greedy, 1.0, s["temperature"])[:, None]
    x, order = torch.sort(x, dim=-1, descending=True, stable=True)   # ties: the lowest index first
    w = torch.exp(x)
    top_k = torch.where(greedy, 1, torch.where(s["top_k"] > 0, s["top_k"], V))
    keep = torch.arange(V, device=DEV)[None] < top_k[:, None]
    # the sums run over up to 256000 terms and decide between neighbours: taken in 64 bits
    before = torch.cumsum(torch.where(keep, w, 0.0), -1, dtype=torch.float64)
    total = before[:, -1:]
    before = before - w
    keep &= (before < s["top_p"].double()[:, None] * total) & (w >= s["min_p"][:, None])
    keep[:, 0] = True
    w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0.0))
    run_sum = torch.cumsum(w, -1, dtype=torch.float64)
    total = run_sum[:, -1]
    token = (run_sum <= (s["uniform"].double() * total)[:, None]).sum(-1)
    logprob = torch.log(w.gather(1, token[:, None])[:, 0].double() / total)
    return [token.to(torch.int32), logprob.float()]


# ---------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _exact_attention, "moe": _exact_moe, "sample": _exact_sample}[case["op"]](s)


def _exact_attention(s):
    B, kv, D, page = s["batch"], s["kv_heads"], s["dim"], s["page"]
    out = torch.zeros((B, s["heads"], D), dtype=torch.float64, device=DEV)
    for b, n in enumerate(_lengths(s)):
        lo = max(0, n - s["window"]) if s["window"] else 0
        if n == 0:
            continue
        row = s["table"][b, lo // page:-(-n // page)].long()
        keys, values = (t[row].reshape(-1, kv, D)[lo - lo // page * page:][:n - lo].double() for t in (s["k"], s["v"]))
        if s["append"]:
            keys[-1], values[-1] = s["k_new"][b].double(), s["v_new"][b].double()
        q = s["q"][b].double().reshape(kv, -1, D)
        p = torch.softmax(torch.einsum("hgd,nhd->hgn", q, keys) * s["scale"], -1)
        out[b] = torch.einsum("hgn,nhd->hgd", p, values).reshape(-1, D)
    return [out, None, None] if s["append"] else [out]


def _exact_weight(weight, e, K, s):
    qw, qz, sc = (t[e] for t in weight)
    bits, (G, N) = s["bits"], sc.shape
    at = lambda n: (torch.arange(n, device=DEV) * bits)  # noqa: E731

    def field(stream, n):      # bit by bit
        code = torch.zeros((n, stream.shape[1]), dtype=torch.int64, device=DEV)
        for j in range(bits):
            b = at(n) + j
            code += ((stream.long()[b // 32] >> (b % 32)[:, None]) & 1) << j
        return code

    q = field(qw, K)
    z = field(qz.T.contiguous(), N).T + (2 - s["fmt"])
    g = torch.arange(K, device=DEV) // (K // G)
    return (q - z[g]).double() * sc.double()[g]


def _exact_moe(s):
    T, E, k = s["tokens"], s["experts"], s["topk"]
    x = s["x"].double()
    p = torch.softmax(x @ s["router"].double().T, -1).cpu()
    ids = [sorted(range(E), key=lambda e: (-float(row[e]), e))[:k] for row in p]
    weights = torch.stack([row[i] for row, i in zip(p, ids)])
    if s["renormalize"]:
        weights = weights / weights.sum(-1, keepdim=True)
    out = torch.zeros((T, s["hidden"]), dtype=torch.float64, device=DEV)
    for e in sorted({e for row in ids for e in row}):
        who = [(t, row.index(e)) for t, row in enumerate(ids) if e in row]
        rows = torch.tensor([t for t, _ in who], device=DEV)
        h = x[rows] @ _exact_weight(s["up"], e, s["hidden"], s)
        h = torch.nn.functional.silu(h[:, :s["inter"]]) * h[:, s["inter"]:]
        y = h @ _exact_weight(s["down"], e, s["inter"], s)
        out[rows] += y * torch.stack([weights[t, j] for t, j in who]).to(DEV)[:, None]
    return [out, torch.tensor(ids, dtype=torch.int32), weights]


def _exact_sample(s):
    tokens, logs = [], []
    greedy = s["temperature"] == 0
    settings = zip(s["logits"].double(), s["uniform"].tolist(), s["temperature"].tolist(), s["top_k"].tolist(), s["top_p"].tolist(),
                   s["min_p"].tolist())
    for row, u, t, k, top_p, min_p in settings:
        if t == 0:
            t, k = 1.0, 1
        w = torch.exp((row - row.max()) / t)
        sorted_w, order = torch.sort(w, descending=True, stable=True)
        n = k if k > 0 else len(w)
        cum = torch.cumsum(sorted_w[:n], 0)
        keep = (torch.cat([cum.new_zeros(1), cum[:-1]]) < top_p * cum[-1]) & (sorted_w[:n] >= min_p)
        keep[0] = True
        kept = torch.sort(order[:n][keep])[0]
        cum = torch.cumsum(w[kept], 0)
        i = int(torch.searchsorted(cum, u * cum[-1], right=True))
        tokens.append(int(kept[i]))
        logs.append(float(torch.log(w[kept[i]] / cum[-1])))
    return [torch.tensor(tokens, dtype=torch.int32), torch.tensor(logs, dtype=torch.float64)]
