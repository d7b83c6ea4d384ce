"""The operators of a step that takes chunks of prompts, as measured cases.

Between the GEMMs of such a step stand: the plan of the step's pages and slots, the norm with the
residual's addition, the rotary embedding with the append to the paged cache, and the attention of
each sequence's new tokens over its cached keys.  Each has a plain form here, in elementary torch
operations and 32 bits (64 for angles), and the call a user makes of the library (``own`` true).
``exact`` computes the same from the definition in 64 bits.
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
        # a follow-up of a few words in a short conversation: the user waits for the first token
        dict(name="chunk_one_short", op="chunk", batch=1, min_new=33, max_new=33, min_past=964, max_past=964, heads=32,
             kv_heads=8, dim=128, page=16, window=0, dtype="bf16", layout="nhd", empty=False),
        # a server's mixed step: most sequences bring a token, some of them a piece of their prompt
        dict(name="chunk_mixed", op="chunk", batch=16, min_new=1, max_new=1024, min_past=512, max_past=3072, heads=32,
             kv_heads=8, dim=128, page=32, window=0, dtype="bf16", layout="nhd", empty=False),
        # fresh prompts of a model without grouped heads, whole
        dict(name="chunk_prompts", op="chunk", batch=4, min_new=1024, max_new=4096, min_past=0, max_past=0, heads=32,
             kv_heads=32, dim=128, page=16, window=0, dtype="f16", layout="nhd", empty=False),
        # the last chunk of a long document
        dict(name="chunk_long", op="chunk", batch=1, min_new=4096, max_new=4096, min_past=28672, max_past=28672, heads=32,
             kv_heads=8, dim=128, page=64, window=0, dtype="bf16", layout="hnd", empty=False),
        # odd everything: three query heads a key head, 80 wide, pages of 13, a sliding window, sequences without tokens
        dict(name="chunk_window_odd", op="chunk", batch=9, min_new=3, max_new=701, min_past=1, max_past=4302, heads=15,
             kv_heads=5, dim=80, page=13, window=1000, dtype="f16", layout="nhd", empty=True),
        # a decode step's batch: q and k of each sequence's token, to be given to the attention
        dict(name="rotary_step", op="rotary", tokens=64, heads=32, kv_heads=8, dim=128, rot=128, interleaved=False, page=16,
             scaling="none", max_pos=8192, dtype="bf16", append=False),
        # a large chunk far into a long context: scaled frequencies, keys and values into the cache
        dict(name="rotary_prompt", op="rotary", tokens=8192, heads=32, kv_heads=8, dim=128, rot=128, interleaved=False, page=64,
             scaling="ramp", max_pos=131072, dtype="bf16", append=True),
        # pairs side by side, part of an odd head, pages of 13, rows of a padded batch
        dict(name="rotary_odd", op="rotary", tokens=777, heads=15, kv_heads=5, dim=80, rot=32, interleaved=True, page=13,
             scaling="bands", max_pos=30000, dtype="f16", append=True),
        # a small decode batch, the residual in the activations' type
        dict(name="norm_step", op="norm", rows=8, hidden=4096, dtype="bf16", residual="bf16", weight=True),
        # a large chunk on a residual of 32 bits
        dict(name="norm_prompt", op="norm", rows=8192, hidden=4096, dtype="bf16", residual="f32", weight=True),
        # a decode step's plan: a token for each sequence
        dict(name="plan_step", op="plan", batch=64, page=16, max_past=8192, max_new=1, drop=False),
        # a server's mixed step: chunks, single tokens, sequences that end or take back what was guessed ahead
        dict(name="plan_chunks", op="plan", batch=512, page=16, max_past=16384, max_new=512, drop=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "rotary", "norm", "plan"])
    if op == "chunk":
        kv, per, dim = rng.choice([(8, 4, 128), (32, 1, 128), (8, 5, 128), (4, 8, 128), (1, 16, 128), (2, 7, 64),
                                   (12, 1, 64), (5, 3, 80), (8, 1, 96), (4, 4, 256), (2, 24, 128)])
        batch = _log_int(rng, 1, 24)
        max_new = _log_int(rng, 1, 4096 if batch <= 4 else 1024)
        # scores of the padded batch, and the products of the whole, stay below the largest listed case's
        most = int(3.0e9 / (batch * max_new * kv * per * max(1.0, dim / 128)))
        max_past = _log_int(rng, 1, max(16, min(32768, most) - max_new))
        return dict(op="chunk", batch=batch, min_new=_log_int(rng, 1, max_new), max_new=max_new,
                    min_past=rng.choice([0, _log_int(rng, 1, max_past)]), max_past=max_past, heads=kv * per, kv_heads=kv, dim=dim,
                    page=rng.choice([8, 13, 16, 16, 32, 64, 128, 256]), window=rng.choice([0, 0, 0, _log_int(rng, 8, 4096)]),
                    dtype=rng.choice(["f16", "bf16"]), layout=rng.choice(["nhd", "hnd"]), empty=rng.choice([False, True]))
    if op == "rotary":
        kv, per, dim = rng.choice([(8, 4, 128), (32, 1, 128), (4, 8, 128), (2, 7, 64), (5, 3, 80), (8, 1, 96), (4, 4, 256)])
        return dict(op="rotary", tokens=_log_int(rng, 1, 6000), heads=kv * per, kv_heads=kv, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2, dim // 16 * 8]), interleaved=rng.choice([False, True]),
                    page=rng.choice([8, 13, 16, 32, 64]), scaling=rng.choice(["none", "linear", "base", "ramp", "bands"]),
                    max_pos=_log_int(rng, 100, 1000000), dtype=rng.choice(["f16", "bf16"]), append=rng.choice([False, True]))
    if op == "norm":
        hidden = rng.choice([_log_int(rng, 64, 16384), 8 * _log_int(rng, 16, 1024), 4096, 5120])
        return dict(op="norm", rows=_log_int(rng, 1, min(16384, int(3.3e7 / hidden))), hidden=hidden,
                    dtype=rng.choice(["f16", "bf16"]), residual=rng.choice(["none", "same", "same", "f32"]),
                    weight=rng.choice([True, True, False]))
    return dict(op="plan", batch=_log_int(rng, 1, 1024), page=rng.choice([1, 8, 13, 16, 32, 64]), max_past=_log_int(rng, 16, 8192),
                max_new=_log_int(rng, 1, 64), drop=rng.choice([False, True]))


def _spread(lo, hi, i):
    """The i-th of a sequence of lengths spread over [lo, hi], evenly in their logarithm where lo > 0."""
    at = (0.618034 * (i + 1)) % 1.0
    if lo <= 0:
        return min(hi, int(at * (hi + 1)))
    return max(lo, min(hi, int(round(math.exp(math.log(lo) + (math.log(hi) - math.log(lo)) * at)))))


def _chunk_lengths(c):
    """(new tokens, keys) of each sequence; the first has the most of both."""
    new = [_spread(c["min_new"], c["max_new"], 3 * i) for i in range(c["batch"])]
    past = [_spread(c["min_past"], c["max_past"], i) for i in range(c["batch"])]
    new[0], past[0] = c["max_new"], c["max_past"]
    if c["min_new"] == 1 and c["batch"] > 4:      # a mixed step: three of four sequences bring one token
        new = [n if i % 4 == 0 else 1 for i, n in enumerate(new)]
    if c["empty"] and c["batch"] > 2:
        new[c["batch"] // 2] = 0                   # one that waits, with its keys in the cache
        new[-1] = past[-1] = 0                     # and one that is not there
    return new, [a + b for a, b in zip(new, past)]


def _plan_lengths(c):
    """(cached, added) of each sequence."""
    cached = [_spread(0, c["max_past"], i) for i in range(c["batch"])]
    added = [1 if c["max_new"] == 1 or i % 4 else _spread(1, c["max_new"], i) for i in range(c["batch"])]
    if c["drop"]:
        for i in range(c["batch"]):
            if i % 7 == 3:
                added[i] = -cached[i]                              # ended
            elif i % 7 == 5:
                added[i] = -min(cached[i], 1 + i % 9)              # guesses that were wrong
            elif i % 7 == 6:
                added[i] = 0                                       # waiting
    return cached, added


def _pages(n, page):
    return -(-n // page)


def _size(name):
    return 4 if name == "f32" else 2


def work(c):
    if c["op"] == "chunk":
        new, lens = _chunk_lengths(c)
        seen, keys, table = 0, 0, 0
        for m, n in zip(new, lens):
            w = c["window"] or n
            first = n - m                                          # position of the first new token
            full = max(0, min(m, w - first - 1))                   # tokens that see all keys before them
            seen += full * first + full * (full + 1) // 2 + (m - full) * w
            live = min(n, m + w - 1) if m else 0
            keys += live
            table += 4 * _pages(live, c["page"])
        io = sum(new) * c["heads"] * (2 * c["dim"] * 2 + 4)
        return {"bytes": keys * c["kv_heads"] * c["dim"] * 4 + io + table + 8 * c["batch"], "flops": 4 * seen * c["heads"] * c["dim"]}
    if c["op"] == "rotary":
        rows = c["heads"] + c["kv_heads"] * (2 if c["append"] else 1)
        return {"bytes": c["tokens"] * (2 * 2 * rows * c["dim"] + 4 + (8 if c["append"] else 0)) + 4 * c["rot"],
                "flops": 3 * c["tokens"] * (c["heads"] + c["kv_heads"]) * c["rot"]}
    if c["op"] == "norm":
        res = {"none": 0, "same": 2, "f32": 4}.get(c["residual"], 2)
        return {"bytes": c["rows"] * c["hidden"] * (4 + 2 * res) + (2 * c["hidden"] if c["weight"] else 0),
                "flops": 4 * c["rows"] * c["hidden"]}
    cached, added = _plan_lengths(c)
    moved = sum(abs(_pages(a + b, c["page"]) - _pages(a, c["page"])) for a, b in zip(cached, added))
    tokens = sum(max(0, b) for b in added)
    return {"bytes": 16 * c["batch"] + 8 * moved + 12 * tokens, "flops": 4 * tokens}


# ---------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = _generator(seed)
    return {"chunk": _prepare_chunk, "rotary": _prepare_rotary, "norm": _prepare_norm, "plan": _prepare_plan}[case["op"]](dict(case), gen)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


def _random_table(need, width, gen, spare=3):
    """(block table, pages): sequence b owns the next need[b] pages of a shuffled order; the rest of its row is -1."""
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    need_t = _ints(need, torch.int64)
    first = torch.cumsum(need_t, 0) - need_t
    j = torch.arange(width, device=DEV)
    table = torch.where(j[None] < need_t[:, None], order[(first[:, None] + j[None]).clamp(max=pages - 1)], -1)
    return table.to(torch.int32), order


def _prepare_chunk(c, gen):
    dt, page = DTYPES[c["dtype"]], c["page"]
    new, lens = _chunk_lengths(c)
    need = [_pages(n, page) for n in lens]
    width = max(1, max(need))
    table, order = _random_table(need, width, gen)
    pages = order.numel()
    shape = (pages, page, c["kv_heads"], c["dim"]) if c["layout"] == "nhd" else (pages, c["kv_heads"], page, c["dim"])
    j = torch.arange(width, device=DEV)
    pos = j[None, :, None] * page + torch.arange(page, device=DEV)
    live = pos < _ints(lens)[:, None, None]
    used = torch.zeros((pages, page), dtype=torch.bool, device=DEV)
    used[table.clamp(min=0).long()[live.any(-1)]] = live[live.any(-1)]
    caches = []
    for _ in range(2):
        t = torch.empty(shape, dtype=dt, device=DEV).normal_(generator=gen)
        t = t if c["layout"] == "nhd" else t.permute(0, 2, 1, 3)
        t[~used] = float("nan")                    # what no sequence has written holds anything at all
        caches.append(t)
    tokens = sum(new)
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    # the queries of the step as the projection leaves them: beside the keys and values of their tokens
    fused = torch.empty((tokens, c["heads"] + 2 * c["kv_heads"], c["dim"]), dtype=dt, device=DEV).normal_(generator=gen)
    s = dict(c, table=table, k=caches[0], v=caches[1], q=fused[:, :c["heads"]], lens=_ints(lens), cu=_ints(cu), tokens=tokens,
             width=width, most_new=max(new), scale=c["dim"] ** -0.5)
    s["lse"] = torch.empty((tokens, c["heads"]), device=DEV)
    if own:   # a program keeps the workspace of its attention calls
        s["workspace"] = _lib().chunk_attention_workspace(c["heads"], c["kv_heads"], c["dim"])
    return s


# how contexts are stretched: factor, the length the model was trained on, and the two limits between which frequencies change over
SCALING = {"none": None, "linear": (4.0, 0.0, 0.0, 0.0), "base": (8.0, 0.0, 0.0, 0.0), "ramp": (32.0, 4096.0, 1.0, 32.0),
           "bands": (8.0, 8192.0, 1.0, 4.0)}
THETA = 500000.0


def _prepare_rotary(c, gen):
    dt, T, D = DTYPES[c["dtype"]], c["tokens"], c["dim"]
    fused = torch.empty((T, c["heads"] + 2 * c["kv_heads"], D), dtype=dt, device=DEV).normal_(generator=gen)
    q, k, v = fused.split([c["heads"], c["kv_heads"], c["kv_heads"]], 1)
    s = dict(c, q=q, k=k, v=v)
    # some sequences' runs of tokens: each starts anywhere in the context
    run = max(1, T // 5)
    start = torch.randint(0, max(1, c["max_pos"] - run), (-(-T // run),), generator=gen, device=DEV)
    t = torch.arange(T, device=DEV)
    s["positions"] = (start[t // run] + t % run).to(torch.int32)
    if c["append"]:
        pages = _pages(T, c["page"]) + 5
        order = torch.randperm(pages, generator=gen, device=DEV)
        slots = order[t // c["page"]] * c["page"] + t % c["page"]
        s["slots"] = torch.where(t % 97 == 13, -1, slots)          # rows of a padded batch
        for name in ("k_cache", "v_cache"):
            s[name] = torch.zeros((pages, c["page"], c["kv_heads"], D), dtype=dt, device=DEV)
    scaling = SCALING[c["scaling"]]
    if own:
        factor, original, low, high = scaling or (1.0, 0.0, 0.0, 0.0)
        s["turns"], s["amplitude"] = _lib().rotary_table(c["rot"], theta=THETA, scaling=c["scaling"], factor=factor,
                                                         original=original, low=low, high=high)
    else:
        s["freq"], s["amplitude"] = _frequencies(c["rot"], c["scaling"])
    return s


def _frequencies(rot, kind):
    """(angle a position of each pair [rot / 2] in 64 bits, amplitude)."""
    i = torch.arange(rot // 2, device=DEV, dtype=torch.float64)
    f = THETA ** (-2 * i / rot)
    if kind == "none":
        return f, 1.0
    factor, original, low, high = SCALING[kind]
    if kind == "linear":
        return f / factor, 1.0
    if kind == "base":
        return (THETA * factor ** (rot / (rot - 2))) ** (-2 * i / rot) if rot > 2 else f, 1.0
    if kind == "ramp":    # pairs that turn more than `high` times over the trained length keep their frequency, fewer than `low` are stretched
        at = lambda turns: rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(THETA))  # noqa: E731
        a, b = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot - 1)
        ramp = ((i - a) / max(b - a, 0.001)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    turns = original * f / (2 * math.pi)
    keep = ((turns - low) / (high - low)).clamp(0, 1)
    return f / factor * (1 - keep) + f * keep, 1.0


def _prepare_norm(c, gen):
    dt = DTYPES[c["dtype"]]
    s = dict(c, x=torch.empty((c["rows"], c["hidden"]), dtype=dt, device=DEV).normal_(generator=gen))
    s["r"] = s["r_out"] = s["w"] = None
    if c["residual"] != "none":
        rt = DTYPES[c["dtype"] if c["residual"] == "same" else c["residual"]]
        r = torch.empty((c["rows"], c["hidden"]), device=DEV).normal_(generator=gen) * 4
        r[:, ::61] *= 20                                           # the few wide channels of a residual stream
        s["r"], s["r_out"] = r.to(rt), torch.empty((c["rows"], c["hidden"]), dtype=rt, device=DEV)
    if c["weight"]:
        s["w"] = (1 + 0.2 * torch.randn(c["hidden"], generator=gen, device=DEV)).to(dt)
    return s


def _prepare_plan(c, gen):
    page = c["page"]
    cached, added = _plan_lengths(c)
    width = max(1, max(_pages(a + max(0, b), page) for a, b in zip(cached, added)))
    have = [_pages(a, page) for a in cached]
    take = sum(max(0, _pages(a + b, page) - h) for a, b, h in zip(cached, added, have))
    table, order = _random_table(have, width, gen, spare=take + 7)
    held = sum(have)
    free = torch.full((order.numel() + 5,), -1, dtype=torch.int32, device=DEV)     # room for every page
    free[:order.numel() - held] = order[held:]
    return dict(c, cached=_ints(cached), added=_ints(added), table=table, free=free, count=_ints([order.numel() - held]),
                count_out=_ints([0]), tokens=sum(max(0, b) for b in added) + 3)    # three rows of padding


# ---------------------------------------------------------------------------------- one pass
def run(s):
    return {"chunk": _chunk, "rotary": _rotary, "norm": _norm, "plan": _plan}[s["op"]](s)


def _chunk(s):
    if own:
        out = _lib().chunk_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], s["cu"], scale=s["scale"], window=s["window"],
                                     lse=s["lse"], workspace=s["workspace"])
        return [out, s["lse"]]
    B, page, D, kv, M = s["batch"], s["page"], s["dim"], s["kv_heads"], s["most_new"]
    L = s["width"] * page
    start, lens, table = s["cu"][:-1].long(), s["lens"].long(), s["table"].clamp(min=0).long()
    new = s["cu"][1:].long() - start
    # every sequence padded to the most new tokens and the most keys
    i = torch.arange(M, device=DEV)
    row = (start[:, None] + i[None]).clamp(max=s["tokens"] - 1)
    at = lens[:, None] - new[:, None] + i[None]                    # positions of the new tokens
    key = torch.arange(L, device=DEV)
    live = (key[None, None] <= at[:, :, None]) & (i[None] < new[:, None])[:, :, None]
    if s["window"]:
        live &= key[None, None] > at[:, :, None] - s["window"]
    k = s["k"][table].reshape(B, L, kv, D).permute(0, 2, 3, 1).float()
    q = s["q"][row].reshape(B, M, kv, -1, D).permute(0, 2, 3, 1, 4).reshape(B, kv, -1, D).float()
    scores = (q @ k * s["scale"]).reshape(B, kv, -1, M, L).masked_fill_(~live[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    base = torch.where(top == float("-inf"), 0.0, top)
    p = scores.sub_(base).exp_()
    total = p.sum(-1, keepdim=True)
    inside = (key[None] < lens[:, None])[:, None, :, None]
    v = s["v"][table].reshape(B, L, kv, D).permute(0, 2, 1, 3).float().masked_fill(~inside, 0.0)
    out = (p.reshape(B, kv, -1, L) @ v).reshape(B, kv, -1, M, D) / torch.where(total == 0, 1.0, total)
    out = out.permute(0, 3, 1, 2, 4).reshape(B, M, s["heads"], D)
    lse = (base + torch.log(total))[..., 0].permute(0, 3, 1, 2).reshape(B, M, s["heads"])
    mine = i[None] < new[:, None]
    return [out[mine].to(s["q"].dtype), lse[mine]]


def _rotary(s):
    if own:
        extra = dict(v=s["v"], k_cache=s["k_cache"], v_cache=s["v_cache"], slots=s["slots"]) if s["append"] else {}
        q, k = _lib().rotary(s["q"], s["k"], s["positions"], s["turns"], amplitude=s["amplitude"], interleaved=s["interleaved"],
                             **extra)
        return [q, s["k_cache"], s["v_cache"]] if s["append"] else [q, k]
    half = s["rot"] // 2
    angle = s["positions"].double()[:, None, None] * s["freq"]
    cos, sin = (f(angle).float() * s["amplitude"] for f in (torch.cos, torch.sin))

    def rotate(x):
        x = x.float()
        part, rest = x[..., :s["rot"]], x[..., s["rot"]:]
        a, b = (part[..., 0::2], part[..., 1::2]) if s["interleaved"] else (part[..., :half], part[..., half:])
        pair = a * cos - b * sin, a * sin + b * cos
        part = torch.stack(pair, -1).flatten(-2) if s["interleaved"] else torch.cat(pair, -1)
        return torch.cat([part, rest], -1).to(s["q"].dtype)

    q, k = rotate(s["q"]), rotate(s["k"])
    if not s["append"]:
        return [q, k]
    keep = s["slots"] >= 0
    page, slot = s["slots"][keep] // s["page"], s["slots"][keep] % s["page"]
    s["k_cache"][page, slot], s["v_cache"][page, slot] = k[keep], s["v"][keep]
    return [q, s["k_cache"], s["v_cache"]]


def _norm(s):
    if own:
        out = _lib().rms_norm(s["x"], s["w"], residual=s["r"], residual_out=s["r_out"], eps=1e-6)
        return [out] if s["r"] is None else [out, s["r_out"]]
    t = s["x"].float() if s["r"] is None else s["x"].float() + s["r"].float()
    y = t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6)
    if s["w"] is not None:
        y = y * s["w"].float()
    out = y.to(s["x"].dtype)
    return [out] if s["r"] is None else [out, t.to(s["r"].dtype)]


def _plan(s):
    if own:
        lens, cu, positions, slots = _lib().page_plan(s["cached"], s["added"], s["table"], s["free"], s["count"], page_size=s["page"],
                                                      max_tokens=s["tokens"], free_count_out=s["count_out"])
        return [lens, cu, positions, slots, s["table"], s["free"], s["count_out"]]
    page, cached, added, table, free = s["page"], s["cached"].long(), s["added"].long(), s["table"], s["free"]
    lens = cached + added
    have, need = (cached + page - 1) // page, (lens + page - 1) // page
    give, take = (have - need).clamp(min=0), (need - have).clamp(min=0)
    j = torch.arange(table.shape[1], device=DEV)[None]
    # pages of dropped tokens go back in order, then pages are taken from the top in order
    back = (j >= need[:, None]) & (j < have[:, None])
    count = s["count"][0].long()
    where = count + (torch.cumsum(give, 0) - give)[:, None] + j - need[:, None]
    free[where[back]] = table[back]
    count = count + give.sum()
    fresh = (j >= have[:, None]) & (j < need[:, None])
    where = count - 1 - (torch.cumsum(take, 0) - take)[:, None] - (j - have[:, None])
    table[fresh] = free[where[fresh]]
    s["count_out"][0] = count - take.sum()
    new = added.clamp(min=0)
    upto = torch.cumsum(new, 0)
    t = torch.arange(s["tokens"], device=DEV)
    seq = torch.searchsorted(upto, t, right=True)
    live = seq < s["batch"]
    seq = seq.clamp(max=s["batch"] - 1)
    at = cached[seq] + t - (upto - new)[seq]
    at = torch.where(live, at, 0)
    entry = table[seq, (at // page).clamp(max=table.shape[1] - 1)].long()
    slots = torch.where(live, entry * page + at % page, -1)
    cu = torch.cat([upto.new_zeros(1), upto])
    return [lens.to(torch.int32), cu.to(torch.int32), at.to(torch.int32), slots, table, free, s["count_out"]]


# ---------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":      # whole numbers: counted sequence by sequence
        return _exact_plan(s)
    return {"chunk": _exact_chunk, "rotary": _exact_rotary, "norm": _exact_norm}[case["op"]](s)


def _exact_chunk(s):
    kv, D, page = s["kv_heads"], s["dim"], s["page"]
    new, lens = _chunk_lengths(s)
    out = torch.zeros((s["tokens"], s["heads"], D), dtype=torch.float64, device=DEV)
    lse = torch.zeros((s["tokens"], s["heads"]), dtype=torch.float64, device=DEV)
    row = 0
    for b, (m, n) in enumerate(zip(new, lens)):
        pages = s["table"][b, :_pages(n, page)].long()
        for h in range(kv if m else 0):
            keys, values = (t[pages][:, :, h].reshape(-1, D)[:n].double() for t in (s["k"], s["v"]))
            heads = slice(h * (s["heads"] // kv), (h + 1) * (s["heads"] // kv))
            for lo in range(0, m, 1024):           # 1024 tokens at a time
                take = slice(row + lo, row + min(m, lo + 1024))
                at = n - m + torch.arange(lo, min(m, lo + 1024), device=DEV)[:, None]
                j = torch.arange(n, device=DEV)[None]
                hidden = j > at
                if s["window"]:
                    hidden = hidden | (j <= at - s["window"])
                x = torch.einsum("thd,nd->htn", s["q"][take, heads].double(), keys) * s["scale"]
                x = x.masked_fill(hidden, float("-inf"))
                out[take, heads] = torch.einsum("htn,nd->thd", torch.softmax(x, -1), values)
                lse[take, heads] = torch.logsumexp(x, -1).T
        row += m
    return [out, lse]


def _exact_rotary(s):
    rot, kind = s["rot"], s["scaling"]
    freq, amplitude = [], 1.0
    factor, original, low, high = SCALING[kind] or (1.0, 0.0, 0.0, 0.0)
    for i in range(rot // 2):
        f = math.exp(-math.log(THETA) * 2 * i / rot)
        if kind == "linear":
            f /= factor
        elif kind == "base" and rot > 2:
            f = math.exp(-(math.log(THETA) + math.log(factor) * rot / (rot - 2)) * 2 * i / rot)
        elif kind == "ramp":
            ends = [rot * math.log(original / (2 * math.pi * n)) / (2 * math.log(THETA)) for n in (high, low)]
            a, b = max(math.floor(ends[0]), 0), min(math.ceil(ends[1]), rot - 1)
            share = min(1.0, max(0.0, (i - a) / max(b - a, 0.001)))
            f = share * f / factor + (1 - share) * f
            amplitude = 1 + math.log(factor) / 10
        elif kind == "bands":
            share = min(1.0, max(0.0, (original * f / (2 * math.pi) - low) / (high - low)))
            f = (1 - share) * f / factor + share * f
        freq.append(f)
    turn = torch.polar(torch.full((s["tokens"], rot // 2), amplitude, dtype=torch.float64, device=DEV),
                       s["positions"].double()[:, None] * torch.tensor(freq, dtype=torch.float64, device=DEV))

    def rotate(x):
        y = x.double().clone()
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if s["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
        z = torch.complex(y[..., a].contiguous(), y[..., b].contiguous()) * turn[:, None]
        y[..., a], y[..., b] = z.real, z.imag
        return y

    q, k = rotate(s["q"]), rotate(s["k"])
    if not s["append"]:
        return [q, k]
    caches = [t.double().reshape(-1, *t.shape[2:]) for t in (s["k_cache"], s["v_cache"])]
    keep = s["slots"] >= 0
    for cache, rows in zip(caches, (k, s["v"].double())):
        cache[s["slots"][keep]] = rows[keep]
    return [q] + [c.reshape(s["k_cache"].shape) for c in caches]


def _exact_norm(s):
    t = s["x"].double()
    if s["r"] is not None:
        t = t + s["r"].double()
    y = torch.nn.functional.normalize(t, dim=-1) * math.sqrt(s["hidden"])
    square = t.square().mean(-1, keepdim=True)
    y = y * (square / (square + 1e-6)).sqrt()
    if s["w"] is not None:
        y = y * s["w"].double()
    return [y] if s["r"] is None else [y, t]


def _exact_plan(s):
    page = s["page"]
    cached, added = _plan_lengths(s)
    table, free, count = s["table"].tolist(), s["free"].tolist(), int(s["count"])
    for b, (a, d) in enumerate(zip(cached, added)):
        for j in range(_pages(a + d, page), _pages(a, page)):
            free[count] = table[b][j]
            count += 1
    cu, positions, slots = [0], [], []
    for b, (a, d) in enumerate(zip(cached, added)):
        for j in range(_pages(a, page), _pages(a + d, page)):
            count -= 1
            table[b][j] = free[count]
        for t in range(a, a + max(0, d)):
            positions.append(t)
            slots.append(table[b][t // page] * page + t % page)
        cu.append(len(positions))
    pad = s["tokens"] - len(positions)
    return [_ints([a + d for a, d in zip(cached, added)]), _ints(cu), _ints(positions + [0] * pad), _ints(slots + [-1] * pad, torch.int64),
            _ints(table), _ints(free), _ints([count])]
