"""gptq_sample where most of the vocabulary lies far below the best token: the tail's mass counts.

One token a gap above a flat tail.  A weight is the fp32 exponential of an fp32 quotient; with |x| < 30
its power of two is off by 2^-18 at most, so a tail of share s of the total is off by 2^-18 s.  A mass is
a whole number of 2^-39 of the best token's, so V tokens are off by V 2^-40 (2^-18 at 2^22).  The token's
interval of the cumulated mass and its log probability therefore agree with 64 bits within
V 2^-40 + 2^-18 s + 2^-23 of the total (and a log probability's own 2^-22 |lp|)."""
import numpy as np
import pytest
import torch

import gptq_bit_weight_gemm_gb300 as g

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_bit_weight_gemm_gb300 import build as lib_build
    lib_build.build()
    assert torch.cuda.is_available()
    yield
    assert g.device_status() == 0


def spread(V, where, n):
    """Uniform numbers around and inside the tail's part of the cumulated mass, and elsewhere."""
    peak, tail = 1.0, float(np.exp(-where))
    total = peak + (V - 1) * tail
    at = V // 3
    edges = np.array([at * tail, at * tail + peak]) / total
    u = np.concatenate([edges[0] * np.linspace(0.02, 0.98, n), edges, edges[1] + (1 - edges[1]) * np.linspace(0.02, 0.98, n), [0.0, 0.5]])
    return np.minimum(u, 1 - 2.0 ** -24).astype(np.float32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("V", [50257, 131072, 256000, 2 ** 22])
@pytest.mark.parametrize("gap", [10.0, 20.0, 22.0, 22.25, 25.0, 27.0])
@pytest.mark.parametrize("kw", [{}, dict(p=1 - 2.0 ** -24), dict(k=1.0)])
def test_a_peak_over_a_flat_tail(V, gap, dtype, kw):
    at = V // 3
    u = spread(V, gap, 3)
    B = len(u)
    x = torch.full((1, V), 1.0, dtype=dtype, device=DEV)
    x[0, at] = 1.0 + gap                              # quarters: exact in every type
    x = x.expand(B, V).contiguous() if V < 2 ** 20 else x.expand(B, V)
    args = {}
    if "p" in kw:
        args["top_p"] = torch.full((B,), kw["p"], device=DEV)
    if "k" in kw:                                     # a long top_k that takes the peak and half of the tail
        args["top_k"] = torch.full((B,), V // 2, dtype=torch.int32, device=DEV)
    if x.stride(0) == 0:                              # rows of 2^22 one at a time
        got = [g.sample(x[b:b + 1], torch.from_numpy(u[b:b + 1]).to(DEV), **{n: t[b:b + 1] for n, t in args.items()}) for b in range(B)]
        tok, lp = (torch.cat([r[i] for r in got]).cpu().numpy() for i in range(2))
    else:
        tok, lp = (t.cpu().numpy() for t in g.sample(x, torch.from_numpy(u).to(DEV), **args))
    w = np.full(V, np.exp(-gap))
    w[at] = 1.0
    tail = np.exp(-gap)
    if "p" in kw:                                     # the shortest prefix of the order that reaches p of the mass
        n_tail = int(min(V - 1, max(0.0, np.ceil((kw["p"] * w.sum() - 1.0) / tail))))
    elif "k" in kw:
        n_tail = V // 2 - 1
    else:
        n_tail = V - 1
    kept = np.zeros(V, bool)
    others = np.delete(np.arange(V), at)
    kept[others[:n_tail]] = kept[at] = True
    cum = np.cumsum(np.where(kept, w, 0.0))
    total = cum[-1]
    share = n_tail * tail / total
    tol = V * 2.0 ** -40 + 2.0 ** -18 * share + 2.0 ** -23
    # with p the cut itself moves by as much: the tail is longer or shorter by tol of the total
    slack = tol * (2 if "p" in kw else 1)
    for b in range(B):
        t = int(tok[b])
        assert 0 <= t < V
        if not kept[t]:
            assert "p" in kw and (t - n_tail) * tail <= slack * total, (b, t, n_tail)
        lo, hi = cum[t] - w[t], cum[t]
        goal = float(u[b]) * total
        assert lo - slack * total <= goal <= hi + slack * total, (b, t, lo, goal, hi)
        want = (0.0 if t == at else -gap) - np.log(total)
        assert abs(float(lp[b]) - want) <= slack + 2.0 ** -22 * abs(want), (b, t, float(lp[b]), want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_three_levels(dtype):
    """A peak, a hundred tokens 2^-8 below and a tail 2^-28 below: masses on both sides of a step of the
    histogram's units, with cuts inside each level."""
    V = 131072
    rng = np.random.default_rng(5)
    order = rng.permutation(V)
    x = np.full(V, -19.5)
    x[order[0]], x[order[1:201]] = 0.0, -5.5
    x[order[101:201]] = -4.75
    row = torch.from_numpy(x).to(dtype)
    w = np.exp(row.double().numpy())
    idx = np.argsort(-row.float().numpy(), kind="stable")
    sw = w[idx]
    before = np.concatenate([[0.0], np.cumsum(sw)[:-1]])
    u = np.linspace(0.01, 0.99, 12).astype(np.float32)
    for p in (0.3, 0.6, 0.9, 0.95, 0.999, 0.9999, 0.99999, 0.9999999, 1.0):
        p32 = float(np.float32(p))
        tok, lp = (t.cpu().numpy() for t in g.sample(row.to(DEV).repeat(12, 1), torch.from_numpy(u).to(DEV),
                                                     top_p=torch.full((12,), p, device=DEV)))
        keep = before < p32 * sw.sum() if p32 < 1 else np.ones(V, bool)
        kept = np.zeros(V, bool)
        kept[idx[keep]] = True
        cum = np.cumsum(np.where(kept, w, 0.0))
        total = cum[-1]
        tol = V * 2.0 ** -40 + 2.0 ** -18 * (1 - 1 / w.sum()) + 2.0 ** -23
        step = float(w[kept].min()) / total           # the cut may move by one token
        for b in range(12):
            t = int(tok[b])
            lo, hi = cum[t] - w[t], cum[t]
            assert lo - (2 * tol + step) * total <= float(u[b]) * total <= hi + (2 * tol + step) * total, (p, b, t)
            assert abs(float(lp[b]) - (np.log(w[t]) - np.log(total))) <= 2 * tol + step + 2.0 ** -21 * abs(np.log(w[t])), (p, b, t)
