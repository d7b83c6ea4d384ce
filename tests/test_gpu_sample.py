"""gptq_sample against its definition in 64 bits.

A token is accepted when the target mass falls into its interval of the cumulated kept mass within
tol = 2^-20 of the total: each weight is an fp32 exp of an fp32 quotient (relative error up to
2^-23 |x| + 2^-22, |x| < 12 where a weight matters at 2^-17) plus 2^-33 from its fixed point.  Where
the settings or the ties decide exactly, equality is required."""
import numpy as np
import pytest
import torch

import gptq_bit_weight_gemm_gb300 as g

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = 2.0 ** -20


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_bit_weight_gemm_gb300 import build as lib_build
    lib_build.build()
    assert torch.cuda.is_available()
    yield
    assert g.device_status() == 0


def kept_sets(row, t, k, top_p, min_p):
    """(weights, the kept mask, the kept mask with top_p and min_p relaxed and tightened by the tolerance)."""
    V = len(row)
    if t == 0 or not top_p > 0 or not min_p <= 1:
        t, k = (t or 1.0), 1
    w = np.exp((row.astype(np.float64) - row.max()) / t)
    order = np.argsort(-row, kind="stable")
    n = k if 0 < k < V else V
    sw = w[order[:n]]
    before = np.concatenate([[0.0], np.cumsum(sw)[:-1]])
    masks = []
    for slack in (-TOL, 0.0, TOL):
        keep = np.ones(n, bool)
        if top_p < 1:
            keep &= before < (top_p + slack) * sw.sum()
        keep &= sw >= min_p * (1 - 8 * slack)
        keep[0] = True
        m = np.zeros(V, bool)
        m[order[:n][keep]] = True
        masks.append(m)
    return w, masks


def accepted(row, u, t, k, top_p, min_p, token, logprob):
    w, masks = kept_sets(row, t, k, top_p, min_p)
    for m in masks:
        cum = np.cumsum(np.where(m, w, 0.0))
        lo, hi, total = cum[token] - w[token], cum[token], cum[-1]
        if (m[token] and lo - TOL * total <= u * total <= hi + TOL * total
                and abs(logprob - np.log(w[token] / total)) <= 1e-5 * (1 + abs(logprob))):
            return True
    return False


def run(logits, u, t=None, k=None, p=None, m=None):
    d = lambda a, dt: None if a is None else torch.tensor(a, dtype=dt, device=DEV)  # noqa: E731
    tok, lp = g.sample(logits, d(u, torch.float32), temperature=d(t, torch.float32), top_k=d(k, torch.int32),
                       top_p=d(p, torch.float32), min_p=d(m, torch.float32))
    torch.cuda.synchronize()
    return tok.cpu().numpy(), lp.cpu().numpy()


def logits_of(B, V, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    x = 2.0 * torch.randn((B, V), generator=gen)
    x.scatter_add_(1, torch.randint(0, V, (B, min(V, 20)), generator=gen), 4 * torch.rand((B, min(V, 20)), generator=gen))
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 31, 1000, 4097, 50257, 131072])
def test_mixed_settings(V, dtype):
    B = 48
    x = logits_of(B, V, dtype, V)
    rng = np.random.default_rng(V)
    u = rng.random(B).astype(np.float32)
    t = np.where(np.arange(B) % 7 == 6, 0.0, rng.uniform(0.3, 2.0, B)).astype(np.float32)
    k = np.where(np.arange(B) % 3 == 0, 0, rng.integers(1, 400, B)).astype(np.int32)
    p = np.where(np.arange(B) % 4 == 0, 1.0, rng.uniform(0.1, 0.99, B)).astype(np.float32)
    m = np.where(np.arange(B) % 2 == 0, 0.0, rng.uniform(0.0, 0.2, B)).astype(np.float32)
    tok, lp = run(x.to(DEV), u, t, k, p, m)
    rows = x.float().numpy()
    for b in range(B):
        assert accepted(rows[b], float(u[b]), float(t[b]), int(k[b]), float(p[b]), float(m[b]), int(tok[b]), float(lp[b])), b
        if t[b] == 0:
            assert tok[b] == int(np.argmax(rows[b])) and lp[b] == 0.0


@pytest.mark.parametrize("kw", [{}, dict(p=0.9), dict(k=50), dict(m=0.05), dict(p=0.999), dict(k=3000), dict(p=0.5, k=10)])
@pytest.mark.parametrize("B", [1, 5, 160, 400])
def test_one_kind_over_batches(B, kw):
    x = logits_of(B, 9001, torch.bfloat16, B)
    u = np.random.default_rng(B).random(B).astype(np.float32)
    full = {n: np.full(B, v) for n, v in kw.items()}
    tok, lp = run(x.to(DEV), u, **full)
    rows = x.float().numpy()
    for b in range(B):
        assert accepted(rows[b], float(u[b]), 1.0, kw.get("k", 0), float(np.float32(kw.get("p", 1.0))),
                        float(np.float32(kw.get("m", 0.0))), int(tok[b]), float(lp[b])), b


@pytest.mark.parametrize("V", [10, 1000, 30011, 262144])
@pytest.mark.parametrize("value", [0.0, -3.5])
def test_equal_logits_count_by_index(V, value):
    # every weight is 1: the kept set is the first n indices and the token is floor(u n)
    u = np.array([0.0, 0.1, 0.25, 0.5, 0.75, 0.999], np.float32)
    x = torch.full((6, V), value, device=DEV)
    for n, kw in ((V, {}), (7, dict(k=[7] * 6)), (-(-V // 2), dict(p=[0.5] * 6)), (1, dict(k=[1] * 6)),
                  (4, dict(k=[8] * 6, p=[0.5] * 6)), (V, dict(m=[1.0] * 6)), (1, dict(p=[0.0] * 6)), (1, dict(m=[1.5] * 6)),
                  (1, dict(p=[float("nan")] * 6)), (1, dict(t=[0.0] * 6)), (1, dict(t=[float("nan")] * 6)),
                  (V, dict(t=[100.0] * 6)), (V, dict(k=[-4] * 6))):
        tok, lp = run(x, u, **kw)
        assert tok.tolist() == [int(v) for v in np.floor(u.astype(np.float64) * n)], (n, kw)
        assert np.allclose(lp, -np.log(n), atol=1e-5)


def test_two_values_split_by_ties():
    # 5 logits 2.0 among 0.0: top-k cuts the ties of 0.0 by index, negative zero counts as zero
    x = torch.zeros((4, 64), dtype=torch.float16)
    x[:, [9, 20, 33, 40, 63]] = 2.0
    x[:, ::3] = torch.where(x[:, ::3] == 0, -0.0, x[:, ::3])
    kept = [0, 1, 2, 9, 20, 33, 40, 63]
    w = np.exp(np.float64([-2, -2, -2, 0, 0, 0, 0, 0]))
    edges = np.cumsum(w) / w.sum()
    u = ((np.concatenate([[0], edges[:-1]]) + edges) / 2).astype(np.float32)
    for i in range(0, 8, 4):
        tok, _ = run(x.to(DEV), u[i:i + 4], k=[8] * 4)
        assert tok.tolist() == kept[i:i + 4]


def test_infinities_and_nan():
    inf, nan = float("inf"), float("nan")
    x = torch.full((6, 5000), -inf)
    x[0, 17] = 1.0                                    # one token alone
    x[1, [5, 4999]] = inf                             # +inf share the mass
    x[1, 7] = 3.0
    x[2, :] = nan
    x[2, 4321] = -2.0                                 # NaN is never chosen
    x[3, :100] = torch.arange(100) * 0.01             # masked tail
    x[4, 3] = torch.finfo(torch.float32).min          # the type's lowest value is a value
    x[5, 8], x[5, 9] = 1.0, torch.finfo(torch.float32).min
    tok, lp = run(x.to(DEV), [0.3, 0.7, 0.99, 0.9999, 0.5, 0.9999])
    assert tok[0] == 17 and tok[1] == 4999 and tok[2] == 4321 and tok[4] == 3 and tok[5] == 8 and tok[3] in (98, 99)
    assert lp[0] == 0.0 and abs(lp[1] + np.log(2)) < 1e-6
    for kw in (dict(k=[4000] * 6), dict(p=[0.95] * 6), dict(k=[2] * 6, p=[0.9] * 6, m=[0.01] * 6)):
        tok, _ = run(x.to(DEV), [0.3, 0.7, 0.99, 0.2, 0.5, 0.9999], **kw)
        assert tok[0] == 17 and tok[1] == 4999 and tok[2] == 4321 and tok[4] == 3 and tok[5] == 8


def test_no_token():
    x = torch.full((3, 777), float("-inf"), device=DEV)
    x[1, 5] = 0.0
    x[2] = float("nan")
    tok, lp = run(x, [0.5] * 3)
    assert tok.tolist() == [-1, 5, -1] and np.isnan(lp[0]) and np.isnan(lp[2])
    assert g.device_status() == g.DEV_NO_TOKEN


def test_uniform_outside_its_range():
    x = torch.zeros((4, 100), device=DEV)
    x[:, 90:] = float("-inf")
    tok, _ = run(x, [-1.0, float("nan"), 1.0, 7.0])
    assert tok.tolist() == [0, 0, 89, 89]


def test_strided_rows_and_alignment():
    # rows that start at any element, as slices of a larger buffer
    full = logits_of(8, 3001, torch.float16, 8).to(DEV)
    part = full[:, 3:2998]
    u = np.linspace(0.01, 0.97, 8).astype(np.float32)
    tok, lp = run(part, u, p=[0.9] * 8)
    tok2, lp2 = run(part.contiguous(), u, p=[0.9] * 8)
    assert tok.tolist() == tok2.tolist() and lp.tolist() == lp2.tolist()


def test_frequencies_follow_the_distribution():
    # 4096 evenly spaced numbers hit each token in proportion to its probability, within one hit
    n = 4096
    row = torch.tensor([0.0, 1.0, -1.0, 2.0, 0.5, -3.0])
    u = ((np.arange(n) + 0.5) / n).astype(np.float32)
    tok, _ = run(row.repeat(n, 1).to(DEV), u)
    p = torch.softmax(row.double(), 0).numpy()
    assert np.all(np.abs(np.bincount(tok, minlength=6) - p * n) <= 1.0 + 1e-3)


def test_wide_flat_distribution():
    # a crossing inside the bulk: thousands of tokens share the boundary's neighbourhood
    gen = torch.Generator().manual_seed(2)
    x = (torch.randn((6, 200000), generator=gen) * 0.05).to(torch.bfloat16)
    u = np.random.default_rng(2).random(6).astype(np.float32)
    for kw in (dict(p=[0.7] * 6), dict(k=[100000] * 6), dict(k=[60000] * 6, p=[0.5] * 6)):
        tok, lp = run(x.to(DEV), u, **kw)
        for b in range(6):
            assert accepted(x[b].float().numpy(), float(u[b]), 1.0, kw.get("k", [0])[0], float(np.float32(kw.get("p", [1.0])[0])), 0.0,
                            int(tok[b]), float(lp[b])), (b, kw)


@pytest.mark.parametrize("kw", [dict(p=[0.9] * 2), dict(k=[40] * 2, p=[0.8] * 2), dict(k=[5000] * 2), dict(k=[30000] * 2, p=[0.3] * 2)])
def test_row_longer_than_the_histograms_hold(kw):
    # 8 CTAs of more than 65535 tokens each: masses do not go into 32-bit sums
    x = logits_of(2, 600001, torch.float16, 6)
    u = np.array([0.31, 0.87], np.float32)
    tok, lp = run(x.to(DEV), u, **kw)
    for b in range(2):
        assert accepted(x[b].float().numpy(), float(u[b]), 1.0, kw.get("k", [0])[0], float(np.float32(kw.get("p", [1.0])[0])), 0.0,
                        int(tok[b]), float(lp[b])), b


def test_masked_vocabulary():
    # all but a few tokens at the type's lowest value or -inf, as a grammar leaves them
    x = torch.full((4, 100003), torch.finfo(torch.float16).min, dtype=torch.float16)
    x[1::2] = float("-inf")
    keep = [3, 17, 50001, 77777, 100002]
    x[:, keep] = torch.tensor([0.0, 1.0, -1.0, 2.0, 0.5], dtype=torch.float16)
    w = np.exp(np.float64([0.0, 1.0, -1.0, 2.0, 0.5]))
    edges = np.cumsum(w) / w.sum()
    mids = ((np.concatenate([[0], edges[:-1]]) + edges) / 2).astype(np.float32)
    for kw in ({}, dict(k=[100] * 4), dict(p=[0.9999] * 4), dict(k=[2000] * 4, p=[0.9999] * 4)):
        for i in range(5):
            tok, _ = run(x.to(DEV), [mids[i]] * 4, **kw)
            assert tok.tolist() == [keep[i]] * 4, (kw, i, tok)


@pytest.mark.parametrize("temperature", [1e-38, 1e-6, 1e-3, 50.0, 1e30])
def test_extreme_temperatures(temperature):
    x = torch.zeros((3, 5000))
    x[:, 100:110] = 1.0                               # ten equal best tokens
    u = [0.05, 0.55, 0.95]
    for kw in (dict(), dict(k=[30] * 3), dict(p=[0.5] * 3)):
        tok, lp = run(x.to(DEV), u, t=[temperature] * 3, **kw)
        if temperature <= 1e-3:
            n = 5 if "p" in kw else 10
            assert tok.tolist() == [100 + int(n * np.float32(v)) for v in u], (kw, tok)
        else:
            rows = x.numpy()
            for b in range(3):
                assert accepted(rows[b], float(np.float32(u[b])), temperature, kw.get("k", [0])[0], kw.get("p", [1.0])[0], 0.0,
                                int(tok[b]), float(lp[b])), (kw, b)


def test_side_stream_and_repeatable():
    x = logits_of(4, 20000, torch.float32, 1).to(DEV)
    u = torch.rand(4, device=DEV)
    first = g.sample(x, u, top_p=torch.full((4,), 0.9, device=DEV))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(5):
            again = g.sample(x, u, top_p=torch.full((4,), 0.9, device=DEV))
    s.synchronize()
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_wrong_tensors_are_refused():
    x, u = torch.zeros((2, 10), device=DEV), torch.zeros(2, device=DEV)
    for a, kw in (((x.cpu(), u), {}), ((x, u[:1]), {}), ((x.t().contiguous().t(), u), {}), ((x, u), dict(top_p=u[:1]))):
        with pytest.raises(ValueError):
            g.sample(*a, **kw)
    for a, kw in (((x.double(), u), {}), ((x, u.double()), {}), ((x, u), dict(top_k=u))):
        with pytest.raises(TypeError):
            g.sample(*a, **kw)
