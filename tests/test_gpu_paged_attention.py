"""gptq_paged_attention against softmax attention in 64 bits, over the sequence's own keys gathered
page by page.

Tolerance, for u = 2^-11 (fp16) or 2^-8 (bf16), the unit roundoff of the cache's type, and A = sum_j
p_j |v_j|:  |out - ref| <= u |ref| + (u + 2^-16 (1 + max|s|)) A + 2^-24.  The first term is the one
rounding of the result; the second allows the probabilities one rounding to 16 bits and the scores
the error of fp32 sums (a score off by d moves its probability by a factor e^d); the last is fp16's
smallest step.  lse: 2^-16 (1 + max|s|).
Everything a sequence has not written -- cache slots past its length, unused pages, block-table entries
past its pages -- holds NaN or an out-of-range index."""
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


class Case:
    def __init__(self, lens, heads, kv, dim, page, dtype, layout="nhd", append=False, seed=0, spread=1.0, width=None):
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.heads, self.kv, self.dim, self.page, self.dtype = list(lens), heads, kv, dim, page, dtype
        B = len(self.lens)
        need = [-(-n // page) for n in self.lens]
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=gen).tolist()
        width = width or max(1, max(need)) + 1
        table = np.full((B, width), 2 ** 31 - 1, np.int32)
        shape = {"nhd": (pages, page, kv, dim), "hnd": (pages, kv, page, dim), "hpn": (kv, pages, page, dim)}[layout]
        perm = {"nhd": (0, 1, 2, 3), "hnd": (0, 2, 1, 3), "hpn": (1, 2, 0, 3)}[layout]
        self.k = torch.full(shape, float("nan"), dtype=dtype).permute(*perm)
        self.v = torch.full(shape, float("nan"), dtype=dtype).permute(*perm)
        self.keys, self.values = [], []
        rnd = lambda *s: (torch.randn(*s, generator=gen) * spread).to(dtype)  # noqa: E731
        self.k_new, self.v_new = (rnd(B, kv, dim), rnd(B, kv, dim)) if append else (None, None)
        for b, n in enumerate(self.lens):
            ids, order = order[:need[b]], order[need[b]:]
            table[b, :need[b]] = ids
            kk, vv = rnd(n, kv, dim), rnd(n, kv, dim)
            for j in range(n - (1 if append else 0)):
                self.k[ids[j // page], j % page], self.v[ids[j // page], j % page] = kk[j], vv[j]
            if append and n:
                kk[n - 1], vv[n - 1] = self.k_new[b], self.v_new[b]
            self.keys.append(kk)
            self.values.append(vv)
        self.q, self.table = rnd(B, heads, dim), table

    def gpu(self):
        d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
        return dict(q=d(self.q), k_cache=d(self.k), v_cache=d(self.v), block_table=d(torch.from_numpy(self.table)),
                    seq_lens=torch.tensor(self.lens, dtype=torch.int32, device=DEV), k_new=d(self.k_new), v_new=d(self.v_new))

    def ref(self, scale, window):
        """(out, tolerance, lse, lse tolerance) in 64 bits."""
        u = 2.0 ** (-11 if self.dtype == torch.float16 else -8)
        out, tol, lse, lse_tol = [], [], [], []
        for b, n in enumerate(self.lens):
            lo = max(0, n - window) if window else 0
            if n == 0:
                z = torch.zeros(self.heads, self.dim, dtype=torch.float64)
                out.append(z), tol.append(z), lse.append(torch.full((self.heads,), -np.inf, dtype=torch.float64))
                lse_tol.append(torch.zeros(self.heads, dtype=torch.float64))
                continue
            q = self.q[b].double().to(DEV).reshape(self.kv, -1, self.dim)
            k, v = (t[b][lo:].double().to(DEV) for t in (self.keys, self.values))
            s = torch.einsum("hgd,nhd->hgn", q, k) * scale
            p = torch.softmax(s, -1)
            o = torch.einsum("hgn,nhd->hgd", p, v)
            big = 1 + s.abs().amax(-1)
            A = torch.einsum("hgn,nhd->hgd", p, v.abs())
            out.append(o.reshape(self.heads, -1).cpu())
            tol.append((u * o.abs() + (u + 2.0 ** -16 * big[..., None]) * A + 2.0 ** -24).reshape(self.heads, -1).cpu())
            lse.append(torch.logsumexp(s, -1).reshape(-1).cpu())
            lse_tol.append((2.0 ** -16 * big).reshape(-1).cpu())
        return torch.stack(out), torch.stack(tol), torch.stack(lse), torch.stack(lse_tol)


def check(c, scale=None, window=0, workspace=None, a=None):
    scale = c.dim ** -0.5 if scale is None else scale
    a = a or c.gpu()
    lse = torch.full((len(c.lens), c.heads), float("nan"), device=DEV)
    out = g.paged_attention(**a, scale=scale, window=window, lse=lse, workspace=workspace)
    torch.cuda.synchronize()
    ref, tol, rl, rlt = c.ref(scale, window)
    err = (out.double().cpu() - ref).abs()
    assert bool((err <= tol).all()), "max error %g, %d outside" % (float(err.nan_to_num(np.inf).max()), int((~(err <= tol)).sum()))
    got = lse.double().cpu()
    live = torch.isfinite(rl)
    assert torch.equal(got[~live], rl[~live]) and bool(((got - rl).abs()[live] <= rlt[live]).all())
    return out


LENS = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 0, 200, 511]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads,kv,dim", [(8, 8, 128), (8, 2, 64), (15, 5, 80), (14, 2, 128), (16, 1, 96), (24, 1, 128),
                                          (4, 4, 256), (6, 2, 8), (40, 1, 72)])
def test_heads_and_dims(dtype, heads, kv, dim):
    check(Case(LENS, heads, kv, dim, 16, dtype, seed=dim))


@pytest.mark.parametrize("page", [1, 3, 8, 13, 16, 64, 100, 1024])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "hpn"])
def test_pages_and_layouts(page, layout):
    check(Case(LENS, 8, 2, 64, page, torch.float16, layout=layout, seed=page))


@pytest.mark.parametrize("window", [1, 2, 16, 33, 64, 100, 511, 512, 5000])
def test_sliding_window(window):
    check(Case(LENS + [700], 8, 4, 64, 13, torch.bfloat16, seed=window), window=window)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads,kv", [(8, 2), (20, 1)])
def test_append_writes_the_slot_and_nothing_else(dtype, heads, kv):
    c = Case(LENS, heads, kv, 64, 16, dtype, append=True, seed=3)
    a = c.gpu()
    bits = lambda t: t.contiguous().view(torch.int16).cpu().numpy()  # noqa: E731
    before = [bits(a["k_cache"]), bits(a["v_cache"])]
    check(c, a=a)
    for cache, old, new in (("k_cache", before[0], c.k_new), ("v_cache", before[1], c.v_new)):
        want = old.copy()
        for b, n in enumerate(c.lens):
            if n:
                want[c.table[b, (n - 1) // 16], (n - 1) % 16] = bits(new[b])
        assert np.array_equal(bits(a[cache]), want), cache


@pytest.mark.parametrize("batch", [1, 3])
@pytest.mark.parametrize("length", [4096, 20011])
def test_long(batch, length):
    check(Case([length] + [length // 7] * (batch - 1), 8, 2, 128, 64, torch.bfloat16, seed=length))


def test_many_sequences_and_one_long_one():
    lens = [(i * 37) % 90 for i in range(700)]
    lens[311] = 9000
    check(Case(lens, 4, 2, 64, 16, torch.float16, seed=9))


def test_large_scores():
    # scores of hundreds: the running maximum carries the whole softmax
    check(Case(LENS, 8, 2, 64, 16, torch.float16, seed=4, spread=6.0), scale=1.0)


def test_one_workspace_for_every_shape_and_repeatable():
    ws = g.paged_attention_workspace(16, 1, 256)
    need = ws.numel()
    outs = {}
    for turn in range(3):
        for i, (lens, heads, kv, dim) in enumerate([([5000], 16, 1, 64), (LENS, 8, 2, 64), ([3000, 1, 2500], 8, 8, 128)]):
            size = g.paged_attention_workspace_size(heads, kv, dim)
            w = ws if size <= need else g.paged_attention_workspace(heads, kv, dim)
            out = check(Case(lens, heads, kv, dim, 16, torch.float16, seed=i), workspace=w)
            if turn:
                assert torch.equal(out, outs[i])       # the same bits every time
            outs[i] = out


def test_strided_queries_and_side_stream():
    # q, k_new and v_new as slices of one projection's output, on a stream of their own
    c = Case([40, 3, 100], 8, 2, 64, 16, torch.float16, append=True, seed=5)
    a = c.gpu()
    fused = torch.cat([a["q"].reshape(3, -1), a["k_new"].reshape(3, -1), a["v_new"].reshape(3, -1)], 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = g.paged_attention(fused[:, :512].view(3, 8, 64), a["k_cache"], a["v_cache"], a["block_table"], a["seq_lens"],
                                k_new=fused[:, 512:640].view(3, 2, 64), v_new=fused[:, 640:].view(3, 2, 64))
    s.synchronize()
    ref, tol, _, _ = c.ref(64 ** -0.5, 0)
    assert bool(((out.double().cpu() - ref).abs() <= tol).all())


def test_cache_past_32_bit_offsets():
    # the last page starts past 2^31 elements: 5 GB of cache, of which two pages are live
    pages, page, kv, dim = 2 ** 31 // (256 * 2 * 64) + 40, 256, 2, 64
    k = torch.empty((pages, page, kv, dim), dtype=torch.float16, device=DEV)
    v = torch.empty_like(k)
    ids = [pages - 1, 3, pages - 7]
    gen = torch.Generator(device=DEV).manual_seed(1)
    for i in ids:
        k[i].normal_(generator=gen), v[i].normal_(generator=gen)
    n = 2 * page + 100
    q = torch.randn((1, 8, dim), device=DEV, generator=gen).half()
    out = g.paged_attention(q, k, v, torch.tensor([ids], dtype=torch.int32, device=DEV),
                            torch.tensor([n], dtype=torch.int32, device=DEV))
    kk, vv = (torch.cat([t[i] for i in ids])[:n].double() for t in (k, v))
    s = torch.einsum("hgd,nhd->hgn", q[0].double().reshape(kv, 4, dim), kk) * dim ** -0.5
    p = torch.softmax(s, -1)
    ref = torch.einsum("hgn,nhd->hgd", p, vv).reshape(8, dim)
    A = torch.einsum("hgn,nhd->hgd", p, vv.abs()).reshape(8, dim)
    tol = 2.0 ** -11 * ref.abs() + (2.0 ** -11 + 2.0 ** -16 * (1 + float(s.abs().max()))) * A + 2.0 ** -24
    assert bool(((out[0].double() - ref).abs() <= tol).all())


def test_bad_table_entries_and_lengths_are_flagged():
    c = Case([40, 50, 33], 8, 2, 64, 16, torch.float16, seed=6)
    a = c.gpu()
    good = g.paged_attention(**a)
    a["block_table"][1, 1] = -5                       # keys 16..31 of sequence 1
    out = g.paged_attention(**a)
    assert g.device_status() == g.DEV_PAGE_RANGE
    assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    k, v = (torch.cat([t[1][:16], t[1][32:]]).double() for t in (c.keys, c.values))
    s = torch.einsum("hgd,nhd->hgn", c.q[1].double().reshape(2, 4, 64), k) / 8
    ref = torch.einsum("hgn,nhd->hgd", torch.softmax(s, -1), v).reshape(8, 64)
    assert float((out[1].double().cpu() - ref).abs().max()) < 0.01
    a = c.gpu()
    a["seq_lens"][0] = -3
    a["seq_lens"][2] = 10 ** 9                        # longer than the block table
    a["block_table"][2] = a["block_table"][1]
    a["block_table"][2, 2:] = -1
    out = g.paged_attention(**a)
    assert g.device_status() == g.DEV_SEQ_LEN | g.DEV_PAGE_RANGE
    assert float(out[0].abs().max()) == 0.0 and torch.equal(out[1], good[1])


def test_wrong_tensors_are_refused():
    a = Case([4], 8, 2, 64, 16, torch.float16).gpu()
    for kw in (dict(q=a["q"].cpu()), dict(k_cache=a["k_cache"][..., :32]), dict(block_table=a["block_table"][0]),
               dict(k_new=a["q"][:, :2].contiguous())):
        with pytest.raises(ValueError):
            g.paged_attention(**dict(a, **kw))
    for kw in (dict(q=a["q"].float()), dict(v_cache=a["v_cache"].bfloat16()), dict(seq_lens=a["seq_lens"].long())):
        with pytest.raises(TypeError):
            g.paged_attention(**dict(a, **kw))
    with pytest.raises(g.GPTQError) as e:
        g.paged_attention(**a, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    assert e.value.code == -4
