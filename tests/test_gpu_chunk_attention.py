"""gptq_chunk_attention against causal softmax attention in 64 bits, over each sequence's own keys gathered
page by page.

Tolerance, for u = 2^-11 (fp16) or 2^-8 (bf16), the unit roundoff of the type, and A = sum_j p_j |v_j|:
  |out - ref| <= u |ref| + (u + 2^-16 (1 + max|s|)) A + n 2^-30 max|v| + 2^-24.
The first term is the one rounding of the result; the second allows the probabilities one rounding to the type and
the scores the error of fp32 sums (a score off by d moves its probability by a factor e^d); the third what fp16
cannot hold of a probability (half of 2^-24, taken times 2^7 and at most 2^8 below the largest); the last is
fp16's smallest step.  lse: 2^-16 (1 + max|s|).
Everything a sequence has not written -- cache slots past its length, unused pages, block-table entries past its
pages -- holds NaN or an out-of-range index; rows outside every sequence hold a mark that has to stay."""
import numpy as np
import pytest
import torch

import gptq_bit_weight_gemm_gb300 as g

pytestmark = pytest.mark.gpu
DEV = "cuda"
MARK = 77.0


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_bit_weight_gemm_gb300 import build as lib_build
    lib_build.build()
    assert torch.cuda.is_available()
    yield
    assert g.device_status() == 0


class Case:
    """new[b] tokens and lens[b] keys of each sequence; pad rows behind the last."""

    def __init__(self, new, lens, heads, kv, dim, page, dtype, layout="nhd", seed=0, spread=1.0, pad=0, strided=False):
        gen = torch.Generator().manual_seed(seed)
        self.new, self.lens, self.heads, self.kv, self.dim, self.page, self.dtype = list(new), list(lens), heads, kv, dim, page, dtype
        B = len(self.lens)
        need = [-(-n // page) for n in self.lens]
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=gen).tolist()
        table = np.full((B, max(1, max(need)) + 1), 2 ** 31 - 1, np.int32)
        shape = {"nhd": (pages, page, kv, dim), "hnd": (pages, kv, page, dim), "hpn": (kv, pages, page, dim)}[layout]
        perm = {"nhd": (0, 1, 2, 3), "hnd": (0, 2, 1, 3), "hpn": (1, 2, 0, 3)}[layout]
        self.k = torch.full(shape, float("nan"), dtype=dtype).permute(*perm)
        self.v = torch.full(shape, float("nan"), dtype=dtype).permute(*perm)
        rnd = lambda *s: (torch.randn(*s, generator=gen) * spread).to(dtype)  # noqa: E731
        self.keys, self.values, self.pages = [], [], []
        for b, n in enumerate(self.lens):
            ids, order = order[:need[b]], order[need[b]:]
            table[b, :need[b]] = ids
            kk, vv = rnd(n, kv, dim), rnd(n, kv, dim)
            at = torch.arange(n)
            where = torch.tensor(ids, dtype=torch.long)[at // page], at % page
            self.k[where], self.v[where] = kk, vv
            self.keys.append(kk)
            self.values.append(vv)
            self.pages.append(where)
        self.tokens = sum(self.new) + pad
        self.table = torch.from_numpy(table)
        self.q = rnd(self.tokens, heads, dim)
        self.strided = strided
        self.cu = torch.tensor([0] + list(np.cumsum(self.new)), dtype=torch.int32)

    def gpu(self):
        q = self.q.to(DEV)
        if self.strided:    # a slice of a wider projection
            q = torch.cat([q, torch.full((self.tokens, 3, self.dim), float("nan"), dtype=self.dtype, device=DEV)], 1)[:, :self.heads]
        return dict(q=q, k_cache=self.k.to(DEV), v_cache=self.v.to(DEV), block_table=self.table.to(DEV),
                    seq_lens=torch.tensor(self.lens, dtype=torch.int32, device=DEV), cu_tokens=self.cu.to(DEV))

    def one_head(self, b, row, h):
        """The same problem of sequence b and kv head h alone (without a cache)."""
        c, g_ = object.__new__(Case), self.heads // self.kv
        c.new, c.lens, c.heads, c.kv, c.dim, c.dtype = [self.new[b]], [self.lens[b]], g_, 1, self.dim, self.dtype
        c.q = self.q[row:row + self.new[b], h * g_:(h + 1) * g_]
        c.keys, c.values = [self.keys[b][:, h:h + 1]], [self.values[b][:, h:h + 1]]
        return c

    def ref(self, scale, window):
        """(out, tolerance, lse, lse tolerance) of the sequences' rows, in 64 bits."""
        u = 2.0 ** (-11 if self.dtype == torch.float16 else -8)
        out, tol, lse, lse_tol, row = [], [], [], [], 0
        for b, (m, n) in enumerate(zip(self.new, self.lens)):
            if m == 0:
                continue
            if m * n * self.heads > 1 << 28:
                parts = [self.one_head(b, row, h).ref(scale, window) for h in range(self.kv)]
                for into, x in zip((out, tol, lse, lse_tol), zip(*parts)):
                    into.append(torch.cat(x, 1))
                row += m
                continue
            q = self.q[row:row + m].double().to(DEV).reshape(m, self.kv, self.heads // self.kv, self.dim)
            row += m
            k, v = (t[b].double().to(DEV) for t in (self.keys, self.values))
            at = n - m + torch.arange(m, device=DEV)[:, None]
            j = torch.arange(n, device=DEV)[None]
            live = (j <= at) & ((j > at - window) if window else (j >= 0))
            s = torch.einsum("thgd,nhd->hgtn", q, k) * scale
            s = s.masked_fill(~live, -np.inf)
            none = ~live.any(-1)
            p = torch.softmax(s, -1).masked_fill(none[:, None], 0.0) if n else s
            big = 1 + s.abs().masked_fill(~live, 0.0).amax(-1) if n else torch.ones(s.shape[:-1], dtype=torch.float64, device=DEV)
            o = torch.einsum("hgtn,nhd->thgd", p, v)
            A = torch.einsum("hgtn,nhd->thgd", p, v.abs())
            top = v.abs().amax() if n else 0.0
            out.append(o.reshape(m, self.heads, -1))
            bigt = big.permute(2, 0, 1)
            tol.append((u * o.abs() + (u + 2.0 ** -16 * bigt[..., None]) * A + n * 2.0 ** -30 * top + 2.0 ** -24).reshape(m, self.heads, -1))
            lse.append(torch.logsumexp(s, -1).permute(2, 0, 1).reshape(m, -1) if n else torch.full((m, self.heads), -np.inf, device=DEV).double())
            lse_tol.append((2.0 ** -16 * bigt).reshape(m, -1))
        return tuple(torch.cat(t) for t in (out, tol, lse, lse_tol))


def check(c, scale=None, window=0, workspace=None, a=None):
    scale = c.dim ** -0.5 if scale is None else scale
    a = a or c.gpu()
    out = torch.full((c.tokens, c.heads, c.dim), MARK, dtype=c.dtype, device=DEV)
    lse = torch.full((c.tokens, c.heads), MARK, device=DEV)
    g.chunk_attention(**a, scale=scale, window=window, out=out, lse=lse, workspace=workspace)
    torch.cuda.synchronize()
    ref, tol, rl, rlt = c.ref(scale, window)
    live = ref.shape[0]
    err = (out[:live].double() - ref).abs()
    assert bool((err <= tol).all()), "max error %g, %d outside, first %s" % (
        float(err.nan_to_num(np.inf).max()), int((~(err <= tol)).sum()), (~(err <= tol)).nonzero()[0].tolist())
    got = lse[:live].double()
    fin = torch.isfinite(rl)
    assert torch.equal(got[~fin], rl[~fin]) and bool(((got - rl).abs()[fin] <= rlt[fin]).all())
    assert bool((out[live:] == MARK).all()) and bool((lse[live:] == MARK).all())
    return out


NEW = [1, 2, 15, 16, 17, 0, 33, 64, 65, 127, 129, 1, 200, 0, 3]
LENS = [1, 2, 15, 40, 17, 9, 300, 64, 193, 128, 129, 511, 333, 0, 256]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads,kv,dim", [(8, 8, 128), (8, 2, 64), (15, 5, 80), (14, 2, 128), (16, 1, 96), (24, 1, 128),
                                          (4, 4, 256), (6, 2, 8), (40, 1, 72), (2, 1, 200), (300, 1, 16)])
def test_heads_and_dims(dtype, heads, kv, dim):
    check(Case(NEW, LENS, heads, kv, dim, 16, dtype, seed=dim, pad=5))


@pytest.mark.parametrize("page", [1, 3, 8, 13, 16, 64, 100, 1024])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "hpn"])
def test_pages_and_layouts(page, layout):
    check(Case(NEW, LENS, 8, 2, 64, page, torch.float16, layout=layout, seed=page, strided=True))


@pytest.mark.parametrize("window", [1, 2, 16, 33, 64, 100, 127, 128, 129, 511, 512, 5000])
@pytest.mark.parametrize("dim", [64, 256])
def test_sliding_window(window, dim):
    check(Case(NEW + [70], LENS + [700], 8, 4, dim, 13, torch.bfloat16, seed=window), window=window)


@pytest.mark.parametrize("new,length", [(1, 4096), (3, 20011), (257, 20011), (1500, 1500), (2000, 5003)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_long(new, length, dtype):
    check(Case([new, 1], [length, length // 7], 8, 2, 128, 64, dtype, seed=length))


@pytest.mark.parametrize("new,lens,heads,kv,dim,window,dtype", [
    # many items, the last of them small: dealt out whole (a CTA's share is some 90 key tiles and more, the smallest item 2)
    ([2600, 0, 2300, 40], [2600, 50, 2300, 40], 64, 64, 64, 0, torch.float16),
    ([1, 3000, 700], [9, 3100, 700], 96, 32, 128, 0, torch.bfloat16),
    ([2900, 2500], [2900, 2700], 64, 64, 64, 1700, torch.bfloat16),
    # as many, the last of them large: cut into runs
    ([2300, 40, 2600], [2300, 40, 4000], 32, 32, 64, 0, torch.float16)])
def test_prompts_of_many_items(new, lens, heads, kv, dim, window, dtype):
    check(Case(new, lens, heads, kv, dim, 32, dtype, seed=len(new), pad=3), window=window)


def test_long_without_grouped_heads_dim_256():
    check(Case([700, 1, 130], [3000, 2500, 130], 2, 2, 256, 16, torch.bfloat16, seed=1))


def test_many_sequences_and_one_long_one():
    lens = [(i * 37) % 90 for i in range(700)]
    new = [min(n, (i * 11) % 40) for i, n in enumerate(lens)]
    lens[311], new[311] = 9000, 1
    check(Case(new, lens, 4, 2, 64, 16, torch.float16, seed=9))


def test_rows_before_the_first_key_are_zero():
    # fewer keys than new tokens: the first rows stand before the sequence
    for window in (0, 50, 2 ** 31 - 1):
        check(Case([40, 9, 300], [33, 0, 170], 8, 2, 64, 16, torch.float16, seed=2, pad=1), window=window)


@pytest.mark.parametrize("scale", [1.0, -0.7, 0.0])
def test_large_negative_and_no_scores(scale):
    # scores of hundreds: the running maximum carries the whole softmax, and moves all the time
    check(Case(NEW, LENS, 8, 2, 64, 16, torch.float16, seed=4, spread=6.0 if scale else 1.0), scale=scale)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_growing_scores(dtype):
    # every key's score is larger than the one before: the maximum moves with each tile, by little and by much
    for step in (0.02, 0.3):
        c = Case([300], [900], 4, 1, 64, 16, dtype, seed=5)
        c.q[:] = 0
        c.q[..., 0] = 8
        ramp = (torch.arange(900) * step).to(dtype)
        c.keys[0][..., 0] = ramp[:, None]
        c.k[c.pages[0]] = c.keys[0]
        check(c)


def test_flat_tail_behind_one_large_score():
    c = Case([20], [6000], 4, 1, 64, 16, torch.float16, seed=6)
    c.keys[0][:] = 0
    c.keys[0][0, :, 0] = 10.0
    c.q[:] = 0
    c.q[..., 0] = 8.0                     # 10 above the others, in exponents of e
    c.k[c.pages[0]] = c.keys[0]
    check(c)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim,window", [(64, 0), (128, 40), (256, 0), (128, 0)])
def test_what_a_row_does_not_see_does_not_reach_it(dtype, dim, window):
    # infinite and NaN keys and values in the middle of the chunk: rows before them (and with a window those behind
    # it) are those of the same problem with finite ones
    bad = {150: float("nan"), 171: float("inf"), 290: float("-inf")}
    c = Case([200], [330], 8, 2, dim, 16, dtype, seed=7)
    clean = check(c, window=window)
    a = c.gpu()
    for j, x in bad.items():
        at = c.pages[0][0][j], c.pages[0][1][j]
        a["v_cache"][at][:, ::3] = x
        a["k_cache"][at][:, :1] = float("nan") if x != x else 0.0
    out = torch.full_like(clean, MARK)
    g.chunk_attention(**a, window=window, out=out)
    t = torch.arange(130, 330, device=DEV)
    sees = lambda j: (t >= j) & ((t < j + window) if window else (t >= 0))  # noqa: E731
    touched = sees(150) | sees(171) | sees(290)
    assert torch.equal(out[~touched], clean[~touched])
    assert bool(torch.isnan(out[sees(150)]).all())                       # a NaN score leaves nothing of its row
    only = sees(171) & ~sees(150) & ~sees(290)
    assert bool((out[only][..., ::3] == float("inf")).all()) and bool(torch.isfinite(out[only][..., 1::3]).all())
    only = sees(290) & ~sees(150) & ~sees(171)
    assert bool((out[only][..., ::3] == float("-inf")).all()) and bool(torch.isfinite(out[only][..., 1::3]).all())


def test_one_workspace_for_every_shape_and_repeatable():
    ws = g.chunk_attention_workspace(16, 1, 256)
    ws.fill_(255)
    need = ws.numel()
    outs = {}
    for turn in range(3):
        for i, (new, lens, heads, kv, dim) in enumerate([([40], [5000], 16, 1, 64), (NEW, LENS, 8, 2, 64), ([300, 1, 5], [3000, 1, 2500], 8, 8, 128),
                                                         ([3, 60], [2000, 400], 4, 2, 256)]):
            size = g.chunk_attention_workspace_size(heads, kv, dim)
            w = ws if size <= need else g.chunk_attention_workspace(heads, kv, dim)
            out = check(Case(new, lens, heads, kv, dim, 16, torch.float16, seed=i), workspace=w)
            if turn:
                assert torch.equal(out, outs[i])       # the same bits every time
            outs[i] = out


def test_captured_and_replayed_with_other_contents():
    # two graphs that share a workspace, replayed in turn while lengths, rows and tables change under them
    cases = [Case(NEW, LENS, 8, 2, 64, 16, torch.float16, seed=11, pad=7), Case([1, 300, 2], [900, 310, 2], 8, 2, 64, 16, torch.float16, seed=12)]
    ws = g.chunk_attention_workspace(8, 2, 64)
    graphs = []
    for c in cases:
        a = c.gpu()
        out = torch.full((c.tokens, c.heads, c.dim), MARK, dtype=c.dtype, device=DEV)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            g.chunk_attention(**a, out=out, workspace=ws)
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            g.chunk_attention(**a, out=out, workspace=ws)
        graphs.append((graph, a, out))
    for turn in range(3):
        for c, (graph, a, out) in zip(cases, graphs):
            if turn:    # the last sequence that has tokens loses one, its last
                b = max(i for i, m in enumerate(c.new) if m > 1)
                c.new[b] -= 1
                c.lens[b] -= 1
                c.keys[b], c.values[b] = c.keys[b][:-1], c.values[b][:-1]
                keep = torch.ones(c.tokens, dtype=torch.bool)
                keep[sum(c.new[:b + 1])] = False
                c.q = torch.cat([c.q[keep], c.q[:1]])
                c.cu = torch.tensor([0] + list(np.cumsum(c.new)), dtype=torch.int32)
                a["q"].copy_(c.q), a["cu_tokens"].copy_(c.cu)
                a["seq_lens"].copy_(torch.tensor(c.lens, dtype=torch.int32))
            out.fill_(MARK)
            graph.replay()
            torch.cuda.synchronize()
            ref, tol, _, _ = c.ref(c.dim ** -0.5, 0)
            assert bool(((out[:ref.shape[0]].double() - ref).abs() <= tol).all())
            assert bool((out[ref.shape[0]:] == MARK).all())


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_keys_and_values_in_different_layouts_and_shared_heads(dim):
    c = Case(NEW, LENS, 8, 4, dim, 16, torch.float16, seed=8)
    a = c.gpu()
    want = check(c, a=a)
    # values in another order than keys, then with padding between rows
    a["v_cache"] = a["v_cache"].permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    assert torch.equal(check(c, a=a), want)
    wide = torch.full(a["v_cache"].shape[:3] + (dim + 24,), float("nan"), dtype=torch.float16, device=DEV)
    wide[..., :dim] = a["v_cache"]
    a["v_cache"] = wide[..., :dim]
    assert torch.equal(check(c, a=a), want)
    # one head's keys and values for all: strides of zero
    c = Case(NEW, LENS, 8, 1, dim, 16, torch.float16, seed=9)
    want = check(c)
    a = c.gpu()
    for name in ("k_cache", "v_cache"):
        a[name] = a[name].expand(-1, -1, 4, -1)
    out = torch.full((c.tokens, 8, dim), MARK, dtype=torch.float16, device=DEV)
    g.chunk_attention(**a, out=out)
    # (the rows of an item are others, and with them what is joined: the tolerance, not the bits)
    ref, tol, _, _ = c.ref(dim ** -0.5, 0)
    assert bool(((out.double() - ref).abs() <= tol).all()) and bool(torch.isfinite(want).all())


def test_two_calls_at_once():
    cases = [Case([500, 1, 60], [3000, 2000, 60], 16, 4, 128, 16, torch.bfloat16, seed=i) for i in (20, 21)]
    args = [c.gpu() for c in cases]
    want = [check(c, a=a) for c, a in zip(cases, args)]
    streams = [torch.cuda.Stream() for _ in cases]
    spaces = [g.chunk_attention_workspace(16, 4, 128) for _ in cases]
    torch.cuda.synchronize()
    got = []
    for turn in range(10):
        for a, s, w in zip(args, streams, spaces):
            got.append(g.chunk_attention(**a, workspace=w, stream=s))
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        assert torch.equal(out, want[i % 2])


def test_infinite_values_of_keys_that_every_row_sees():
    # far behind the chunk, in tiles that all rows see: infinite where it is, not a number elsewhere never
    c = Case([40], [900], 8, 2, 64, 16, torch.bfloat16, seed=10)
    a = c.gpu()
    clean = check(c, a=a)
    at = c.pages[0][0][300], c.pages[0][1][300]
    a["v_cache"][at][:, 5] = float("inf")
    out = g.chunk_attention(**a)
    assert bool((out[..., 5] == float("inf")).all())
    rest = torch.arange(64, device=DEV) != 5
    assert torch.equal(out[..., rest], clean[..., rest])
    # a score of minus infinity is a key that does not count
    a = c.gpu()
    a["q"][:, :, 0] = 1.0
    c.q[:, :, 0] = 1.0
    a["k_cache"][at][:, 0] = float("-inf")
    out = g.chunk_attention(**a)
    keep = torch.arange(900) != 300
    c.keys[0], c.values[0], c.lens, c.new = c.keys[0][keep], c.values[0][keep], [899], [40]
    ref, tol, _, _ = c.ref(64 ** -0.5, 0)
    assert bool(((out.double() - ref).abs() <= tol).all())


def test_side_stream_and_current_stream_is_another():
    c = Case([100, 1, 30], [140, 900, 30], 8, 2, 64, 16, torch.float16, seed=5)
    a = c.gpu()
    want = g.chunk_attention(**a)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    busy = torch.ones((8192, 8192), dtype=torch.bfloat16, device=DEV)
    for _ in range(8):
        busy @ busy                                   # the current stream is late
    out = g.chunk_attention(**a, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    torch.cuda.synchronize()


def test_cache_past_32_bit_offsets():
    # the last page starts past 2^31 elements: 5 GB of cache, of which a few pages are live
    pages, page, kv, dim = 2 ** 31 // (256 * 2 * 64) + 40, 256, 2, 64
    k = torch.empty((pages, page, kv, dim), dtype=torch.float16, device=DEV)
    v = torch.empty_like(k)
    ids = [pages - 1, 3, pages - 7]
    gen = torch.Generator(device=DEV).manual_seed(1)
    for i in ids:
        k[i].normal_(generator=gen), v[i].normal_(generator=gen)
    n, m = 2 * page + 100, 37
    q = torch.randn((m, 8, dim), device=DEV, generator=gen).half()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    out = g.chunk_attention(q, k, v, i32([ids]), i32([n]), i32([0, m]))
    kk, vv = (torch.cat([t[i] for i in ids])[:n].double() for t in (k, v))
    s = torch.einsum("thgd,nhd->hgtn", q.double().reshape(m, kv, 4, dim), kk) * dim ** -0.5
    at = n - m + torch.arange(m, device=DEV)[:, None]
    p = torch.softmax(s.masked_fill(torch.arange(n, device=DEV)[None] > at, -np.inf), -1)
    ref = torch.einsum("hgtn,nhd->thgd", p, vv).reshape(m, 8, dim)
    A = torch.einsum("hgtn,nhd->thgd", p, vv.abs()).reshape(m, 8, dim)
    tol = 2.0 ** -11 * ref.abs() + (2.0 ** -11 + 2.0 ** -16 * (1 + float(s.abs().max()))) * A + 2.0 ** -20
    assert bool(((out.double() - ref).abs() <= tol).all())


def test_bad_table_entries_lengths_and_rows_are_flagged():
    c = Case([40, 50, 33], [40, 60, 33], 8, 2, 64, 16, torch.float16, seed=6)
    a = c.gpu()
    good = g.chunk_attention(**a)
    a["block_table"][1, 1] = -5                       # keys 16 .. 31 of sequence 1
    out = g.chunk_attention(**a)
    assert g.device_status() == g.DEV_PAGE_RANGE
    assert torch.equal(out[:40], good[:40]) and torch.equal(out[90:], good[90:])
    keep = torch.tensor([j for j in range(60) if not 16 <= j < 32])
    k, v = (t[1][keep].double() for t in (c.keys, c.values))
    s = torch.einsum("thgd,nhd->hgtn", c.q[40:90].double().reshape(50, 2, 4, 64), k) / 8
    s = s.masked_fill(keep[None] > 10 + torch.arange(50)[:, None], -np.inf)
    ref = torch.einsum("hgtn,nhd->thgd", torch.softmax(s, -1), v).reshape(50, 8, 64)
    assert float((out[40:90].double().cpu() - ref).abs().max()) < 0.01
    a = c.gpu()
    a["seq_lens"][0] = -3
    out = g.chunk_attention(**a)
    assert g.device_status() == g.DEV_SEQ_LEN
    assert float(out[:40].abs().max()) == 0.0 and torch.equal(out[40:], good[40:])
    a = c.gpu()
    a["cu_tokens"][3] = 10 ** 9                       # past the rows: cut to them
    out = g.chunk_attention(**a)
    assert g.device_status() == g.DEV_TOKEN_ROWS
    assert torch.equal(out, good)
    a["cu_tokens"].copy_(torch.tensor([-7, 40, 20, 123]))
    g.chunk_attention(**a)
    assert g.device_status() == g.DEV_TOKEN_ROWS


def test_wrong_tensors_are_refused():
    a = Case([4], [9], 8, 2, 64, 16, torch.float16).gpu()
    for kw in (dict(q=a["q"].cpu()), dict(k_cache=a["k_cache"][..., :32]), dict(block_table=a["block_table"][0]),
               dict(cu_tokens=a["cu_tokens"][:1]), dict(q=a["q"].transpose(0, 1)), dict(out=a["q"][:2]),
               dict(v_cache=a["v_cache"][:1])):
        with pytest.raises(ValueError):
            g.chunk_attention(**dict(a, **kw))
    for kw in (dict(q=a["q"].float()), dict(v_cache=a["v_cache"].bfloat16()), dict(seq_lens=a["seq_lens"].long())):
        with pytest.raises(TypeError):
            g.chunk_attention(**dict(a, **kw))
    with pytest.raises(g.GPTQError) as e:
        g.chunk_attention(**a, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    assert e.value.code == -4
