"""gptq_chunk_attention at edges that the sizes and masks do not reach: infinite values under probabilities that are
nothing in 16 bits, and lengths and rows that do not fit.  A probability is above 0 in the definition, however
small: an infinite value of a key that a row sees is infinite in the row, wherever the key lies."""
import pytest
import torch

import gptq_bit_weight_gemm_gb300 as g
from test_gpu_chunk_attention import DEV, MARK, Case, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_bit_weight_gemm_gb300 import build as lib_build
    lib_build.build()
    assert torch.cuda.is_available()
    yield
    assert g.device_status() == 0


def one_large_score(new, lens, heads, kv, dim, page, dtype, gap):
    """The first key of each sequence scores `gap` above all others, which score 0."""
    c = Case(new, lens, heads, kv, dim, page, dtype, seed=dim + int(gap), pad=1)
    c.q[:] = 0
    c.q[..., 0] = 8
    for b in range(len(lens)):
        c.keys[b][:] = 0
        c.keys[b][0, :, 0] = gap
        c.k[c.pages[b]] = c.keys[b]
    return c


# e^-40 of the largest is nothing in fp16, e^-100 in fp32's normal numbers, e^-300 in fp32
@pytest.mark.parametrize("gap", [10.0, 40.0, 100.0, 300.0])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("new,lens,heads,kv,dim,page", [
    ([40], [900], 4, 1, 64, 16), ([9, 300], [6000, 2000], 8, 2, 128, 16), ([1, 70], [1500, 900], 2, 2, 256, 16),
    ([33], [1000], 6, 2, 80, 13), ([4] * 160, [450] * 160, 8, 8, 72, 16)])
def test_infinite_values_of_faint_keys_stay_infinite(gap, dtype, new, lens, heads, kv, dim, page):
    c = one_large_score(new, lens, heads, kv, dim, page, dtype, gap)
    a = c.gpu()
    scale = 0.125                         # of 8: the first key's score is its value
    clean = check(c, scale=scale, a=a)
    inf = float("inf")
    for b in range(len(lens)):
        at = lambda j: (c.pages[b][0][j], c.pages[b][1][j])  # noqa: E731,B023
        for j, d, x in ((300, 5, inf), (150, 9, -inf), (300, 11, inf), (140, 11, -inf), (301, 13, float("nan")), (0, 14, inf),
                        (200, dim - 1, inf)):
            a["v_cache"][at(j)][:, d] = x
    out = torch.full_like(clean, MARK)
    g.chunk_attention(**a, scale=scale, out=out)
    rows = sum(new)
    for d, want in ((5, inf), (9, -inf), (14, inf), (dim - 1, inf)):
        assert bool((out[:rows, :, d] == want).all()), d
    assert bool(out[:rows, :, 11].isnan().all()) and bool(out[:rows, :, 13].isnan().all())
    rest = torch.ones(dim, dtype=torch.bool, device=DEV)
    rest[[5, 9, 11, 13, 14, dim - 1]] = False
    assert torch.equal(out[..., rest], clean[..., rest]) and bool((out[rows:] == MARK).all())


def test_rows_of_a_nan_score_and_finite_sums_beside_infinite_ones():
    # one row's query is not a number: all of its results are, and the rows beside it keep theirs
    c = one_large_score([64], [700], 4, 1, 64, 16, torch.float16, 40.0)
    a = c.gpu()
    a["q"][7, 2] = float("nan")
    a["v_cache"][c.pages[0][0][200], c.pages[0][1][200]][:, 3] = float("inf")
    out = g.chunk_attention(**a, scale=0.125)
    assert bool(out[7, 2].isnan().all())
    live = torch.ones((65, 4), dtype=torch.bool, device=DEV)
    live[7, 2] = live[64] = False
    assert bool((out[live][:, 3] == float("inf")).all())
    rest = torch.arange(64, device=DEV) != 3
    assert bool(torch.isfinite(out[live][:, rest]).all())


def test_a_length_past_the_table_is_cut_to_it():
    c = Case([40, 33], [48, 33], 8, 2, 64, 16, torch.float16, seed=21, pad=2)
    a = c.gpu()
    a["block_table"] = a["block_table"][:, :3].contiguous()          # 48 keys
    clean = check(c, a=a)
    for length in (49, 1000, 2 ** 31 - 1):
        a["seq_lens"][0] = length
        assert torch.equal(check(c, a=a), clean)
        assert g.device_status() == g.DEV_SEQ_LEN


def test_rows_that_decrease_or_lie_outside():
    c = Case([40, 50, 33], [40, 60, 33], 8, 2, 64, 16, torch.float16, seed=6, pad=5)
    a = c.gpu()
    check(c, a=a)
    ref, tol, _, _ = c.ref(c.dim ** -0.5, 0)

    def rows(cu):
        a["cu_tokens"].copy_(torch.tensor(cu))
        out = torch.full((c.tokens, 8, 64), MARK, dtype=torch.float16, device=DEV)
        g.chunk_attention(**a, out=out)
        return out, lambda x, y: bool(((out[x:y].double() - ref[x:y]).abs() <= tol[x:y]).all())
    # the first sequence is cut to its rows from 0 on, the second has none, the third gets 103 rows for 33 keys: 20 .. 39 are
    # the first's too, 40 .. 89 stand before its first key
    out, right = rows([-7, 40, 20, 123])
    assert g.device_status() == g.DEV_TOKEN_ROWS
    assert right(0, 20) and right(90, 123)
    twice = (out[20:40].double() - ref[20:40]).abs() <= tol[20:40]
    assert bool((twice | (out[20:40] == 0)).all())
    assert bool((out[40:90] == 0).all()) and bool((out[123:] == MARK).all())
    # no rows but the middle sequence's
    out, right = rows([40, 40, 90, 90])
    assert g.device_status() == 0
    assert right(40, 90) and bool((out[:40] == MARK).all()) and bool((out[90:] == MARK).all())
    # all of them outside
    for cu in ([-9, -8, -2, -1], [500, 600, 700, 800]):
        out, _ = rows(cu)
        assert g.device_status() == g.DEV_TOKEN_ROWS
        assert bool((out == MARK).all())
