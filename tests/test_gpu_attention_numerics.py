"""gptq_paged_attention's probabilities: they reach the product with v in more bits than the result has.

The error's 2-norm against 64 bits is that of rounding the exact result once, r, within a tenth.  What
else there is: scores as fp32 sums, off by some 2^-21 of |s| < 8, and probabilities of at least 15
significant bits (2^-16): against r = 2^-9.2 (bf16) and 2^-12.2 (fp16) the sum of squares grows by less
than 2^-8."""
import numpy as np
import pytest
import torch

import gptq_bit_weight_gemm_gb300 as g
from test_gpu_paged_attention import Case, LENS, check

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_bit_weight_gemm_gb300 import build as lib_build
    lib_build.build()
    assert torch.cuda.is_available()
    yield
    assert g.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads,kv,dim", [(8, 2, 64), (8, 8, 128), (32, 8, 128), (16, 1, 96), (24, 1, 128), (40, 1, 64), (4, 4, 256),
                                          (12, 1, 256)])
def test_only_the_output_is_rounded_to_16_bits(dtype, heads, kv, dim):
    c = Case(LENS + [3000], heads, kv, dim, 16, dtype, seed=dim + heads)
    out = check(c).double().cpu()
    ref = c.ref(dim ** -0.5, 0)[0]
    own = float((ref.to(dtype).double() - ref).norm() / ref.norm())
    err = float((out - ref).norm() / ref.norm())
    assert err <= 1.1 * own, (err, own)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("group", [1, 12])
@pytest.mark.parametrize("halvings", [12, 16, 20, 23.5, 25.5, 28])
def test_a_peak_over_a_flat_tail(dtype, group, halvings):
    """One key of probability near 1 and value 0 before thousands of equal ones with value 1: the result
    is the tail's mass, each of whose terms is 2^-halvings of the peak's."""
    B, kv, n, dim, page = 48, 8, 4001, 64, 32
    pages = -(-n // page)
    k = torch.zeros((pages, page, kv, dim), dtype=dtype, device=DEV)
    v = torch.ones_like(k)
    q = torch.zeros((B, kv * group, dim), dtype=dtype, device=DEV)
    q[:, :, 0] = 4.0
    k[0, 0, :, 0] = halvings * np.log(2.0) / 4.0
    v[0, 0] = 0.0
    table = torch.arange(pages, dtype=torch.int32, device=DEV).repeat(B, 1)
    out = g.paged_attention(q, k, v, table, torch.full((B,), n, dtype=torch.int32, device=DEV), scale=1.0)
    s = float(k[0, 0, 0, 0]) * 4.0
    ref = (n - 1) * np.exp(-s) / (1.0 + (n - 1) * np.exp(-s))
    # the tolerance of the attention tests: A = ref, as all values that count are 1
    u = 2.0 ** (-11 if dtype == torch.float16 else -8)
    tol = (2 * u + 2.0 ** -16 * (1 + s)) * ref + 2.0 ** -24
    assert float((out.double() - ref).abs().max()) <= tol, (float(out.min()), float(out.max()), ref)


def test_a_cut_length_appends_nothing():
    """A length past the block table is cut to it and flagged; the new token then has no slot: neither the
    cache nor the result takes it."""
    c = Case([30, 64, 48], 8, 2, 64, 16, torch.float16, seed=11, width=4)
    a = c.gpu()
    gen = torch.Generator().manual_seed(1)
    new = [torch.randn((3, 2, 64), generator=gen).half().to(DEV) for _ in range(2)]
    a["seq_lens"][1] = 65                             # four pages of 16 hold 64 keys
    keys, values = a["k_cache"].clone(), a["v_cache"].clone()
    out = g.paged_attention(**dict(a, k_new=new[0], v_new=new[1]))
    assert g.device_status() == g.DEV_SEQ_LEN
    ref, tol, _, _ = c.ref(64 ** -0.5, 0)             # sequence 1: its 64 cached keys
    assert bool(((out[1].double().cpu() - ref[1]).abs() <= tol[1]).all())
    for cache, old, fresh in ((a["k_cache"], keys, new[0]), (a["v_cache"], values, new[1])):
        for b, n in ((0, 30), (2, 48)):               # the others' new tokens are in their slots
            old[int(c.table[b, (n - 1) // 16]), (n - 1) % 16] = fresh[b]
        assert torch.equal(cache.view(torch.int16), old.view(torch.int16))


def test_strides_of_dimensions_of_one():
    """A dimension of one is never stepped over: its stride may be anything."""
    gen = torch.Generator(device=DEV).manual_seed(3)
    q = torch.randn((1, 4, 64), generator=gen, device=DEV).half()
    k, v = (torch.randn((3, 16, 1, 64), generator=gen, device=DEV).half() for _ in range(2))
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([41], dtype=torch.int32, device=DEV)
    want = g.paged_attention(q, k, v, table, lens)
    odd = lambda t: torch.as_strided(t, t.shape, (16 * 64, 64, 3, 1))  # noqa: E731
    assert torch.equal(g.paged_attention(q, odd(k), odd(v), table, lens), want)
    one = [t[2:3].contiguous() for t in (k, v)]       # one page of one head
    odd = [torch.as_strided(t, t.shape, (5, 64, 7, 1)) for t in one]
    args = (torch.zeros((1, 1), dtype=torch.int32, device=DEV), torch.tensor([13], dtype=torch.int32, device=DEV))
    assert torch.equal(g.paged_attention(q, *odd, *args), g.paged_attention(q, *one, *args))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("group", [1, 4, 12])
def test_infinite_values_stay_infinite(dtype, group):
    """An infinite value of a live key makes its dimension of the result infinite, with its sign, whatever the
    key's probability (here from 2^-12 of the largest to 1); the other dimensions do not see it.  NaN
    stays NaN, and two signs give NaN."""
    n, kv, dim = 200, 2, 64
    gen = torch.Generator(device=DEV).manual_seed(group)
    q = torch.randn((1, kv * group, dim), generator=gen, device=DEV).to(dtype)
    k = torch.randn((13, 16, kv, dim), generator=gen, device=DEV).to(dtype)
    v = torch.randn((13, 16, kv, dim), generator=gen, device=DEV).to(dtype)
    args = (torch.arange(13, dtype=torch.int32, device=DEV)[None], torch.tensor([n], dtype=torch.int32, device=DEV))
    plain = g.paged_attention(q, k, v, *args)
    inf = float("inf")
    flat_v = v.view(-1, kv, dim)
    flat_v[5, :, 3], flat_v[77, :, 9], flat_v[199, :, 17] = inf, -inf, inf
    flat_v[20, :, 30], flat_v[21, :, 30], flat_v[100, :, 40] = inf, -inf, float("nan")
    out = g.paged_attention(q, k, v, *args)[0].float()
    for d, want in ((3, inf), (9, -inf), (17, inf)):
        assert bool((out[:, d] == want).all()), (d, out[:, d])
    assert bool(out[:, 30].isnan().all()) and bool(out[:, 40].isnan().all())
    rest = [d for d in range(dim) if d not in (3, 9, 17, 30, 40)]
    assert torch.equal(out[:, rest], plain[0].float()[:, rest])
