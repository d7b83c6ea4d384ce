"""gptq_rms_norm against the formula in 64 bits.

Tolerance, for u the unit roundoff of an output's type (2^-11, 2^-8, 2^-24): the sum s carries one rounding to fp32,
2^-24 |s|; a sum of n squares, taken by 128 threads and more and joined pairwise, is off by at most (n / 128 + 16)
2^-24 of itself, of which the square root leaves half; root, division and two products add 8 2^-24:
  |out - ref| <= (u + ((n / 128 + 16) / 2 + 10) 2^-24) |ref| + 2^-25 (fp16's smallest step, halved),
  |residual_out - ref| <= (u + 2^-24) |ref| + 2^-25."""
import pytest
import torch

import gptq_bit_weight_gemm_gb300 as g

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
U = {F16: 2.0 ** -11, BF16: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_bit_weight_gemm_gb300 import build as lib_build
    lib_build.build()
    assert torch.cuda.is_available()
    yield
    assert g.device_status() == 0


def make(rows, hidden, dtype, residual, weight, seed=0, pad=0, offset=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def matrix(t, spread):
        wide = torch.randn((rows, hidden + pad + offset), device=DEV, generator=gen) * spread
        return wide.to(t)[:, offset:offset + hidden]
    x = matrix(dtype, 1.0)
    r = None if residual is None else matrix(residual, 3.0)
    w = None if weight is None else (1 + 0.3 * torch.randn(hidden, device=DEV, generator=gen)).to(weight)
    return x, r, w


def check(x, r, w, eps=1e-6, dtype=None, **kw):
    s = x.double() if r is None else x.double() + r.double()
    ref = s * torch.rsqrt(s.square().mean(-1, keepdim=True) + eps)
    ref = ref if w is None else ref * w.double()
    r0 = None if r is None else r.clone()
    out = g.rms_norm(x, w, residual=r, eps=eps, dtype=dtype, **kw)
    assert out.dtype == (dtype or x.dtype)
    n = x.shape[1]
    err = (out.double() - ref).abs()
    tol = (U[out.dtype] + ((n / 128 + 16) / 2 + 10) * 2.0 ** -24) * ref.abs() + 2.0 ** -25
    assert bool((err <= tol).all()), "max error %g" % float(err.max())
    if r is not None:
        got = kw.get("residual_out", r)
        err = (got.double() - s).abs()
        assert bool((err <= (U[r.dtype] + 2.0 ** -24) * s.abs() + 2.0 ** -25).all())
        if got is not r:
            assert torch.equal(r, r0)
    return out


@pytest.mark.parametrize("rows,hidden", [(1, 1), (1, 8), (3, 7), (2, 64), (5, 100), (1, 4096), (17, 4096), (300, 1000), (3, 1001), (4, 5120),
                                         (2, 8192), (2, 16384), (1, 20000), (1, 33333), (2, 65536), (1, 262145), (4000, 256)])
@pytest.mark.parametrize("dtype,residual,weight", [(BF16, None, BF16), (F16, F16, F16), (BF16, F32, BF16), (F32, F32, None), (BF16, BF16, F32)])
def test_sizes_and_types(rows, hidden, dtype, residual, weight):
    check(*make(rows, hidden, dtype, residual, weight, seed=hidden))


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("out", [F16, BF16, F32])
@pytest.mark.parametrize("residual", [None, F16, F32])
def test_every_pair_of_types(dtype, out, residual):
    for hidden in (1024, 999):
        check(*make(9, hidden, dtype, residual, BF16, seed=3), dtype=out)


@pytest.mark.parametrize("pad,offset", [(8, 0), (8, 8), (3, 0), (0, 1), (5, 2)])
def test_strided_rows_and_odd_alignment(pad, offset):
    x, r, w = make(33, 512, BF16, F32, BF16, seed=4, pad=pad, offset=offset)
    wide = torch.full((33, 700), 7.0, dtype=BF16, device=DEV)
    out = wide[:, 3:515]
    check(x, r, w, out=out)
    assert bool((wide[:, :3] == 7).all()) and bool((wide[:, 515:] == 7).all())


def test_in_place_and_apart():
    for hidden in (2048, 77):
        x, r, w = make(20, hidden, BF16, BF16, BF16, seed=5)
        want = check(x, r.clone(), w).clone()
        check(x, r, w, residual_out=torch.full_like(r, float("nan")))
        r2, x2 = r.clone(), x.clone()
        got = g.rms_norm(x2, w, residual=r2, out=x2)
        assert got.data_ptr() == x2.data_ptr() and torch.equal(got, want)


def test_large_small_and_empty_rows():
    x, r, w = make(6, 4096, F32, None, None, seed=6)
    x[0] = 0.0
    x[1] *= 1e15
    x[2] *= 1e-15
    check(x, None, None)
    check(x, None, None, eps=1.0)
    b = torch.full((2, 300), 60000.0, dtype=F16, device=DEV)
    check(b, None, None)
    assert bool((g.rms_norm(torch.zeros((3, 40), device=DEV), eps=0.0).isnan()).all())   # 0 / 0
    assert g.rms_norm(torch.zeros((0, 40), device=DEV)).shape == (0, 40)


def test_a_bad_row_stays_alone():
    x, r, w = make(8, 4096, BF16, BF16, BF16, seed=7)
    want = g.rms_norm(x, w, residual=r.clone())
    x[3, 100] = float("nan")
    x[5, 7] = float("inf")
    got = g.rms_norm(x, w, residual=r.clone())
    good = torch.tensor([0, 1, 2, 4, 6, 7], device=DEV)
    assert torch.equal(got[good], want[good]) and bool(got[3].isnan().all()) and bool(got[5, 7].isnan())


def test_past_32_bit_offsets():
    # rows whose last starts past 2^31 elements
    hidden, stride = 4096, 1 << 22
    store = torch.empty(600 * stride, dtype=BF16, device=DEV)
    x = store.as_strided((600, hidden), (stride, 1))
    x.copy_(torch.randn((600, hidden), device=DEV, generator=torch.Generator(device=DEV).manual_seed(8)))
    check(x, None, None)


def test_captured_and_on_another_stream():
    x, r, w = make(64, 4096, BF16, F32, BF16, seed=9)
    r_out = torch.empty_like(r)
    want = g.rms_norm(x, w, residual=r, residual_out=r_out)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = g.rms_norm(x, w, residual=r, residual_out=r_out, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = g.rms_norm(x, w, residual=r, residual_out=r_out)
    x.copy_(-x)
    r.copy_(-r)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, -want)


def test_wrong_tensors_are_refused():
    x, r, w = make(4, 64, BF16, BF16, BF16)
    for kw in (dict(x=x.cpu()), dict(weight=w[:32]), dict(residual=r[:2]), dict(x=x.t().contiguous().t()), dict(residual_out=r, residual=None),
               dict(out=torch.empty((4, 32), dtype=BF16, device=DEV))):
        with pytest.raises(ValueError):
            g.rms_norm(**dict(dict(x=x, weight=w, residual=r), **kw))
    for kw in (dict(x=x.long()), dict(weight=w.double()), dict(residual=r.double()), dict(dtype=torch.int8)):
        with pytest.raises(TypeError):
            g.rms_norm(**dict(dict(x=x, weight=w, residual=r), **kw))
    with pytest.raises(TypeError):
        g.rms_norm(x, w, residual=r, residual_out=torch.empty((4, 64), device=DEV))
    with pytest.raises(g.GPTQError) as e:
        g.rms_norm(x, w, residual=r, residual_out=x)
    assert e.value.code == -1
