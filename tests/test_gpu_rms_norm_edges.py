"""gptq_rms_norm on tensors whose rows start on 16 bytes, but at other places of a run of 8 elements than one another's:
fp32 rows 16 and not 32 bytes aligned beside 16-bit rows.  Tolerances as in test_gpu_rms_norm.py."""
import pytest
import torch

import gptq_bit_weight_gemm_gb300 as g
from test_gpu_rms_norm import BF16, DEV, F16, F32, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_bit_weight_gemm_gb300 import build as lib_build
    lib_build.build()
    assert torch.cuda.is_available()
    yield
    assert g.device_status() == 0


def at(rows, hidden, dtype, place, pad, gen):
    """[rows, hidden] that starts `place` elements behind a 32-byte boundary, rows hidden + pad elements apart."""
    store = torch.randn(rows * (hidden + pad) + 32, device=DEV, generator=gen).to(dtype)
    return store[place:].as_strided((rows, hidden), (hidden + pad, 1))


# (x type and place, residual type and place, out type and place, weight type and place, pads of x, residual, out)
CASES = [
    ((BF16, 0), (F32, 4), (BF16, 0), (BF16, 0), (0, 0, 0)),
    ((BF16, 0), (F32, 0), (BF16, 0), (F32, 4), (8, 4, 16)),
    ((F32, 4), None, (F16, 0), None, (4, 0, 0)),
    ((F32, 4), (F32, 0), (F32, 4), (F32, 4), (4, 12, 0)),
    ((F32, 0), (BF16, 0), (F32, 4), (BF16, 0), (0, 8, 4)),
    ((BF16, 3), (F32, 7), (BF16, 3), (BF16, 3), (5, 1, 5)),
    ((BF16, 3), (F32, 6), (BF16, 3), (BF16, 0), (5, 1, 5)),
    ((F16, 8), (F32, 4), (F16, 1), (F16, 5), (8, 4, 8)),
    ((F32, 5), (F32, 1), (F32, 5), (F32, 1), (3, 7, 3)),
    ((F32, 6), None, (F32, 3), None, (1, 0, 2)),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("rows,hidden", [(1, 64), (5, 1000), (3, 1003), (2, 4096), (33, 250), (2, 40000)])
def test_places_and_strides_of_each_tensor(case, rows, hidden):
    x, r, o, w, pads = CASES[case]
    gen = torch.Generator(device=DEV).manual_seed(case)
    xt = at(rows, hidden, *x, pads[0], gen)
    rt = None if r is None else at(rows, hidden, *r, pads[1], gen)
    ot = at(rows, hidden, *o, pads[2], gen)
    wt = None if w is None else at(1, hidden, *w, 0, gen)[0]
    kw = {} if r is None else dict(residual_out=at(rows, hidden, *r, pads[1], gen))
    check(xt, rt, wt, dtype=o[0], out=ot, **kw)
    if rt is not None:
        check(xt, rt, wt, dtype=o[0])              # the residual in place
    if x[0] == o[0]:
        want = check(xt, rt if rt is None else rt.clone(), wt)
        r2 = None if rt is None else rt.clone()
        got = g.rms_norm(xt, wt, residual=r2, out=xt)
        tol = 2 * torch.finfo(want.dtype).eps
        # (the sum's order goes by the places)
        assert bool(((got.double() - want.double()).abs() <= tol * want.double().abs() + 2.0 ** -24).all())
