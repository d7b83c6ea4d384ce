"""The failure path of chunk attention's bounded waits, on valid calls whose waits give up too early: the call returns, the
status word says so, nothing outside the sequences' rows is written, and the next ordinary call is right.  Waits that
give up at different times leave different work in flight (queries, tiles of keys and values, products); all of
it is waited for before the kernel ends."""
import ctypes

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


@pytest.fixture
def limit():
    hook = g.lib().gptq_selftest_chunk_attention_wait
    hook.restype, hook.argtypes = ctypes.c_int, [ctypes.c_uint]

    def set_to(ns):
        assert hook(ns) == 0
    yield set_to
    set_to(0)


# boxes, odd pages (cp.async), one accumulator, values looked over at the diagonal and in a window
@pytest.mark.parametrize("heads,kv,dim,page,window", [(8, 2, 64, 16, 0), (8, 8, 128, 13, 0), (4, 4, 256, 64, 0), (8, 1, 128, 32, 150)])
def test_waits_that_give_up_leave_a_usable_context(limit, heads, kv, dim, page, window):
    c = Case([40, 300, 1], [600, 1500, 900], heads, kv, dim, page, torch.bfloat16, seed=dim, pad=3)
    a = c.gpu()
    ws = g.chunk_attention_workspace(heads, kv, dim)
    ws.zero_()
    want = check(c, a=a, window=window, workspace=ws)
    gave_up = 0
    for ns in (1, 1500, 4000):
        out = torch.full_like(want, MARK)
        limit(ns)
        g.chunk_attention(**a, window=window, out=out, workspace=ws)
        limit(0)
        status = g.device_status()
        assert status in (0, g.DEV_TIMEOUT)
        gave_up += status != 0
        assert status or torch.equal(out, want)
        assert bool((out[-3:] == MARK).all())
        assert torch.equal(check(c, a=a, window=window, workspace=ws), want)
        assert g.device_status() == 0
    assert gave_up                                     # a load takes longer than 1 ns
