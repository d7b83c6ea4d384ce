"""stream= given while another stream is current: what a call makes for itself (workspaces, their zeros,
outputs) belongs to the stream that it runs on.

Each call is made three ways against the same call on the current stream: with the current stream busy
for milliseconds (a fill queued there would come late), with the call's own stream busy and the current
one overwriting whatever memory it can get (a workspace released too early would be hit), and with
fills of just-released memory still queued on the current stream (an output placed there would be
hit)."""
import pytest
import torch

import gptq_bit_weight_gemm_gb300 as g
from test_gpu_moe import make
from test_gpu_paged_attention import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"
SIZES = (512, 4096, 65536, 1 << 20, 3 << 20, 9 << 20, 20 << 20)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_bit_weight_gemm_gb300 import build as lib_build
    lib_build.build()
    assert torch.cuda.is_available()
    yield
    assert g.device_status() == 0


def attention():
    a = Case([5000, 1, 3000], 8, 2, 64, 16, torch.float16, seed=1).gpu()
    return lambda stream: [g.paged_attention(**a, stream=stream)]


def experts():
    a = make(9, 16, 4, 512, 512, 4, 64, g.V2, torch.float16, seed=2)[0]
    return lambda stream: list(g.moe_layer(**a, return_routing=True, stream=stream))


def sampling():
    x = torch.randn((5, 30000), generator=torch.Generator().manual_seed(3)).to(DEV)
    u = torch.rand(5, generator=torch.Generator().manual_seed(4)).to(DEV)
    p = torch.full((5,), 0.9, device=DEV)
    return lambda stream: list(g.sample(x, u, top_p=p, stream=stream))


def gemm():
    gen = torch.Generator(device=DEV).manual_seed(5)
    W = torch.randn((1024, 2048), device=DEV, generator=gen)
    w = g.quantize_rtn(W, bits=4, group=128)
    A = torch.randn((300, 1024), device=DEV, generator=gen).bfloat16()
    return lambda stream: [g.gemm(A, *w, bits=4, group=128, stream=stream)] + list(g.quantize_rtn(W, bits=4, group=128, stream=stream))


def busy():
    a = torch.ones((8192, 8192), dtype=torch.bfloat16, device=DEV)
    for _ in range(12):
        a @ a


def overwrite():
    """Fills of released memory of every size on the current stream, the memory released again."""
    held = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in SIZES for _ in range(3)]
    del held


@pytest.mark.parametrize("make_call", [attention, experts, sampling, gemm])
@pytest.mark.parametrize("way", ["current busy", "own stream busy", "fills queued"])
def test_the_current_stream_is_another(make_call, way):
    call = make_call()
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (torch.cuda.current_stream(), s):    # memory that is not zero to begin with, in both pools
        with torch.cuda.stream(stream):
            overwrite()
    torch.cuda.synchronize()
    if way == "own stream busy":
        with torch.cuda.stream(s):
            busy()
    else:
        busy()
    if way == "fills queued":
        overwrite()
    got = call(s)
    if way == "own stream busy":
        overwrite()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    s.wait_stream(torch.cuda.current_stream())
