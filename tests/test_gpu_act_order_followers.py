"""What follows an act-order gptq_gemm on its stream sees the whole product.

The call's last launch is the per-row kernel, which has nothing to do when the rows could be sorted.  The
next call's kernels start as programmatic dependents of it: sampling from the product (an act-order
head's logits), attention with it as the new token's value, a second GEMM on it.  Each pair is issued
back to back many times, against the same calls with a synchronisation between them."""
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


def act_order(K, N, bits, seed, equal=True):
    """A random act-order checkpoint; equal: groups of the same size (the rows can be sorted)."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    words = lambda *s: torch.randint(-2 ** 31, 2 ** 31, s, dtype=torch.int64, device=DEV, generator=gen).to(torch.int32)  # noqa: E731
    G = K // 128
    g_idx = np.random.default_rng(seed).permutation(K) // 128
    if not equal:
        g_idx[0] = (g_idx[0] + 1) % G
    scales = (0.01 * (0.5 + torch.rand((G, N), device=DEV, generator=gen))).half()
    return words(K * bits // 32, N), words(G, N * bits // 32), scales, torch.from_numpy(g_idx.astype(np.int32)).to(DEV)


@pytest.mark.parametrize("equal", [True, False])
@pytest.mark.parametrize("M", [1, 7, 32])
@pytest.mark.parametrize("bits", [3, 4])
def test_a_follower_reads_the_whole_product(bits, M, equal):
    K, N = 4096, 16384
    w = act_order(K, N, bits, seed=bits * 10 + M, equal=equal)
    heads, dim, n = 128, 128, 40
    gen = torch.Generator(device=DEV).manual_seed(M)
    cache = [torch.randn((M * 3, 16, heads, dim), device=DEV, generator=gen).half() for _ in range(2)]
    table = torch.arange(M * 3, dtype=torch.int32, device=DEV).view(M, 3)
    lens = torch.full((M,), n, dtype=torch.int32, device=DEV)
    q, k_new = (torch.randn((M, heads, dim), device=DEV, generator=gen).half() for _ in range(2))
    u = torch.rand(M, device=DEV, generator=gen)
    second = g.quantize_rtn(torch.randn((N, 512), device=DEV, generator=gen) * N ** -0.5, bits=4, group=128)
    ws = torch.empty(g.act_order_workspace_size(M, K, N, bits, 128), dtype=torch.uint8, device=DEV)
    attention_ws = g.paged_attention_workspace(heads, heads, dim)
    out = torch.empty((M, N), dtype=torch.float16, device=DEV)

    def followers(logits):
        yield lambda: g.sample(logits, u)
        yield lambda: (g.paged_attention(q, *cache, table, lens, k_new=k_new, v_new=logits.view(M, heads, dim), workspace=attention_ws),)
        yield lambda: (g.gemm(logits, *second, bits=4, group=128),)

    inputs = [torch.randn((M, K), device=DEV, generator=gen).half() for _ in range(4)]
    for follow in followers(out):
        want = []
        for A in inputs:
            g.gemm(A, *w, bits=bits, group=128, out=out, workspace=ws)
            torch.cuda.synchronize()
            want.append([t.clone() for t in follow()])
            torch.cuda.synchronize()
        for turn in range(6):
            got = []
            for A in inputs:
                g.gemm(A, *w, bits=bits, group=128, out=out, workspace=ws)
                got.append([t.clone() for t in follow()])
            torch.cuda.synchronize()
            for a, b in zip(want, got):
                assert all(torch.equal(x, y) for x, y in zip(a, b))
