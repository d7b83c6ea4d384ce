"""gptq_moe where the arithmetic, not the layout, decides: groups whose codes equal their zero under
large scales, activations with outlier channels, and the accuracy of the whole layer against 64 bits.

The bounds of `test_gpu_moe.check` are proportional to sum |x w|, which is 0 for a column of such groups:
what the layer returns there has to be 0 up to fp16's smallest step, whatever the scale and the
activations, as gptq_gemm_grouped does."""
import numpy as np
import pytest
import torch

import gptq_bit_weight_gemm_gb300 as g
import oracle
from test_gpu_moe import check

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_bit_weight_gemm_gb300 import build as lib_build
    lib_build.build()
    assert torch.cuda.is_available()
    yield
    assert g.device_status() == 0


def packed(rng, E, K, N, bits, group, fmt, scale, columns):
    """Random codes, zeros and scales, packed by the oracle; every code of `columns` equals its group's
    zero, under a scale of 2 to 16.  (packed tensors on the GPU, fp64 weights [E, K, N])"""
    G = 1 if group == -1 else K // group
    top = (1 << bits) - 1
    off = 1 if fmt == g.V1 else 0
    qw, qz, sc, W = [], [], [], np.empty((E, K, N))
    for e in range(E):
        q = rng.integers(0, top + 1, (K, N)).astype(np.uint8)
        z = rng.integers(0, top + 1, (G, N)).astype(np.int32)
        s = (scale * (0.5 + rng.random((G, N)))).astype(np.float16)
        z[:, columns] = np.minimum(z[:, columns], top - off)       # a runtime zero of 2^bits is no code
        q[:, columns] = np.repeat(z[:, columns] + off, K // G, 0)
        s[:, columns] = (2.0 + 14.0 * rng.random((G, len(columns)))).astype(np.float16)
        qw.append(oracle.pack_k(q, bits))
        qz.append(oracle.pack_n(z, bits))
        sc.append(s)
        W[e] = (q.astype(np.float64) - np.repeat(z + off, K // G, 0)) * np.repeat(s.astype(np.float64), K // G, 0)
    return tuple(torch.from_numpy(np.stack(t)).to(DEV) for t in (qw, qz, sc)), torch.from_numpy(W).to(DEV)


def outliers(rng, T, H, dtype, most):
    """N(0, 1) with 1 % of the channels scaled by 100 to `most`."""
    x = rng.standard_normal((T, H))
    at = rng.choice(H, max(1, H // 100), replace=False)
    x[:, at] *= rng.uniform(100.0, most, len(at))
    return torch.from_numpy(x).to(dtype).to(DEV)


DEAD = [0, 1, 33, 100, 127, 128, 200, 255]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("fmt", [g.V1, g.V2])
@pytest.mark.parametrize("bits,group", [(2, 64), (3, 128), (4, 32), (4, 128), (4, -1), (8, 32), (8, 128), (8, -1)])
@pytest.mark.parametrize("tokens", [1, 6, 20])
def test_groups_of_zeros_stay_zero(bits, group, fmt, dtype, tokens):
    """Dead output columns (down), dead gate columns and dead up columns, in one layer."""
    rng = np.random.default_rng(100 * bits + tokens)
    E, topk, H, I = 4, 2, 1024, 256
    # the live weights are small enough for fp16 outputs: gate and up of order 10, h of order 100
    up, Wu = packed(rng, E, H, 2 * I, bits, group, fmt, 0.02 / 2 ** bits, DEAD + [I + n for n in (2, 64, 129)])
    down, Wd = packed(rng, E, I, H, bits, group, fmt, 0.02 / 2 ** bits, DEAD + [513, 1023])
    router = torch.from_numpy(rng.standard_normal((E, H)) * 0.002).to(dtype).to(DEV)
    a = dict(x=outliers(rng, tokens, H, dtype, 1000.0), router=router, up=up, down=down, topk=topk, bits=bits, group=group, fmt=fmt)
    out = check(a, Wu, Wd)
    assert float(out[:, DEAD + [513, 1023]].abs().max()) <= 2.0 ** -24
    assert float(out.abs().max()) > 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens,E,topk,H,I,bits,group", [(1, 4, 2, 1024, 512, 4, 128), (3, 8, 2, 2048, 384, 4, -1), (8, 8, 2, 1024, 320, 8, 32),
                                                          (16, 16, 4, 1024, 512, 8, 128), (32, 4, 2, 512, 1024, 4, 64),
                                                          (32, 8, 2, 1024, 512, 3, 128), (5, 6, 1, 1024, 512, 2, 64)])
def test_only_the_output_is_rounded_to_16_bits(tokens, E, topk, H, I, bits, group, dtype):
    """The 2-norm of the error against 64 bits is that of rounding the exact result once, r, within a
    tenth.  What else there is: fp32 sums of up to 2048 products, 2^-24 each step of a sum that grows as a
    random walk, so some 2^-22 of sum |h w|, which for random signs is sqrt(I) < 32 times the result
    (2^-17), and an inner activation of at least 20 significant bits (2^-21 each): with r = 2^-12.2 in
    fp16 the sum of squares grows by 2^-9."""
    rng = np.random.default_rng(tokens + H)
    up, Wu = packed(rng, E, H, 2 * I, bits, group, g.V2, 0.1 / 2 ** bits, [])
    down, Wd = packed(rng, E, I, H, bits, group, g.V2, 0.1 / 2 ** bits, [])
    x = torch.from_numpy(rng.standard_normal((tokens, H))).to(dtype).to(DEV)
    router = torch.from_numpy(rng.standard_normal((E, H)) * 2 / H ** 0.5).to(dtype).to(DEV)
    out, ids, w = g.moe_layer(x, router, up, down, topk=topk, bits=bits, group=group, return_routing=True)
    p = torch.softmax(x.double() @ router.double().T, -1).gather(1, ids.long())
    p = p / p.sum(-1, keepdim=True)
    ref = torch.zeros((tokens, H), dtype=torch.float64, device=DEV)
    for t in range(tokens):
        for j in range(topk):
            e = int(ids[t, j])
            y = x[t].double() @ Wu[e]
            ref[t] += p[t, j] * ((torch.nn.functional.silu(y[:I]) * y[I:]) @ Wd[e])
    own = float((ref.to(dtype).double() - ref).norm() / ref.norm())
    err = float((out.double() - ref).norm() / ref.norm())
    assert err <= 1.1 * own, (err, own)
