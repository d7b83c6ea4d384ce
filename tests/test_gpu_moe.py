"""gptq_moe against the layer in 64 bits on weights dequantized from the same packed words.

Tolerance.  With A = sum_k |x w| of a projection, the fp32 sums of up to 4096 products (about 300
accumulations) are off by at most 2^-16 A.  The inner activation h = silu(g) u then moves by
1.1 |u| dg + |silu(g)| du, and its rounding to 11 bits relative to a run of 128 adds 2^-11 |h| plus
2^-24 of the run's largest; bf16 activations taken to fp16 add 2^-24 of the largest |x| of a run to
each product.  The down projection passes these on through |w| and adds its own 2^-16 sum |h w|.  A
routing logit is an fp32 sum of products, off by at most d = 2^-20 sum |x r|, and moves its weight by a
factor e^(2d); below 2^-126 a weight loses its bits.  out is rounded once (2^-11 or 2^-8, and fp16's
step 2^-24)."""
import numpy as np
import pytest
import torch

import gptq_bit_weight_gemm_gb300 as g
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_bit_weight_gemm_gb300 import build as lib_build
    lib_build.build()
    assert torch.cuda.is_available()
    yield
    assert g.device_status() == 0


def packed(rng, E, K, N, bits, group, fmt, scale):
    """(packed tensors on the GPU, fp64 weights [E, K, N])."""
    G = 1 if group == -1 else K // group
    qw = rng.integers(-2 ** 31, 2 ** 31, (E, K * bits // 32, N), dtype=np.int64).astype(np.int32)
    qz = rng.integers(-2 ** 31, 2 ** 31, (E, G, N * bits // 32), dtype=np.int64).astype(np.int32)
    sc = (scale * (0.5 + rng.random((E, G, N)))).astype(np.float16)
    W = np.empty((E, K, N))
    for e in range(E):
        z = oracle.unpack_n(qz[e], G, N, bits).astype(np.float64) + (1 if fmt == g.V1 else 0)
        # the stream of a column along K: rows of words become rows of the transposed stream
        q = oracle.unpack_n(np.ascontiguousarray(qw[e].T), N, K, bits).T.astype(np.float64)
        W[e] = (q - np.repeat(z, K // G, 0)) * np.repeat(sc[e].astype(np.float64), K // G, 0)
    return tuple(torch.from_numpy(t).to(DEV) for t in (qw, qz, sc)), torch.from_numpy(W).to(DEV)


def make(T, E, topk, H, I, bits, group, fmt, dtype, seed=0, x=None, spread=1.0):
    rng = np.random.default_rng(seed)
    up, Wu = packed(rng, E, H, 2 * I, bits, group, fmt, 0.1 / 2 ** bits)
    down, Wd = packed(rng, E, I, H, bits, group, fmt, 0.1 / 2 ** bits)
    x = torch.from_numpy(rng.standard_normal((T, H))).mul(spread).to(dtype).to(DEV) if x is None else x
    router = torch.from_numpy(rng.standard_normal((E, H)) * 2 / H ** 0.5).to(dtype).to(DEV)
    return dict(x=x, router=router, up=up, down=down, topk=topk, bits=bits, group=group, fmt=fmt), Wu, Wd


def run_max(t, run=128):
    """The largest |t| of each run of 128 along the last dimension, repeated over the run."""
    n = t.shape[-1]
    pad = torch.nn.functional.pad(t.abs(), (0, -n % run)).reshape(*t.shape[:-1], -1, run).amax(-1)
    return pad.repeat_interleave(run, -1)[..., :n]


def check(a, Wu, Wd, renormalize=True, workspace=None):
    out, ids, weights = g.moe_layer(**a, renormalize=renormalize, workspace=workspace, return_routing=True)
    torch.cuda.synchronize()
    x, router, k = a["x"].double(), a["router"].double(), a["topk"]
    T, I = x.shape[0], Wd.shape[1]
    p = torch.softmax(x @ router.T, -1)
    order = torch.sort(p, dim=-1, descending=True, stable=True)[1][:, :k]
    assert torch.equal(ids.long(), order)
    w = p.gather(1, order)
    if renormalize:
        w = w / w.sum(-1, keepdim=True)
    dlogit = 2.0 ** -20 * (x.abs() @ router.abs().T).amax(-1, keepdim=True)
    dw = torch.expm1(2 * dlogit).clamp(max=1) * w + 2.0 ** -16 * w + 2.0 ** -126
    assert bool(((weights.double() - w).abs() <= dw).all())
    ref, tol = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(T):
        for j in range(k):
            e = int(order[t, j])
            y, A = x[t] @ Wu[e], x[t].abs() @ Wu[e].abs()
            dy = 2.0 ** -16 * A + 2.0 ** -24 * (run_max(x[t]) @ Wu[e].abs())
            gate, u = y[:I], y[I:]
            silu = gate * torch.sigmoid(gate)
            h = silu * u
            dh = 1.1 * u.abs() * dy[:I] + silu.abs() * dy[I:] + 2.0 ** -11 * h.abs() + 2.0 ** -24 * run_max(h)
            yd = h @ Wd[e]
            ref[t] += w[t, j] * yd
            tol[t] += w[t, j] * (dh @ Wd[e].abs() + 2.0 ** -16 * (h.abs() @ Wd[e].abs())) + dw[t, j] * yd.abs()
    u = 2.0 ** (-11 if out.dtype == torch.float16 else -8)
    tol = tol + u * ref.abs() + 2.0 ** -24
    err = (out.double() - ref).abs()
    assert bool((err <= tol).all()), "max error %g of %g, %d outside" % (float(err.max()), float(ref.abs().max()), int((err > tol).sum()))
    return out


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("fmt", [g.V1, g.V2])
@pytest.mark.parametrize("bits,group", [(2, 64), (2, 128), (3, 128), (4, 32), (4, 128), (4, -1), (8, 16), (8, 32), (8, 128), (3, -1),
                                        (8, -1), (2, -1)])
def test_widths_and_groups(bits, group, fmt, dtype):
    check(*make(5, 6, 2, 256, 384, bits, group, fmt, dtype, seed=bits))


@pytest.mark.parametrize("tokens", [1, 2, 7, 8, 9, 15, 16, 17, 24, 31, 32])
@pytest.mark.parametrize("E,topk", [(8, 2), (4, 4), (1, 1)])
def test_token_counts(tokens, E, topk):
    check(*make(tokens, E, topk, 256, 256, 4, 128, g.V2, torch.float16, seed=tokens))


@pytest.mark.parametrize("H,I,group", [(32, 32, 32), (1056, 672, 32), (96, 2048, -1), (1920, 96, 96), (544, 160, 32), (4096, 128, 128)])
@pytest.mark.parametrize("tokens", [1, 11])
def test_odd_shapes(H, I, group, tokens):
    check(*make(tokens, 5, 3, H, I, 4, group, g.V2, torch.bfloat16, seed=H), renormalize=False)


def test_many_experts():
    check(*make(32, 200, 8, 256, 128, 4, 128, g.V2, torch.bfloat16, seed=1))
    check(*make(3, 1024, 16, 64, 32, 4, 32, g.V2, torch.float16, seed=2))


def test_all_tokens_on_one_expert():
    a, Wu, Wd = make(32, 8, 1, 256, 256, 4, 64, g.V2, torch.float16, seed=3)
    a["router"][:] = 0
    a["router"][5] = 0.01
    a["x"] = a["x"].abs()
    check(a, Wu, Wd)


def test_equal_logits_take_the_lowest_index():
    a, Wu, Wd = make(4, 8, 3, 256, 256, 4, 128, g.V2, torch.float16, seed=4)
    a["router"][:] = a["router"][2:3].clone()
    _, ids, weights = g.moe_layer(**a, return_routing=True)
    assert ids.tolist() == [[0, 1, 2]] * 4 and torch.allclose(weights, torch.full_like(weights, 1 / 3))


def test_large_and_small_activations():
    # |h| far past fp16's largest value and far below its smallest, in one batch
    x = torch.randn((4, 256), generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).to(DEV)
    x[0] *= 3000.0
    x[1] *= 1e-6
    x[2, :128] *= 1000.0
    check(*make(4, 4, 2, 256, 384, 4, 64, g.V2, torch.bfloat16, seed=6, x=x))


def test_nan_stays_in_its_token():
    a, Wu, Wd = make(6, 4, 2, 256, 256, 4, 64, g.V2, torch.float16, seed=7)
    good = g.moe_layer(**a)
    a["x"][3, 17] = float("nan")
    out = g.moe_layer(**a)
    assert bool(out[3].isnan().all())
    keep = [0, 1, 2, 4, 5]
    ref = good[keep].double()
    assert bool(((out[keep].double() - ref).abs() <= 2.0 ** -9 * ref.abs().max()).all())


def test_one_workspace_repeatable_and_side_stream():
    ws = g.moe_workspace(32, 512, 512, 64, 8)
    shapes = [(1, 8, 2, 256, 512), (32, 64, 8, 512, 256), (9, 16, 4, 512, 512)]
    outs = {}
    for turn in range(3):
        for i, (T, E, k, H, I) in enumerate(shapes):
            case = make(T, E, k, H, I, 4, 64, g.V2, torch.float16, seed=i)
            out = check(*case, workspace=ws)
            if turn:
                assert torch.equal(out, outs[i])       # the same bits every time
            outs[i] = out
    a = make(*shapes[1], 4, 64, g.V2, torch.float16, seed=1)[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = g.moe_layer(**a)
    s.synchronize()
    assert torch.equal(out, outs[1])


def test_full_width_expert():
    # the 8 x [4096, 14336] layer at a slice of its width: long rows, every expert busy
    check(*make(8, 8, 2, 4096, 1024, 4, 128, g.V2, torch.float16, seed=8))


def test_wrong_tensors_are_refused():
    a = make(2, 4, 2, 256, 256, 4, 64, g.V2, torch.float16)[0]
    for kw in (dict(x=a["x"].cpu()), dict(router=a["router"][:, :128]), dict(group=128), dict(bits=8),
               dict(down=(a["down"][0][:3], a["down"][1], a["down"][2]))):
        with pytest.raises(ValueError):
            g.moe_layer(**dict(a, **kw))
    with pytest.raises(TypeError):
        g.moe_layer(**dict(a, router=a["router"].float()))
    with pytest.raises(g.GPTQError) as e:
        g.moe_layer(**dict(a, x=a["x"].repeat(20, 1)))
    assert e.value.code == -2
