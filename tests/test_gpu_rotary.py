"""gptq_rotary against the rotation in 64 bits.

Tolerance, for u = 2^-11 (fp16) or 2^-8 (bf16): the angle is exact but for one rounding of its turns to fp32 (pi
2^-25 rad), sine and cosine are within 2^-22, the two products and their sum round three times:
  |out - ref| <= u |ref| + 2^-20 amplitude (|a| + |b|) + 2^-25.
Dimensions that are not turned, and values, have to be the same bits; so has everything a row does not own."""
import math

import pytest
import torch

import gptq_bit_weight_gemm_gb300 as g

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_bit_weight_gemm_gb300 import build as lib_build
    lib_build.build()
    assert torch.cuda.is_available()
    yield
    assert g.device_status() == 0


def bits(t):
    return t.contiguous().view(torch.int16)


def make(tokens, heads, kv, dim, dtype, seed=0, far=5000, contiguous=False):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    fused = torch.randn((tokens, heads + 2 * kv, dim), device=DEV, generator=gen).to(dtype)
    q, k, v = fused.split([heads, kv, kv], 1)
    if contiguous:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    return q, k, v, torch.randint(0, far, (tokens,), device=DEV, generator=gen, dtype=torch.int32)


def ref(x, positions, freq, rot, interleaved, amplitude):
    """(rotated, tolerance) in 64 bits."""
    u = 2.0 ** (-11 if x.dtype == F16 else -8)
    y = x.double().clone()
    tol = torch.zeros_like(y)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    t = (positions.double()[:, None] * freq)[:, None]
    c, s, p, r = t.cos() * amplitude, t.sin() * amplitude, y[..., a].clone(), y[..., b].clone()
    y[..., a], y[..., b] = p * c - r * s, p * s + r * c
    for w in (a, b):
        tol[..., w] = u * y[..., w].abs() + 2.0 ** -20 * amplitude * (p.abs() + r.abs()) + 2.0 ** -25
    return y, tol


def close(got, x, positions, freq, rot, interleaved, amplitude=1.0):
    want, tol = ref(x, positions, freq, rot, interleaved, amplitude)
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), "max error %g" % float(err.nan_to_num(math.inf).max())
    assert torch.equal(bits(got[..., rot:]), bits(x[..., rot:]))


def frequencies(rot, theta=10000.0):
    return theta ** (-2 * torch.arange(rot // 2, device=DEV, dtype=torch.float64) / rot)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("heads,kv,dim,rot", [(32, 8, 128, 128), (8, 8, 64, 64), (15, 5, 80, 80), (15, 5, 80, 32), (15, 5, 80, 40), (4, 1, 256, 256),
                                              (1, 1, 8, 8), (2, 1, 16, 2), (3, 1, 96, 6), (5, 2, 128, 10), (6, 3, 24, 20), (64, 4, 128, 64),
                                              (2, 2, 256, 254), (70, 1, 64, 48)])
def test_heads_and_parts(dtype, interleaved, heads, kv, dim, rot):
    turns, amp = g.rotary_table(rot)
    for tokens in (1, 37):
        q, k, _, pos = make(tokens, heads, kv, dim, dtype, seed=rot)
        qo, ko = g.rotary(q, k, pos, turns, interleaved=interleaved)
        assert qo.is_contiguous() and ko.is_contiguous()
        close(qo, q, pos, frequencies(rot), rot, interleaved)
        close(ko, k, pos, frequencies(rot), rot, interleaved)


def test_far_and_negative_positions():
    turns, _ = g.rotary_table(128, theta=500000.0)
    q, k, _, pos = make(300, 4, 2, 128, F16, seed=1)
    pos[::3] = torch.randint(10 ** 6, 2 ** 31 - 1, (100,), device=DEV, dtype=torch.int32)
    pos[1] = 0
    pos[2], pos[5] = 2 ** 31 - 1, -2 ** 31
    pos[4::30] *= -1
    # a frequency off by 2^-52 and an angle of 2^31 of them: 2^-21 rad more than close() allows
    qo, ko = g.rotary(q, k, pos, turns)
    for got, x in ((qo, q), (ko, k)):
        want, tol = ref(x, pos, frequencies(128, 500000.0), 128, False, 1.0)
        more = 2.0 ** -49 * pos.double().abs()[:, None, None] * (x.double().abs() + x.double().roll(64, -1).abs())
        assert bool(((got.double() - want).abs() <= tol + more).all())


@pytest.mark.parametrize("kind,kw", [("linear", dict(factor=4.0)), ("base", dict(factor=8.0)), ("ramp", dict(factor=16.0, original=4096.0)),
                                     ("bands", dict(factor=8.0, original=8192.0, low=1.0, high=4.0))])
def test_scaled_frequencies_and_amplitude(kind, kw):
    turns, amp = g.rotary_table(64, scaling=kind, **kw)
    freq = turns.double() / 2.0 ** 64 * 2 * math.pi
    q, k, _, pos = make(50, 4, 2, 64, BF16, seed=2, far=100000)
    qo, ko = g.rotary(q, k, pos, turns, amplitude=amp)
    close(qo, q, pos, freq, 64, False, amp)
    close(ko, k, pos, freq, 64, False, amp)


@pytest.mark.parametrize("page", [1, 13, 16, 64])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "hpn"])
@pytest.mark.parametrize("tokens,dim,rot,interleaved", [(1, 128, 128, False), (100, 64, 64, True), (61, 80, 40, False)])
def test_append_writes_the_slots_and_nothing_else(page, layout, tokens, dim, rot, interleaved):
    heads, kv = 6, 3
    q, k, v, pos = make(tokens, heads, kv, dim, BF16, seed=page)
    pages = -(-tokens // page) * 2 + 1
    shape = {"nhd": (pages, page, kv, dim), "hnd": (pages, kv, page, dim), "hpn": (kv, pages, page, dim)}[layout]
    perm = {"nhd": (0, 1, 2, 3), "hnd": (0, 2, 1, 3), "hpn": (1, 2, 0, 3)}[layout]
    caches = [torch.full(shape, float("nan"), dtype=BF16, device=DEV).permute(*perm) for _ in range(2)]
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(page))[:tokens].to(DEV)
    slots[tokens // 2::7] = -1
    turns, _ = g.rotary_table(rot)
    plain = g.rotary(q, k, pos, turns, interleaved=interleaved)
    qo, ko = g.rotary(q, k, pos, turns, interleaved=interleaved, v=v, k_cache=caches[0], v_cache=caches[1], slots=slots)
    assert ko is None and torch.equal(bits(qo), bits(plain[0]))
    keep = slots >= 0
    where = slots[keep] // page, slots[keep] % page
    for cache, rows in zip(caches, (plain[1], v)):
        want = torch.full((pages, page, kv, dim), float("nan"), dtype=BF16, device=DEV)
        want[where] = rows[keep]
        assert torch.equal(bits(cache), bits(want))
    ko = torch.empty_like(plain[1])
    got = g.rotary(q, k, pos, turns, interleaved=interleaved, v=v, k_cache=caches[0], v_cache=caches[1], slots=slots, k_out=ko)
    assert got[1] is ko and torch.equal(bits(ko), bits(plain[1]))


def test_slots_past_the_cache_are_flagged():
    q, k, v, pos = make(5, 2, 1, 64, F16, seed=3)
    turns, _ = g.rotary_table(64)
    cache = torch.zeros((2, 2, 4, 1, 64), dtype=F16, device=DEV)
    slots = torch.tensor([0, 8, 7, 2 ** 62, -2 ** 62], device=DEV)
    g.rotary(q, k, pos, turns, v=v, k_cache=cache[0], v_cache=cache[1], slots=slots)
    assert g.device_status() == g.DEV_SLOT_RANGE
    assert torch.equal(cache[1].reshape(8, 1, 64)[[0, 7]], v[[0, 2]]) and float(cache[1].reshape(8, 64)[1:7].abs().max()) == 0.0


@pytest.mark.parametrize("rot,interleaved", [(64, False), (64, True), (20, False), (6, True)])
def test_in_place(rot, interleaved):
    q, k, _, pos = make(41, 6, 2, 64, F16, seed=4)
    turns, _ = g.rotary_table(rot)
    want = [t.clone() for t in g.rotary(q, k, pos, turns, interleaved=interleaved)]
    got = g.rotary(q, k, pos, turns, interleaved=interleaved, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(bits(q), bits(want[0])) and torch.equal(bits(k), bits(want[1]))


def test_many_tokens_cache_past_32_bits_and_strides():
    tokens, kv, dim = 3000, 2, 64
    q, k, v, pos = make(tokens, 4, kv, dim, F16, seed=5, contiguous=True)
    pages, page = 2 ** 31 // (256 * kv * dim) + 40, 256
    caches = [torch.empty((pages, page, kv, dim), dtype=F16, device=DEV) for _ in range(2)]
    slots = pages * page - 1 - torch.arange(tokens, device=DEV) * 3
    turns, _ = g.rotary_table(dim)
    ko = torch.empty_like(k)
    g.rotary(q, k, pos, turns, v=v, k_cache=caches[0], v_cache=caches[1], slots=slots, k_out=ko)
    for cache, rows in zip(caches, (ko, v)):
        assert torch.equal(bits(cache[slots // page, slots % page]), bits(rows))
    close(ko, k, pos, frequencies(dim), dim, False)


def test_captured_and_on_another_stream():
    q, k, _, pos = make(77, 8, 2, 128, BF16, seed=6)
    turns, _ = g.rotary_table(128)
    want = g.rotary(q, k, pos, turns)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = g.rotary(q, k, pos, turns, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = g.rotary(q, k, pos, turns)
    pos += 5
    want = [t.clone() for t in g.rotary(q, k, pos, turns)]
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_wrong_tensors_are_refused():
    q, k, v, pos = make(4, 4, 2, 64, F16)
    turns, _ = g.rotary_table(64)
    cache = torch.zeros((3, 4, 2, 64), dtype=F16, device=DEV)
    a = dict(q=q, k=k, positions=pos, turns=turns)
    slots = torch.zeros(4, dtype=torch.int64, device=DEV)
    for kw in (dict(q=q.cpu()), dict(k=k[:, :, :32]), dict(positions=pos[:3]), dict(k_cache=cache), dict(v=v), dict(slots=slots),
               dict(v=v, k_cache=cache, v_cache=cache[..., :32], slots=slots), dict(q=q.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(ValueError):
            g.rotary(**dict(a, **kw))
    for kw in (dict(q=q.float()), dict(k=k.bfloat16()), dict(positions=pos.long()), dict(turns=turns.int()),
               dict(v=v, k_cache=cache, v_cache=cache.clone(), slots=slots.int())):
        with pytest.raises(TypeError):
            g.rotary(**dict(a, **kw))
    with pytest.raises(g.GPTQError) as e:      # more dimensions than the head has
        g.rotary(q, k, pos, g.rotary_table(128)[0])
    assert e.value.code == -2
    assert g.rotary(q[:0], k[:0], pos[:0], turns)[0].shape == (0, 4, 64)
