"""Refusals of a prompt step's operators (include/gptq_prompt.h) and the table of rotary frequencies: every
argument check answers before anything is launched, so none of this needs a GPU."""
import ctypes
import math

import numpy as np
import pytest

import gptq_bit_weight_gemm_gb300 as g
from gptq_bit_weight_gemm_gb300 import build as lib_build

P = ctypes.c_void_p
FAKE, FAKE2, FAKE3 = P(0x10000), P(0x20000), P(0x30000)   # never dereferenced: validation fails before any device work
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    return g.lib()


def test_exports_every_declared_symbol(lib):
    declared = g.header_functions(g.PROMPT_HEADER)
    assert declared == ["gptq_chunk_attention", "gptq_chunk_attention_workspace_size", "gptq_page_plan", "gptq_rms_norm",
                        "gptq_rotary", "gptq_rotary_table"]
    for name in declared:
        assert hasattr(lib, name), name


# ------------------------------------------------------------------------------ page plan
PLAN = dict(cached=FAKE, added=FAKE, batch=2, page=16, table=FAKE, width=4, free=FAKE, capacity=8, count=FAKE, count_out=FAKE,
            lens=FAKE, cu=FAKE, positions=FAKE, slots=FAKE, tokens=64)


def plan(lib, **kw):
    a = dict(PLAN, **kw)
    return lib.gptq_page_plan(a["cached"], a["added"], a["batch"], a["page"], a["table"], a["width"], a["free"], a["capacity"],
                              a["count"], a["count_out"], a["lens"], a["cu"], a["positions"], a["slots"], a["tokens"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(cached=None), -1), (dict(added=None), -1), (dict(table=None), -1), (dict(free=None), -1), (dict(count=None), -1),
    (dict(count_out=None), -1), (dict(lens=None), -1), (dict(cu=None), -1), (dict(positions=None), -1), (dict(slots=None), -1),
    (dict(batch=-1), -2), (dict(batch=8193), -2), (dict(page=0), -2), (dict(width=0), -2), (dict(capacity=-1), -2),
    (dict(tokens=-1), -2), (dict(page=1 << 16, width=(1 << 14) + 1), -2),
    (dict(cached=P(0x10002)), -3), (dict(slots=P(0x10004)), -3), (dict(count_out=P(0x10001)), -3),
])
def test_plan_refusals(lib, kw, code):
    assert plan(lib, **kw) == code


# ------------------------------------------------------------------------------ norm
NORM = dict(x=FAKE, rows=2, hidden=64, xs=64, dtype=0, r=None, rs=0, rd=0, ro=None, ros=0, w=None, wd=0, eps=1e-6, out=FAKE2, os=64,
            od=0)


def norm(lib, **kw):
    a = dict(NORM, **kw)
    return lib.gptq_rms_norm(a["x"], a["rows"], a["hidden"], a["xs"], a["dtype"], a["r"], a["rs"], a["rd"], a["ro"], a["ros"], a["w"],
                             a["wd"], a["eps"], a["out"], a["os"], a["od"], None)


RES = dict(r=FAKE3, rs=64, rd=2, ro=FAKE3, ros=64)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), -1), (dict(od=-1), -1), (dict(x=None), -1), (dict(out=None), -1), (dict(r=FAKE), -1), (dict(ro=FAKE), -1),
    (dict(w=FAKE, wd=3), -1), (dict(RES, rd=7), -1),
    (dict(rows=-1), -2), (dict(hidden=0), -2), (dict(hidden=(1 << 20) + 1, xs=1 << 21, os=1 << 21), -2), (dict(xs=63), -2),
    (dict(os=63), -2), (dict(RES, rs=63), -2), (dict(RES, ros=63), -2),
    (dict(x=P(0x10001)), -3), (dict(dtype=2, x=P(0x10002)), -3), (dict(od=2, out=P(0x10002)), -3), (dict(w=P(0x10001)), -3),
    (dict(RES, r=P(0x10002)), -3),
    # in place, but not the same bytes row by row
    (dict(out=FAKE, od=1), -1), (dict(out=FAKE, os=128), -1), (dict(RES, ros=128), -1), (dict(RES, ro=FAKE), -1),
    (dict(RES, ro=FAKE2), -1), (dict(RES, r=FAKE2, ro=FAKE3), -1),
])
def test_norm_refusals(lib, kw, code):
    assert norm(lib, **kw) == code


def test_norm_no_rows_is_noop(lib):
    assert norm(lib, rows=0, x=None, out=None) == 0


# ------------------------------------------------------------------------------ rotary
ROTARY = dict(q=FAKE, k=FAKE, v=FAKE, tokens=4, heads=8, kv=2, dim=64, rot=64, inter=0, dtype=0,
              strides=(512, 128, 128, 512, 128, 2048, 128, 64, 2048, 128, 64), positions=FAKE, turns=FAKE, qo=FAKE2, ko=FAKE3, kc=None,
              vc=None, pages=0, page=0, slots=None)


def rotary(lib, **kw):
    a = dict(ROTARY, **kw)
    strides = None if a["strides"] is None else (ctypes.c_longlong * 11)(*a["strides"])
    return lib.gptq_rotary(a["q"], a["k"], a["v"], a["tokens"], a["heads"], a["kv"], a["dim"], a["rot"], a["inter"], a["dtype"],
                           strides, a["positions"], a["turns"], 1.0, a["qo"], a["ko"], a["kc"], a["vc"], a["pages"], a["page"],
                           a["slots"], None)


APPEND = dict(kc=FAKE, vc=FAKE2, pages=4, page=16, slots=FAKE)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), -1), (dict(inter=2), -1), (dict(strides=None), -1), (dict(q=None), -1), (dict(k=None), -1), (dict(qo=None), -1),
    (dict(ko=None), -1), (dict(positions=None), -1), (dict(turns=None), -1), (dict(kc=FAKE), -1), (dict(vc=FAKE), -1),
    (dict(APPEND, v=None), -1), (dict(APPEND, slots=None), -1),
    (dict(tokens=-1), -2), (dict(heads=0), -2), (dict(kv=0), -2), (dict(dim=60), -2), (dict(dim=264), -2), (dict(rot=0), -2),
    (dict(rot=7), -2), (dict(rot=66), -2), (dict(APPEND, pages=0), -2), (dict(APPEND, page=0), -2), (dict(heads=1 << 17), -2),
    (dict(strides=(512, 128, 128, 504, 128) + (0,) * 6), -2), (dict(strides=(512, 128, 128, 512, 120) + (0,) * 6), -2),
    (dict(APPEND, strides=(512, 128, 128, 512, 128, 1 << 41, 128, 64, 2048, 128, 64)), -2),
    (dict(q=P(0x10008)), -3), (dict(APPEND, kc=P(0x10008)), -3), (dict(positions=P(0x10002)), -3), (dict(turns=P(0x10004)), -3),
    (dict(strides=(508, 128, 128, 512, 128) + (0,) * 6), -3), (dict(strides=(-512, 128, 128, 512, 128) + (0,) * 6), -3),
    (dict(APPEND, strides=(512, 128, 128, 512, 128, 2044, 128, 64, 2048, 128, 64)), -3),
    (dict(qo=FAKE, strides=(1024, 128, 128, 512, 128) + (0,) * 6), -1), (dict(ko=FAKE, k=FAKE, strides=(512, 256, 128, 512, 128) + (0,) * 6), -1),
])
def test_rotary_refusals(lib, kw, code):
    assert rotary(lib, **kw) == code


def test_rotary_no_tokens_is_noop(lib):
    assert rotary(lib, tokens=0, q=None, k=None, qo=None, ko=None) == 0


def table(rot, **kw):
    t, a = g.rotary_table(rot, device="cpu", **kw)
    return t.numpy().astype(np.uint64).astype(np.float64) / 2.0 ** 64 * 2 * math.pi, a


@pytest.mark.parametrize("rot", [2, 6, 64, 128])
def test_rotary_table_follows_the_formulas(lib, rot):
    # a power, a logarithm or a division of 64 bits is off by a few 2^-53; the whole numbers by 2^-64 turns
    i = np.arange(rot // 2)
    for theta in (10000.0, 500000.0):
        f = theta ** (-2.0 * i / rot)
        close = lambda got, want: np.testing.assert_allclose(got, want, rtol=2 ** -48, atol=2 * math.pi * 2 ** -64)  # noqa: E731
        got, amp = table(rot, theta=theta)
        close(got, f)
        assert amp == 1.0
        close(table(rot, theta=theta, scaling="linear", factor=4.0)[0], f / 4)
        if rot > 2:
            close(table(rot, theta=theta, scaling="base", factor=8.0)[0], (theta * 8.0 ** (rot / (rot - 2))) ** (-2.0 * i / rot))
        got, amp = table(rot, theta=theta, scaling="ramp", factor=32.0, original=4096.0, low=1.0, high=32.0)
        turns = 4096 * f / (2 * math.pi)
        close(got[turns >= 32][:1], f[turns >= 32][:1])
        unit = 2 * math.pi * 2 ** -64
        assert bool((got <= f * (1 + 2 ** -48) + unit).all()) and bool((got >= f / 32 * (1 - 2 ** -48) - unit).all())
        assert abs(amp - (0.1 * math.log(32) + 1)) < 1e-15
        got, amp = table(rot, theta=theta, scaling="bands", factor=8.0, original=8192.0, low=1.0, high=4.0)
        turns = 8192 * f / (2 * math.pi)
        close(got[turns >= 4], f[turns >= 4])
        close(got[turns <= 1], f[turns <= 1] / 8)
        keep = np.clip((turns - 1) / 3, 0, 1)
        close(got, f / 8 * (1 - keep) + f * keep)
        assert amp == 1.0


def test_rotary_table_ramp_between_its_limits(lib):
    # rot 128, theta 10000: the pair that turns n times over `original` positions is 64 ln(original / (2 pi n)) / ln theta
    got, _ = table(128, theta=10000.0, scaling="ramp", factor=4.0, original=4096.0, low=1.0, high=32.0)
    i = np.arange(64)
    f = 10000.0 ** (-i / 64)
    at = lambda n: 64 * math.log(4096 / (2 * math.pi * n)) / math.log(10000.0)  # noqa: E731
    a, b = math.floor(at(32)), math.ceil(at(1))
    share = np.clip((i - a) / (b - a), 0, 1)
    np.testing.assert_allclose(got, f / 4 * share + f * (1 - share), rtol=2 ** -48, atol=2 * math.pi * 2 ** -64)


@pytest.mark.parametrize("rot,kw,code", [
    (0, {}, -2), (3, {}, -2), (65538, {}, -2), (64, dict(theta=1.0), -1), (64, dict(theta=float("nan")), -1),
    (64, dict(scaling="linear", factor=0.5), -1), (64, dict(scaling="base", factor=float("nan")), -1),
    (64, dict(scaling="ramp", factor=2.0, original=0.0), -1), (64, dict(scaling="bands", factor=2.0, original=100.0, low=4.0, high=4.0), -1),
    (64, dict(scaling="ramp", factor=2.0, original=100.0, low=0.0), -1),
])
def test_rotary_table_refusals(lib, rot, kw, code):
    with pytest.raises(g.GPTQError) as e:
        g.rotary_table(rot, device="cpu", **kw)
    assert e.value.code == code


def test_rotary_table_unknown_scaling(lib):
    with pytest.raises(ValueError):
        g.rotary_table(64, scaling="wider", device="cpu")


# ------------------------------------------------------------------------------ chunk attention
CHUNK = dict(q=FAKE, tokens=8, heads=8, dtype=0, kc=FAKE, vc=FAKE, pages=4, page=16, kv=2, dim=64,
             strides=(512, 2048, 128, 64, 2048, 128, 64), table=FAKE, width=2, lens=FAKE, cu=FAKE, batch=2, scale=1.0, window=0, out=FAKE2,
             lse=None, ws=FAKE3, ws_bytes=BIG)


def chunk(lib, **kw):
    a = dict(CHUNK, **kw)
    strides = None if a["strides"] is None else (ctypes.c_longlong * 7)(*a["strides"])
    return lib.gptq_chunk_attention(a["q"], a["tokens"], a["heads"], a["dtype"], a["kc"], a["vc"], a["pages"], a["page"], a["kv"],
                                    a["dim"], strides, a["table"], a["width"], a["lens"], a["cu"], a["batch"], a["scale"],
                                    a["window"], a["out"], a["lse"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), -1), (dict(strides=None), -1), (dict(q=None), -1), (dict(out=None), -1), (dict(ws=None), -1),
    (dict(lens=None), -1), (dict(cu=None), -1), (dict(table=None), -1),
    (dict(tokens=-1), -2), (dict(batch=-1), -2), (dict(heads=9), -2), (dict(kv=0), -2), (dict(dim=60), -2), (dict(dim=264), -2),
    (dict(pages=0), -2), (dict(page=0), -2), (dict(width=0), -2), (dict(window=-1), -2), (dict(width=1 << 20, page=1 << 12), -2),
    (dict(tokens=1 << 28), -2), (dict(batch=1 << 28), -2), (dict(heads=1 << 17), -2),
    (dict(strides=(512, 1 << 41, 128, 64, 2048, 128, 64)), -2), (dict(pages=1 << 25), -2),
    (dict(q=P(0x10008)), -3), (dict(kc=P(0x10002)), -3), (dict(table=P(0x10002)), -3), (dict(cu=P(0x10001)), -3),
    (dict(lse=P(0x10002)), -3), (dict(strides=(508, 2048, 128, 64, 2048, 128, 64)), -3),
    (dict(strides=(512, 2048, 132, 64, 2048, 128, 64)), -3), (dict(strides=(512, 2048, 128, 64, -2048, 128, 64)), -3),
    (dict(ws_bytes=16), -4),
])
def test_chunk_refusals(lib, kw, code):
    assert chunk(lib, **kw) == code


def test_chunk_nothing_to_do_is_noop(lib):
    assert chunk(lib, batch=0, q=None, out=None) == 0
    assert chunk(lib, tokens=0, q=None, out=None) == 0


def test_chunk_workspace_size(lib):
    assert g.chunk_attention_workspace_size(32, 8, 128) > 0
    for bad in ((0, 8, 128), (32, 0, 128), (33, 8, 128), (32, 8, 0), (32, 8, 257), (32, 8, 12), (1 << 17, 1, 64)):
        assert g.chunk_attention_workspace_size(*bad) == 0, bad
