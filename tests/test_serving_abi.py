"""Refusals of the decode-step operators (include/gptq_serving.h): every argument check answers
before anything is launched, so none of this needs a GPU."""
import ctypes

import pytest

import gptq_bit_weight_gemm_gb300 as g
from gptq_bit_weight_gemm_gb300 import build as lib_build

P = ctypes.c_void_p
FAKE = P(0x10000)   # never dereferenced: validation fails before any device work
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    return g.lib()


def test_exports_every_declared_symbol(lib):
    declared = g.header_functions(g.SERVING_HEADER)
    assert declared == ["gptq_moe", "gptq_moe_workspace_size", "gptq_paged_attention",
                        "gptq_paged_attention_workspace_size", "gptq_sample"]
    for name in declared:
        assert hasattr(lib, name), name


ATTENTION = dict(q=FAKE, batch=2, heads=8, dtype=0, k_cache=FAKE, v_cache=FAKE, pages=4, page_size=16, kv_heads=2,
                 dim=64, strides=(1024, 0, 0, 2048, 128, 64, 2048, 128, 64), table=FAKE, width=2, lens=FAKE,
                 k_new=None, v_new=None, scale=1.0, window=0, out=FAKE, lse=None, workspace=FAKE, ws_bytes=BIG)


def attention(lib, **kw):
    a = dict(ATTENTION, **kw)
    strides = None if a["strides"] is None else (ctypes.c_longlong * 9)(*a["strides"])
    return lib.gptq_paged_attention(a["q"], a["batch"], a["heads"], a["dtype"], a["k_cache"], a["v_cache"], a["pages"],
                                    a["page_size"], a["kv_heads"], a["dim"], strides, a["table"], a["width"], a["lens"],
                                    a["k_new"], a["v_new"], a["scale"], a["window"], a["out"], a["lse"], a["workspace"],
                                    a["ws_bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), -1), (dict(strides=None), -1), (dict(k_new=FAKE), -1), (dict(q=None), -1), (dict(out=None), -1),
    (dict(workspace=None), -1), (dict(lens=None), -1),
    (dict(batch=-1), -2), (dict(heads=9), -2), (dict(kv_heads=0), -2), (dict(dim=60), -2), (dict(dim=264), -2),
    (dict(dim=0), -2), (dict(pages=0), -2), (dict(page_size=0), -2), (dict(width=0), -2), (dict(window=-1), -2),
    (dict(width=1 << 20, page_size=1 << 12), -2), (dict(batch=1 << 22), -2),
    (dict(q=P(0x10008)), -3), (dict(k_cache=P(0x10002)), -3), (dict(table=P(0x10002)), -3), (dict(lens=P(0x10001)), -3),
    (dict(strides=(1024, 0, 0, 2048, 132, 64, 2048, 128, 64)), -3),
    (dict(strides=(1024, 0, 0, -2048, 128, 64, 2048, 128, 64)), -3),
    (dict(ws_bytes=16), -4),
])
def test_attention_refusals(lib, kw, code):
    assert attention(lib, **kw) == code


def test_attention_empty_batch_is_noop(lib):
    assert attention(lib, batch=0, q=None, out=None) == 0


def test_attention_workspace_size(lib):
    assert g.paged_attention_workspace_size(32, 8, 128) > 0
    for bad in ((0, 8, 128), (32, 0, 128), (33, 8, 128), (32, 8, 0), (32, 8, 257), (32, 8, 12)):
        assert g.paged_attention_workspace_size(*bad) == 0, bad


MOE = dict(x=FAKE, tokens=4, hidden=256, inter=512, dtype=0, router=FAKE, experts=8, topk=2, renorm=1, uq=FAKE, uz=FAKE,
           us=FAKE, dq=FAKE, dz=FAKE, ds=FAKE, bits=4, group=128, fmt=2, out=FAKE, ids=None, weights=None,
           workspace=FAKE, ws_bytes=BIG)


def moe(lib, **kw):
    a = dict(MOE, **kw)
    return lib.gptq_moe(a["x"], a["tokens"], a["hidden"], a["inter"], a["dtype"], a["router"], a["experts"], a["topk"],
                        a["renorm"], a["uq"], a["uz"], a["us"], a["dq"], a["dz"], a["ds"], a["bits"], a["group"], a["fmt"],
                        a["out"], a["ids"], a["weights"], a["workspace"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(bits=5), -1), (dict(fmt=3), -1), (dict(dtype=2), -1), (dict(renorm=2), -1), (dict(x=None), -1),
    (dict(router=None), -1), (dict(dq=None), -1), (dict(out=None), -1), (dict(workspace=None), -1),
    (dict(tokens=-1), -2), (dict(tokens=33), -2), (dict(hidden=264), -2), (dict(inter=0), -2), (dict(topk=0), -2),
    (dict(topk=9), -2), (dict(experts=0), -2), (dict(experts=1025), -2), (dict(experts=64, topk=17), -2),
    (dict(group=96), -2), (dict(group=0), -2), (dict(group=16), -2), (dict(bits=2, group=32), -2),
    (dict(bits=3, group=64), -2), (dict(bits=3, group=-1, inter=544), -2), (dict(group=256, inter=384), -2),
    (dict(x=P(0x10008)), -3), (dict(ds=P(0x10002)), -3), (dict(ids=P(0x10002)), -3),
    (dict(ws_bytes=4096), -4),
])
def test_moe_refusals(lib, kw, code):
    assert moe(lib, **kw) == code


def test_moe_no_tokens_is_noop(lib):
    assert moe(lib, tokens=0, x=None, out=None, workspace=None, ws_bytes=0) == 0


def test_moe_workspace_size(lib):
    assert g.moe_workspace_size(32, 4096, 14336, 8, 2) > 0
    for bad in ((0, 4096, 14336, 8, 2), (33, 4096, 14336, 8, 2), (1, 4100, 14336, 8, 2), (1, 4096, 14336, 8, 9),
                (1, 4096, 14336, 2048, 2)):
        assert g.moe_workspace_size(*bad) == 0, bad
    # a workspace serves every smaller shape
    big = g.moe_workspace_size(32, 1024, 512, 64, 8)
    for small in ((1, 1024, 512, 64, 8), (32, 1024, 480, 64, 8), (32, 992, 512, 64, 8), (32, 1024, 512, 64, 7),
                  (32, 1024, 512, 63, 8)):
        assert g.moe_workspace_size(*small) <= big


SAMPLE = dict(logits=FAKE, batch=2, vocab=1000, row=1000, dtype=2, uniform=FAKE, t=None, k=None, p=None, m=None, token=FAKE,
              logprob=None)


def sample(lib, **kw):
    a = dict(SAMPLE, **kw)
    return lib.gptq_sample(a["logits"], a["batch"], a["vocab"], a["row"], a["dtype"], a["uniform"], a["t"], a["k"], a["p"],
                           a["m"], a["token"], a["logprob"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), -1), (dict(logits=None), -1), (dict(uniform=None), -1), (dict(token=None), -1),
    (dict(batch=-1), -2), (dict(vocab=0), -2), (dict(vocab=(1 << 22) + 1, row=1 << 23), -2), (dict(row=999), -2),
    (dict(logits=P(0x10002)), -3), (dict(dtype=0, logits=P(0x10001)), -3), (dict(uniform=P(0x10002)), -3),
    (dict(k=P(0x10002)), -3), (dict(logprob=P(0x10002)), -3),
])
def test_sample_refusals(lib, kw, code):
    assert sample(lib, **kw) == code


def test_sample_empty_batch_is_noop(lib):
    assert sample(lib, batch=0, logits=None, uniform=None, token=None) == 0
