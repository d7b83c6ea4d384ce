"""Refusals of a prompt step's operators at the edges of what their arguments can say.  Every check answers before
anything is launched, so none of this needs a GPU."""
import ctypes

import pytest

import gptq_bit_weight_gemm_gb300 as g
from test_prompt_abi import APPEND, lib, rotary  # noqa: F401


# ------------------------------------------------------------------------------ caches that overlap themselves
@pytest.mark.parametrize("at,stride", [(5, 0), (6, 0), (7, 0), (8, 0), (9, 0), (10, 0), (7, 56), (10, 8), (6, 32)])
def test_rotary_refuses_to_append_to_a_cache_whose_rows_overlap(lib, at, stride):  # noqa: F811
    # (k and v page, slot and head: a stride below a row's length writes several rows' values to one place)
    strides = [512, 128, 128, 512, 128, 2048, 128, 64, 2048, 128, 64]
    strides[at] = stride
    assert rotary(lib, **dict(APPEND, strides=tuple(strides))) == -2


def test_rotary_does_not_look_at_strides_of_dimensions_of_one(lib):  # noqa: F811
    # a single page, slot and head: past the strides' checks, refused for the alignment of the positions
    from test_prompt_abi import P
    strides = (512, 128, 128, 512, 128, 0, 0, 0, 0, 0, 0)
    assert rotary(lib, **dict(APPEND, pages=1, page=1, kv=1, strides=strides, positions=P(0x10002))) == -3


# ------------------------------------------------------------------------------ whole numbers past 32 bits, from Python
@pytest.mark.parametrize("name", ["page_size", "max_tokens"])
@pytest.mark.parametrize("value", [2 ** 32 + 16, 2 ** 31, -2 ** 32 + 16])
def test_page_plan_refuses_numbers_past_32_bits(name, value):
    with pytest.raises(ValueError, match=name):
        g.page_plan(None, None, None, None, None, **dict(dict(page_size=16, max_tokens=16), **{name: value}))


@pytest.mark.parametrize("rot", [2 ** 32 + 64, 2 ** 31, -2 ** 32 + 64])
def test_rotary_table_refuses_numbers_past_32_bits(rot):
    with pytest.raises((ValueError, g.GPTQError)):
        g.rotary_table(rot, device="cpu")


@pytest.mark.parametrize("window,used", [(0, 0), (5, 5), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1)])
def test_a_window_past_32_bits_hides_nothing(window, used):
    assert g._window(window) == used


def test_a_negative_window_stays_negative():
    assert g._window(-1) == -1 and -2 ** 31 <= g._window(-2 ** 32 + 5) < 0


def test_chunk_wait_hook_refuses_more_than_four_seconds(lib):  # noqa: F811
    hook = lib.gptq_selftest_chunk_attention_wait
    hook.restype, hook.argtypes = ctypes.c_int, [ctypes.c_uint]
    assert hook(4 * 10 ** 9 + 1) == -1 and hook(4 * 10 ** 9) == 0 and hook(1) == 0 and hook(0) == 0


# ------------------------------------------------------------------------------ the ramp's ends
@pytest.mark.parametrize("original,low", [(5.0, 1.0), (6.0, 1.0), (100.0, 20.0)])
def test_a_ramp_over_fewer_positions_than_the_fastest_pair_needs(lib, original, low):  # noqa: F811
    # pair 0 turns original / (2 pi) times, no more than `low`: every pair is divided by the factor
    turns, _ = g.rotary_table(64, scaling="ramp", factor=4.0, original=original, low=low, high=32.0, device="cpu")
    plain, _ = g.rotary_table(64, device="cpu")
    want = plain.double() / 4
    assert bool(((turns.double() - want).abs() <= 2.0 ** -48 * want + 1).all())


def test_a_ramp_over_more_positions_than_the_slowest_pair_needs(lib):  # noqa: F811
    turns, _ = g.rotary_table(64, scaling="ramp", factor=4.0, original=1e9, low=1.0, high=32.0, device="cpu")
    assert turns.equal(g.rotary_table(64, device="cpu")[0])
