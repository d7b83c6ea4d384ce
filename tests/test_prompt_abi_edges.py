"""Refusals of a prompt step's operators at the edges of what their arguments can say.  Every check answers before
anything is launched, so none of this needs a GPU."""
import pytest

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
