"""Refusals of the FP8 and balance binding that need no GPU."""

import pytest

import moe_decode_layer_router_amd as mb

FAKE = 0x7F0000000000  # never dereferenced


@pytest.mark.parametrize("nbytes", [None, -1, -(2**40)])
def test_workspace_of_unknown_or_negative_size(nbytes):
    """A raw pointer without a size, and a size that would turn into a huge one."""
    with pytest.raises(ValueError):
        mb._workspace(FAKE, nbytes, mb._t(), 0)


def test_workspace_of_a_raw_pointer():
    assert mb._workspace(FAKE, 4096, mb._t(), 0) == (FAKE, 4096)
    assert mb._workspace(None, None, mb._t(), 0) == (None, 0)
