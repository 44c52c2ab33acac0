"""Limits of the draft-tree entry points that are refused on the host, without a GPU."""
import pytest

from tests.test_abi_tree_cpu import UNSUPPORTED, call


@pytest.mark.parametrize("name", ["kda_tree_conv", "kda_tree_conv_commit"])
def test_channel_numbers_fit_an_int(name):
    for C in ((1 << 31) - 1, (1 << 31) - 512):
        assert call(name, C=C, W=1) == UNSUPPORTED
