"""Calls of the operators of drafted trees that their documentation allows and those next to them that it does not, without a GPU."""
import pytest
import torch

from test_paged_cpu import lib  # noqa: F401
from test_tree_cpu import _call


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
@pytest.mark.parametrize("axes", [2, 4])
def test_axes_may_share_their_positions(lib, axes):  # noqa: F811
    """One row of positions for all axes (a text's tokens under several axes): its expanded view has a stride of 0."""
    assert _call(lib, "rope", dict(axes=axes, position_stride=0)) == -5


@pytest.mark.parametrize("stride", [1, 2, -3, -1])
def test_axes_that_overlap_in_part_are_refused(lib, stride):  # noqa: F811
    assert _call(lib, "rope", dict(position_stride=stride)) == -1
