"""CPU tests of the sizes that the scalar-gated delta rule's and the q/k
preparation's entries take: workspaces of refused sizes, and the launch limits
(descriptors alone: the checks read no memory)."""

import pytest

from tests.test_delta_host import gdn2  # noqa: F401


@pytest.mark.parametrize("args", [
    (130, 2, 2, 4, 16, 16), (130, 2, 2, 4, 1, 1), (130, 2, 2, 4, 96, 96), (130, 2, 2, 4, 64, 128), (130, 2, 3, 4, 64, 64),
    (130, 2, 2, 4, 1 << 30, 1 << 30), (64, 1 << 20, 1, 1 << 18, 1 << 27, 1 << 27), (1 << 31, 1, 1, 1, 64, 64),
    (1 << 62, 1, 1, 1, 64, 64), (64, (1 << 31) - 1, 1, (1 << 31) - 1, 64, 64), (64, 1, 1, 1 << 18, 64, 64), (130, -1, 2, 4, 64, 64)])
def test_no_backward_workspace_for_refused_sizes(gdn2, args):
    """(Head sizes under 32 divided by zero here and ended the process.)"""
    assert gdn2.delta_chunk_bwd_workspace(*args) == 0


@pytest.mark.parametrize("args", [(1 << 31, 1, 1), (1 << 62, 1, 1), (64, (1 << 31) - 1, (1 << 31) - 1), (64, 5592405, 2), (64, -1, 2)])
def test_no_forward_workspace_for_refused_sizes(gdn2, args):
    assert gdn2.delta_chunk_fwd_workspace(*args) == 0


def test_no_preparation_workspace_for_refused_sizes(gdn2):
    for args in ((9, 2, 2, 32), (1 << 31, 2, 2, 64), (9, (1 << 31) - 1, (1 << 31) - 1, 64)):
        assert gdn2.qk_norm_rope_bwd_workspace(*args) == 0
