"""Workspaces of the vocabulary projection's cross entropy, without a GPU."""

import pytest

from block_sparse_long_bwd_b200 import binding as bb


@pytest.mark.parametrize("N,V", [(16384, 50021), (131072, 131072), (200001, 200000),
                                 (1 << 20, 131072), (1 << 20, 1 << 24), (129, 1 << 24),
                                 (128, 1 << 24), (1, 1 << 24)])
@pytest.mark.parametrize("D", [64, 1024])
def test_the_forwards_workspace_does_not_grow_with_the_logits(N, D, V):
    """The packed rows and 256 MiB of (max, sum) pairs at most, plus a few
    words per row."""
    need = bb.bb_linear_ce_workspace_size(N, D, V, 0)
    rows = -(-N // 256) * 256
    assert need <= 2 * rows * D + (256 << 20) + 32 * rows + 4096
