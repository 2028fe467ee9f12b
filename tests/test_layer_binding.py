"""Arguments that the binding of the operators around the attention refuses,
without a GPU."""

import pytest
import torch

from block_sparse_long_bwd_b200 import binding as bb


@pytest.mark.parametrize("call", [lambda *a: bb.bb_dropout_fwd(torch.zeros(16), None, 0.1, *a),
                                  lambda *a: bb.bb_dropout_bwd(torch.zeros(16), 0.1, *a)])
def test_sites_past_their_word(call):
    """They would be cut to 32 bits, and two sites share their decisions."""
    for site in (-1, 1 << 32, (1 << 32) + 3):
        with pytest.raises(ValueError, match="site"):
            call(0, site)
    for site in (0, (1 << 32) - 1):
        with pytest.raises(ValueError, match="CUDA tensor"):  # these pass on
            call(7, site)
