"""The gamma gradients' sum over very many rows.  Components of +-1 have unit
norm (eps 0), without rotation the term of a row is dy x, and dy is a multiple
of 2^-10 below 4: what a block sums is a multiple of 2^-10 below 2^13, exact in
fp32.  The blocks' sums are added with the rounded-off parts kept (here multiples
of 2^-10, so exact too): the result is the exact sum rounded once."""

import pytest
import torch

from block_sparse_long_bwd_b200 import binding as bb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,H,L", [(1, 12, 5003), (2, 3, 16001), (1, 1, 33), (4, 8, 4096)])
def test_gamma_gradients_lose_nothing_between_blocks(B, H, L, dtype):
    g = torch.Generator(device="cuda").manual_seed(L)
    bits = 12 if dtype is torch.float32 else 7  # of dy, so that it is exact
    x, dy = [], []
    for _ in range(2):
        x.append((torch.randint(0, 2, (B, H, L, 64), generator=g, device="cuda") * 2 - 1)
                 .to(dtype))
        m = torch.randint(1 << (bits - 1), 1 << bits, (B, H, L, 64), generator=g, device="cuda")
        dy.append(x[-1] * (m * 2.0 ** (2 - bits)).to(dtype))  # terms of one sign
    desc = bb.make_qk_desc(B, H, L, dtype, eps=0.0, rot_dim=0)
    out = bb.bb_qk_norm_rope_bwd(desc, x[0], x[1], None, None, None, dy[0], dy[1])
    for i in range(2):
        want = (x[i].double() * dy[i].double()).sum((0, 1, 2))
        assert torch.equal(out[2 + i], want.float())


def test_an_infinite_term_stays_infinite():
    """One infinite dy: its component's sum is that infinity, and outside its
    pair (components are taken two by two, rotated or not) nothing changes."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = (torch.randint(0, 2, (1, 2, 4000, 64), generator=g, device="cuda") * 2 - 1).float()
    dy = torch.randint(-64, 65, (1, 2, 4000, 64), generator=g, device="cuda").float()
    desc = bb.make_qk_desc(1, 2, 4000, torch.float32, eps=0.0, rot_dim=0)
    want = bb.bb_qk_norm_rope_bwd(desc, x, x, None, None, None, dy, dy)[2].clone()
    dy[0, 1, 1234, 7] = -float("inf")
    got = bb.bb_qk_norm_rope_bwd(desc, x, x, None, None, None, dy, dy)[2]
    assert got[7] == -x[0, 1, 1234, 7] * float("inf")
    rest = torch.ones(64, dtype=torch.bool, device="cuda")
    rest[6:8] = False
    assert torch.equal(got[rest], want[rest])
