"""The rotation's angle, by itself: rows of one component of 8 have unit norm
(mean square 1, eps 0), so the outputs are 8 cos and 8 sin of the angle.

Bound, relative to the 8: sincospif is within 1 unit in the last place of its
result, the correction by what the fp32 argument dropped rounds it once more
(1.5 units, below 1.5 2^-23 of the value), and the angle's last bit, 2^-32 of a
turn, is 0.025 2^-24; the reference's own angle is off by less than that at
these positions.  Products with 8 and 1 are exact."""

import pytest
import torch

from block_sparse_long_bwd_b200 import binding as bb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rot,inter,theta", [(64, False, 10000.0), (64, True, 500000.0),
                                             (36, False, 1e6)])
def test_cos_and_sin_are_as_exact_as_their_type(rot, inter, theta):
    L, half = 4096, rot // 2
    g = torch.Generator().manual_seed(rot)
    pos = torch.randint(0, 1 << 20, (1, L), generator=g, dtype=torch.int32)
    pos[0, :4] = torch.tensor([0, 1, 2, 3])
    q = torch.zeros(1, half, L, 64, device="cuda")  # head i: pair i
    a = [2 * i if inter else i for i in range(half)]
    b = [2 * i + 1 if inter else i + half for i in range(half)]
    for i in range(half):
        q[0, i, :, a[i]] = 8.0
    desc = bb.make_qk_desc(1, half, L, torch.float32, eps=0.0, theta=theta, rot_dim=rot,
                           interleaved=inter)
    y = bb.bb_qk_norm_rope_fwd(desc, q, q, None, None, pos.cuda())[0].double().cpu()
    assert (y[0, torch.arange(half), 0, a] == 8.0).all()
    for i in range(half):
        t = pos[0].double() * theta ** (-2.0 * i / rot)
        for j, want in ((a[i], t.cos()), (b[i], t.sin())):
            err = (y[0, i, :, j] / 8 - want).abs()
            tol = 1.5 * 2.0**-23 * want.abs() + 0.05 * 2.0**-24
            assert (err <= tol).all(), (i, j, (err / tol).max())
