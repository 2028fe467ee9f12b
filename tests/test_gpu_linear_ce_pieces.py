"""The cross entropy where the vocabulary goes by in several pieces (sizes
from the workspace: 256 MiB of pairs in the forward, of dz in the backward)."""

import pytest
import torch

from block_sparse_long_bwd_b200 import binding as bb

pytestmark = pytest.mark.gpu


def _ws(N, D, V, p):
    return torch.full((bb.bb_linear_ce_workspace_size(N, D, V, p),), 0xFF, dtype=torch.uint8,
                      device="cuda")


@pytest.mark.parametrize("N,V,labelled", [(40003, 250001, 300), (150001, 60007, 150),
                                          (1000003, 7000, 77)])
def test_forward(N, V, labelled):
    """Two or three pieces of pairs; few rows have a label (the workspace goes by all).
    Bounds: a logit is off by D 2^-23 of its terms' magnitudes (ez); lse by
    that, 2^-22 for the exponentials, 2^-22 of itself for the logarithm, and
    the sums' additions: 128 per pair, one per 32 pairs, 8 at the merge and two
    per piece, below 2^-13 together."""
    D = 64
    g = torch.Generator().manual_seed(N)
    w = torch.randn(V, D, generator=g).bfloat16().cuda()
    b = torch.randn(V, generator=g)
    b[V // 3 - 700:V // 3 + 700] = float("-inf")
    b = b.cuda()
    rows = torch.randperm(N, generator=g)[:labelled].sort().values.cuda()
    lab = torch.randint(0, V, (labelled,), generator=g).cuda()
    lab[torch.isinf(b[lab])] = 0
    lab[:3] = torch.tensor([0, V // 2, V - 1])
    h = torch.full((N, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    h[rows] = torch.randn(labelled, D, generator=g).bfloat16().cuda()
    labels = torch.full((N,), -1, dtype=torch.int32, device="cuda")
    labels[rows] = lab.int()
    ws = _ws(N, D, V, 0)
    loss, lse = bb.bb_linear_ce_fwd(h, w, b, labels, workspace=ws)
    assert bb.bb_attn_check_status(ws) == 0
    H = h[rows].double()
    z = H @ w.double().t() + b.double()
    ez = D * 2.0**-23 * (H.abs() @ w.double().abs().t()).amax(1)
    ref = z.logsumexp(1)
    at = z.gather(1, lab[:, None])[:, 0]
    el = ez + 2.0**-22 + 2.0**-13 + 2.0**-22 * ref.abs()
    assert ((lse[rows].double() - ref).abs() <= el).all()
    assert ((loss[rows].double() - (ref - at)).abs() <= el + ez + 2.0**-22 * at.abs()).all()
    out = torch.ones(N, dtype=torch.bool, device="cuda")
    out[rows] = False
    assert not loss[out].any() and not lse[out].any()
    # a piece whose every word is excluded, the first or the last, adds nothing
    for keep in (slice(0, V // 4), slice(V - V // 4, V)):
        c = torch.full_like(b, float("-inf"))
        c[keep] = 0.5
        lse = bb.bb_linear_ce_fwd(h, w, c, labels, workspace=ws)[1]
        ref = (H @ w[keep].double().t() + 0.5).logsumexp(1)
        assert ((lse[rows].double() - ref).abs() <= ez + 2.0**-12 + 2.0**-22 * ref.abs()).all()
    # every word excluded: no distribution
    loss = bb.bb_linear_ce_fwd(h, w, torch.full_like(b, float("-inf")), labels)[0]
    assert torch.isnan(loss[rows]).all()
