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


@pytest.mark.parametrize("N,D,V,labelled", [
    (40003, 64, 7001, 40003), (300000, 64, 1201, 300000), (100, 64, (1 << 20) + 700, 90),
    (100, 72, (1 << 20) + 513, 50), (128, 64, (1 << 20) + 1, 128), (3000, 128, 300001, 50),
    (20000, 200, 20001, 64), (9000, 136, 40001, 2000)])
def test_exact_integer_gradients(N, D, V, labelled):
    """Two to seven pieces, the last one ragged; every logit is 0 (h uses
    features that w leaves at zero) and lse 0, so dz, dh, dw and dbias are sums
    of small integers below 2^24: equal to them rounded once.  dz in one part
    and in two."""
    g = torch.Generator().manual_seed(N + V)
    half = D // 2
    h, w = torch.zeros(N, D), torch.zeros(V, D)
    h[:, :half] = torch.randint(-2, 3, (N, half), generator=g).float()
    w[:, half:] = torch.randint(-2, 3, (V, D - half), generator=g).float()
    labels = torch.full((N,), -100, dtype=torch.int32)
    on = torch.randperm(N, generator=g)[:labelled].sort().values
    labels[on] = torch.randint(0, V, (labelled,), generator=g, dtype=torch.int32)
    labels[on[0]], labels[on[-1]] = 0, V - 1
    dl = torch.tensor([1.0, 2.0])[torch.randint(0, 2, (N,), generator=g)]
    off = torch.ones(N, dtype=torch.bool)
    off[on] = False
    h[off], dl[off] = float("nan"), float("nan")
    h, w, labels, dl, on = (t.cuda() for t in (h.bfloat16(), w.bfloat16(), labels, dl, on))
    ws = _ws(N, D, V, 1)
    dh, dw, db = bb.bb_linear_ce_bwd(h, w, torch.zeros(V, device="cuda"), labels,
                                     torch.zeros(N, device="cuda"), dl, workspace=ws)
    assert bb.bb_attn_check_status(ws) == 0
    # dz = dl (1 - onehot): all ones less the labels' words
    H, W, lab, d = h[on].double(), w.double(), labels[on].long(), dl[on].double()
    want = torch.zeros(N, D, dtype=torch.float64, device="cuda")
    want[on] = d[:, None] * (W.sum(0) - W[lab])
    assert torch.equal(dh, want.float().bfloat16())
    want = (d @ H).expand(V, D).clone().index_add_(0, lab, -d[:, None] * H)
    assert torch.equal(dw, want.float().bfloat16())
    want = d.sum().expand(V).clone().index_add_(0, lab, -d)
    assert torch.equal(db, want.float())
