"""Gradients where single rows and words lead: a row of dh is its label's
entry of dz times that word's weights, a row of dW the entries of the rows
that have the word as label.

A word is told apart by two features (its low six bits, the rest), where w
holds 1 and h of a row with that label 20: z = 40 for the label, 20 for words
that share one of the two, 0 for all others, every one of them exact.  lse is
chosen, so the label's probability is any wanted one and the other words' are
below 2^-28 of it.  64 further features are random in w and zero in h, 64 the
other way round: they carry what dh and dW are compared on.

Bounds: p is off by e = 2^-22 |z - lse| + 2^-21 of itself (the exponential and
its argument); entries other than labels' are rounded to bf16 (2^-8 of them,
next to nothing here); sums and the last scaling leave 2^-20 of the terms'
magnitudes; results are rounded once (2^-8).  The labels' own entries are
held in fp32, so nothing of theirs is rounded before: for dh in every row, for
dW in words that at most four rows have as label (above, 2^-8 of the terms).
Up to 64 rows all entries are held in two bf16 parts, which leave 2^-16."""

import pytest
import torch

from block_sparse_long_bwd_b200 import binding as bb

pytestmark = pytest.mark.gpu
HEAVY = 4  # rows of a word whose entries are held exactly
D = 320


def _case(N, V, labelled, words, seed):
    """Labels among the first `words` words; weights 1 .. 2 and probabilities
    0.1 .. 0.6, all different."""
    g = torch.Generator().manual_seed(seed)
    assert V <= 64 * 128
    v = torch.arange(V)
    w = torch.zeros(V, D)
    w[v, v % 64] = 1.0
    w[v, 64 + v // 64] = 1.0
    w[:, 192:256] = torch.randn(V, 64, generator=g)
    lab = torch.randint(0, words, (N,), generator=g) * (V // words)
    n = torch.arange(N)
    h = torch.zeros(N, D)
    h[n, lab % 64] = 20.0
    h[n, 64 + lab // 64] = 20.0
    h[:, 256:] = torch.randn(N, 64, generator=g)
    p = 0.1 + 0.5 * torch.rand(N, generator=g)
    lse = 40.0 - p.log()
    dl = 1.0 + torch.rand(N, generator=g)
    labels = torch.full((N,), -100)
    on = torch.randperm(N, generator=g)[:labelled]
    labels[on] = lab[on]
    c = lambda t: t.cuda()
    return (c(h.bfloat16()), c(w.bfloat16()), c(labels.to(torch.int32)), c(lse), c(dl))


def _bounds(h, w, labels, lse, dl):
    """Results in 64 bits and their bounds, for the rows with a label."""
    rows = (labels >= 0).nonzero()[:, 0]
    H, W = h[rows].double(), w.double()
    lab = labels[rows].long()
    heavy = torch.bincount(lab, minlength=w.shape[0]) > HEAVY
    dh, dw = torch.zeros_like(H), torch.zeros_like(W)
    th, tw = torch.zeros_like(H), torch.zeros_like(W)
    for part in torch.arange(rows.numel(), device="cuda").split(4096):
        z, l = H[part] @ W.t(), lse[rows[part], None].double()
        d = dl[rows[part], None].double()
        p = (z - l).exp()
        hot = torch.nn.functional.one_hot(lab[part], w.shape[0])
        dz, off = d * (p - hot), d * p * (2.0**-22 * (z - l).abs() + 2.0**-21)
        dh[part] = dz @ W
        dw += dz.t() @ H[part]
        two = rows.numel() <= 64
        rest, a = (dz * (1 - hot)).abs() * 2.0**-8 + off, dz.abs()
        a = a * (2.0**-20 + two * 2.0**-16)
        th[part] = (rest + a) @ W.abs()
        tw += (rest + a + 2.0**-8 * (heavy & (not two)) * dz.abs()).t() @ H[part].abs()
    return rows, dh, dw, 2.0**-8 * dh.abs() + th, 2.0**-8 * dw.abs() + tw


@pytest.mark.parametrize("N,V,labelled,words", [
    (1, 700, 1, 1), (64, 700, 64, 64), (65, 700, 65, 350), (100, 8192, 64, 64),
    (100, 3001, 70, 60), (128, 700, 128, 64), (128, 3001, 127, 3001), (129, 700, 129, 350),
    (300, 1537, 300, 192), (400, 8192, 130, 64), (1000, 3001, 65, 65), (1000, 700, 1000, 1),
    (2500, 8192, 2500, 8192), (2500, 8100, 1250, 2025), (40003, 7001, 40003, 7001),
    (20000, 8192, 4000, 4096), (20000, 8192, 60, 60), (30000, 8192, 64, 40)])
def test_labels_entries_are_held_exactly(N, V, labelled, words):
    h, w, labels, lse, dl = _case(N, V, labelled, words, N + V)
    ws = torch.full((bb.bb_linear_ce_workspace_size(N, D, V, 1),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    h[labels < 0] = float("nan")  # rows without a label enter nothing
    dh, dw, _ = bb.bb_linear_ce_bwd(h, w, None, labels, lse, dl, workspace=ws)
    assert bb.bb_attn_check_status(ws) == 0
    rows, eh, ew, th, tw = _bounds(h, w, labels, lse, dl)
    assert rows.numel() == labelled
    err = (dh[rows].double() - eh).abs()
    assert (err <= th).all(), (err / th).max()
    err = (dw.double() - ew).abs()
    assert (err <= tw).all(), (err / tw).max()
    out = torch.ones(N, dtype=torch.bool, device="cuda")
    out[rows] = False
    assert not dh[out].any()


def test_the_same_row_whatever_else_has_a_label():
    """64 rows' dh, alone and with one more row labelled: both within the
    bound, so the results differ by its two halves at most."""
    h, w, labels, lse, dl = _case(65, 2000, 65, 500, 7)
    got = []
    for last in (-100, int(labels[64])):
        labels[64] = last
        dh = bb.bb_linear_ce_bwd(h, w, None, labels, lse, dl)[0]
        rows, eh, _, th, _ = _bounds(h, w, labels, lse, dl)
        assert ((dh[rows].double() - eh).abs() <= th).all()
        got.append(dh[:64].double())
    assert ((got[0] - got[1]).abs() <= 2 * th[:64]).all()


def test_run_to_run_and_streams():
    """The rows of a word are taken in a fixed order: the same bits each time,
    and with the rows' labels replaced in a replayed graph."""
    h, w, labels, lse, dl = _case(700, 900, 500, 150, 8)
    want = bb.bb_linear_ce_bwd(h, w, None, labels, lse, dl)
    for _ in range(3):
        again = bb.bb_linear_ce_bwd(h, w, None, labels, lse, dl)
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
    lab = labels.clone()
    ws = torch.empty(bb.bb_linear_ce_workspace_size(700, D, 900, 1), dtype=torch.uint8,
                     device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = bb.bb_linear_ce_bwd(h, w, None, lab, lse, dl, workspace=ws)
    for new in (labels, labels.flip(0), torch.where(torch.arange(700, device="cuda") % 11 == 0,
                                                    labels, -1), torch.full_like(labels, -1)):
        lab.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        eager = bb.bb_linear_ce_bwd(h, w, None, new.to(torch.int32), lse, dl)
        assert torch.equal(got[0], eager[0]) and torch.equal(got[1], eager[1])
