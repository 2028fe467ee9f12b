"""GPU parity of the vocabulary projection's cross entropy and its gradients
against the definition in 64 bits.

Exact cases: h uses features that w leaves at zero, so every logit is the
bias (0), and lse = 0 makes every probability 1; dz, dh, dw and dbias are then
sums of small integers, exact in fp32, and the results must be equal to them
rounded once.  They check every tile, piece, split and packed row.

General cases, bounds from the arithmetic.  A logit is an fp32 sum of D exact
products: off by at most D 2^-23 sum|h w| (ez).  lse: ez, plus 2^-22 for the
exponential, at most 256 + V / 256 additions of 2^-24, the logarithm and the
final sum 2^-22 |lse|; the loss once more ez.  exp(z - lse) is off by the
factor e = ez + 2^-22 |z - lse| + 2^-21; dz = dloss (p - y) by dloss p e, then
by bf16's 2^-8 of itself.  So with A = |dz|, P = |dloss| p, element by
element: dw within 2^-8 |dw| + (2^-8 + R 2^-23) A^T |h| + P^T (e |h|), dh the
same with w and V, dbias within R 2^-23 sum A + sum P e."""

import numpy as np
import pytest
import torch

import oracle
from block_sparse_long_bwd_b200 import binding as bb

pytestmark = pytest.mark.gpu


def _ws(N, D, V, p, fill=0xFF):
    """Workspaces start as NaN patterns: nothing may depend on their contents."""
    return torch.full((bb.bb_linear_ce_workspace_size(N, D, V, p),), fill, dtype=torch.uint8,
                      device="cuda")


def _labels(N, V, share, g):
    labels = torch.randint(0, V, (N,), generator=g)
    labels[torch.rand(N, generator=g) >= share] = -100
    return labels.to(torch.int32)


@pytest.mark.parametrize("N,D,V,share", [
    (1, 64, 1, 1.0), (1, 64, 300, 1.0), (3, 72, 257, 0.6), (128, 128, 256, 1.0),
    (129, 136, 1000, 1.0), (200, 256, 511, 0.4), (700, 320, 1537, 0.9), (64, 768, 5003, 1.0),
    (300, 776, 20011, 0.3), (2500, 64, 4096, 1.0), (257, 1024, 9001, 0.0),
    (100, 200, 3001, 0.0), (1, 64, 40, 0.0), (128, 512, 30011, 0.5), (65, 1544, 700, 1.0),
    (40003, 64, 300, 0.7)])
def test_exact_integer_gradients(N, D, V, share):
    g = torch.Generator().manual_seed(N + V)
    half = D // 2
    h, w = torch.zeros(N, D), torch.zeros(V, D)
    h[:, :half] = torch.randint(-2, 3, (N, half), generator=g).float()
    w[:, half:] = torch.randint(-2, 3, (V, D - half), generator=g).float()
    labels = _labels(N, V, share, g)
    dl = torch.tensor([1.0, 2.0])[torch.randint(0, 2, (N,), generator=g)]
    h[labels < 0] = float("nan")  # rows without a label enter nothing
    dl[labels < 0] = float("nan")
    ws = _ws(N, D, V, 1)
    c = lambda t: t.cuda()
    dh, dw, db = bb.bb_linear_ce_bwd(c(h.bfloat16()), c(w.bfloat16()), torch.zeros(V, device="cuda"),
                                     c(labels), torch.zeros(N, device="cuda"), c(dl), workspace=ws)
    assert bb.bb_attn_check_status(ws) == 0
    rows = (labels >= 0).nonzero()[:, 0]
    dz = dl[rows, None].double() * (1.0 - torch.nn.functional.one_hot(labels[rows].long(), V))
    want = torch.zeros(N, D, dtype=torch.float64)
    want[rows] = dz @ w.double()
    assert torch.equal(dh.cpu(), want.float().bfloat16())
    assert torch.equal(dw.cpu(), (dz.t() @ h[rows].double()).float().bfloat16())
    assert torch.equal(db.cpu(), dz.sum(0).float())


def _general(N, D, V, share, bias, seed, scale=0.5):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(N, D, generator=g)
    w = torch.randn(V, D, generator=g) * (4 * scale / D**0.5)
    labels = _labels(N, V, share, g)
    lean = torch.rand(N, 1, generator=g) * 2
    h = (h + lean * w[labels.clamp(0).long()] / scale).bfloat16()
    b = torch.randn(V, generator=g) if bias else None
    dl = torch.rand(N, generator=g) + 0.5
    return h, w.bfloat16(), b, labels, dl


def _check_general(h, w, b, labels, dl, loss, lse, grads):
    """Rows with a label against fp64 on the GPU."""
    N, D = h.shape
    V = w.shape[0]
    rows = (labels >= 0).nonzero()[:, 0].cuda()
    R = rows.numel()
    d = lambda t: t.cuda().double()
    hr, wd, lab = d(h)[rows], d(w), labels.cuda()[rows].long()
    z = hr @ wd.t() + (0 if b is None else d(b))
    ez = D * 2.0**-23 * (hr.abs() @ wd.abs().t())
    ref = z.logsumexp(1)
    el = ez.amax(1) + 2.0**-22 + (256 + V / 256) * 2.0**-24 + 2.0**-22 * ref.abs()
    assert ((d(lse)[rows] - ref).abs() <= el).all()
    at = z.gather(1, lab[:, None])[:, 0]
    assert ((d(loss)[rows] - (ref - at)).abs()
            <= el + ez.amax(1) + 2.0**-22 * (ref.abs() + at.abs())).all()
    out = torch.ones(N, dtype=torch.bool, device="cuda")
    out[rows] = False
    assert not loss[out].any() and not lse[out].any()
    if grads is None:
        return
    dh, dw, db = grads
    l64 = d(lse)[rows, None]  # the backward's input
    p = (z - l64).exp()
    e = ez + 2.0**-22 * (z - l64).abs() + 2.0**-21
    dlr = d(dl)[rows, None]
    dz = dlr * (p - torch.nn.functional.one_hot(lab, V))
    A, Pe = dz.abs(), dlr * p * e
    want = dz @ wd
    tol = 2.0**-8 * want.abs() + (2.0**-8 + V * 2.0**-23) * (A @ wd.abs()) + Pe @ wd.abs()
    assert ((d(dh)[rows] - want).abs() <= tol).all()
    assert not dh[out].any()
    want = dz.t() @ hr
    tol = 2.0**-8 * want.abs() + (2.0**-8 + R * 2.0**-23) * (A.t() @ hr.abs()) + Pe.t() @ hr.abs()
    assert ((d(dw) - want).abs() <= tol).all()
    if b is not None:
        assert ((d(db) - dz.sum(0)).abs() <= (R + 8) * 2.0**-23 * A.sum(0) + Pe.sum(0)).all()
    else:
        assert db is None


@pytest.mark.parametrize("N,D,V,share,bias", [
    (1, 64, 1, 1.0, True), (1, 768, 30011, 1.0, False), (5, 200, 31, 0.5, True),
    (77, 776, 3001, 0.9, True), (128, 64, 512, 1.0, False), (500, 1024, 8191, 0.15, True),
    (1111, 768, 12345, 1.0, True), (4096, 512, 2000, 1.0, False), (3000, 128, 50021, 0.7, True)])
def test_loss_and_gradients(N, D, V, share, bias):
    h, w, b, labels, dl = _general(N, D, V, share, bias, N + D)
    if share < 1 and N > 1:
        labels[0] = 0
        h[labels < 0] = float("inf")
    c = lambda t: None if t is None else t.cuda()
    wf, wb = _ws(N, D, V, 0), _ws(N, D, V, 1)
    loss, lse = bb.bb_linear_ce_fwd(c(h), c(w), c(b), c(labels), workspace=wf)
    grads = bb.bb_linear_ce_bwd(c(h), c(w), c(b), c(labels), lse, c(dl), workspace=wb)
    assert bb.bb_attn_check_status(wf) == 0 and bb.bb_attn_check_status(wb) == 0
    _check_general(h, w, b, labels, dl, loss, lse, grads)
    # run to run the same bits
    again = bb.bb_linear_ce_bwd(c(h), c(w), c(b), c(labels), lse, c(dl))
    assert all(x is y or torch.equal(x, y) for x, y in zip(again, grads))


@pytest.mark.parametrize("N,D,V,share,bias", [
    (1, 288, 4321, 1.0, False), (5, 744, 753, 0.5, True), (7, 408, 42639, 0.5, True),
    (63, 64, 300, 1.0, False), (64, 768, 5003, 1.0, True), (100, 200, 2001, 0.3, True),
    (900, 136, 1999, 0.05, True)])
def test_few_rows_are_as_exact_as_their_rounding(N, D, V, share, bias):
    """Up to 64 rows with a label, dz is carried in two bf16 parts, the second
    the rest of the first: 2^-16 of it is left, not 2^-8.  Otherwise the
    bounds of the general case, and of dbias.  Weights spread over a factor of
    256 let single rows lead."""
    h, w, b, labels, _ = _general(N, D, V, share, bias, N + V)
    labels[N // 2] = V // 3
    g = torch.Generator().manual_seed(N)
    dl = torch.exp2(8 * torch.rand(N, generator=g))
    c = lambda t: None if t is None else t.cuda()
    loss, lse = bb.bb_linear_ce_fwd(c(h), c(w), c(b), c(labels))
    dh, dw, db = bb.bb_linear_ce_bwd(c(h), c(w), c(b), c(labels), lse, c(dl),
                                     workspace=_ws(N, D, V, 1))
    rows = (labels >= 0).nonzero()[:, 0].cuda()
    R = rows.numel()
    assert 0 < R <= 64
    d = lambda t: t.cuda().double()
    hr, wd, lab = d(h)[rows], d(w), labels.cuda()[rows].long()
    z = hr @ wd.t() + (0 if b is None else d(b))
    ez = D * 2.0**-23 * (hr.abs() @ wd.abs().t())
    l64, dlr = d(lse)[rows, None], d(dl)[rows, None]
    p = (z - l64).exp()
    e = ez + 2.0**-22 * (z - l64).abs() + 2.0**-21
    dz = dlr * (p - torch.nn.functional.one_hot(lab, V))
    A, Pe = dz.abs(), dlr * p * e
    for got, x, left, K in ((d(dh)[rows], wd, lambda m: m, V),
                            (d(dw), hr, lambda m: m.t(), 2 * R)):
        want = left(dz) @ x
        tol = (2.0**-8 * want.abs() + (2.0**-16 + K * 2.0**-23) * (left(A) @ x.abs())
               + left(Pe) @ x.abs())
        assert ((got - want).abs() <= tol).all()
    if b is not None:
        assert ((d(db) - dz.sum(0)).abs() <= (2 * R + 8) * 2.0**-23 * A.sum(0) + Pe.sum(0)).all()


def test_against_the_oracle_and_differences():
    """The written-out oracle, and the loss's central differences along a few
    weights (h = 2^-3 on bf16 weights that are multiples of 2^-3, exact): the
    losses are within 2^-17 here, the cubic term below h^2."""
    N, D, V = 6, 64, 40
    g = torch.Generator().manual_seed(2)
    h = (torch.randint(-4, 5, (N, D), generator=g) / 8).bfloat16()
    w = (torch.randint(-8, 9, (V, D), generator=g) / 8).bfloat16()
    labels = torch.tensor([3, 39, 0, -1, 7, 7], dtype=torch.int32)
    dl = torch.rand(N, generator=g)
    f = lambda ww: bb.bb_linear_ce_fwd(h.cuda(), ww.cuda(), None, labels.cuda())
    loss, lse = f(w)
    rl, rs = oracle.linear_ce(h.double().numpy(), w.double().numpy(), None, labels.numpy())
    assert np.abs(loss.cpu().numpy() - rl).max() < 2.0**-17
    assert np.abs(lse.cpu().numpy() - rs).max() < 2.0**-17
    dh, dw, _ = bb.bb_linear_ce_bwd(h.cuda(), w.cuda(), None, labels.cuda(), lse, dl.cuda())
    eh, ew, _ = oracle.linear_ce_backward(h.double().numpy(), w.double().numpy(), None,
                                          labels.numpy(), rs, dl.numpy())
    for got, want in ((dh, eh), (dw, ew)):
        # 2^-8 of the terms' magnitudes: below 2^-8 (sum|dz| |w| or |h|) <= 2^-8 * 6
        assert np.abs(got.double().cpu().numpy() - want).max() < 6 * 2.0**-7
    for v, cidx in ((3, 0), (7, 11), (20, 63)):
        s = []
        for d in (0.125, -0.125):
            x = w.clone()
            x[v, cidx] += d
            s.append((f(x)[0].double().cpu() * dl.double()).sum())
        diff = (s[0] - s[1]) / 0.25
        assert abs(diff - ew[v, cidx]) < 2.0**-6 + 6 * 2.0**-15


def test_excluded_words_and_extreme_biases():
    N, D, V = 40, 64, 700
    h, w, b, labels, dl = _general(N, D, V, 1.0, True, 3)
    labels = (labels % 100).to(torch.int32)
    b[100:600] = float("-inf")       # whole 32-column blocks excluded
    b[650:] = torch.finfo(torch.float32).min
    c = lambda t: t.cuda()
    loss, lse = bb.bb_linear_ce_fwd(c(h), c(w), c(b), c(labels))
    dh, dw, db = bb.bb_linear_ce_bwd(c(h), c(w), c(b), c(labels), lse, c(dl))
    keep = torch.cat([torch.arange(100), torch.arange(600, 650)])
    ref = torch.logsumexp(h.double() @ w[keep].double().t() + b[keep].double(), 1)
    assert ((lse.double().cpu() - ref).abs() < 1e-3).all()
    for t in (loss, dh, dw, db):
        assert torch.isfinite(t).all()
    gone = torch.ones(V, dtype=torch.bool)
    gone[keep] = False
    assert not dw[gone.cuda()].any() and not db[gone.cuda()].any()
    # every word at the type's lowest value: a uniform distribution over them
    b2 = torch.full((V,), torch.finfo(torch.float32).min)
    loss, _ = bb.bb_linear_ce_fwd(c(torch.zeros_like(h)), c(w), c(b2), c(labels))
    assert torch.isfinite(loss).all()
    # every word excluded: no distribution, as in the plain formula
    loss, _ = bb.bb_linear_ce_fwd(c(h), c(w), torch.full((V,), -np.inf, device="cuda"), c(labels))
    assert torch.isnan(loss).all()


def test_labels_outside_the_vocabulary_are_flagged():
    h, w, b, labels, dl = _general(300, 64, 500, 0.8, True, 4)
    good = labels.clone()
    labels[5], labels[290] = 500, 2**31 - 1
    good[5] = good[290] = -1
    c = lambda t: t.cuda()
    ws = _ws(300, 64, 500, 0)
    got = bb.bb_linear_ce_fwd(c(h), c(w), c(b), c(labels), workspace=ws)
    assert bb.bb_attn_check_status(ws) == bb.BB_ERR_BAD_LABEL
    want = bb.bb_linear_ce_fwd(c(h), c(w), c(b), c(good), workspace=ws)
    assert bb.bb_attn_check_status(ws) == 0
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    ws = _ws(300, 64, 500, 1)
    got = bb.bb_linear_ce_bwd(c(h), c(w), c(b), c(labels), want[1], c(dl), workspace=ws)
    assert bb.bb_attn_check_status(ws) == bb.BB_ERR_BAD_LABEL
    want = bb.bb_linear_ce_bwd(c(h), c(w), c(b), c(good), want[1], c(dl), workspace=ws)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_upstream_scales_and_zeros():
    """Equal dloss of any size scales the gradients by it (to the rounding of
    the product); dloss of zeros gives zeros."""
    h, w, b, labels, _ = _general(200, 128, 900, 1.0, True, 6)
    c = lambda t: t.cuda()
    _, lse = bb.bb_linear_ce_fwd(c(h), c(w), c(b), c(labels))
    f = lambda s: bb.bb_linear_ce_bwd(c(h), c(w), c(b), c(labels), lse,
                                      torch.full((200,), s, device="cuda"))
    one = f(1.0)
    for s in (2.0**-20, -4.0, 2.0**60):
        for x, y in zip(f(s), one):
            assert torch.equal(x.float(), y.float() * s)
    assert not any(x.any() for x in f(0.0))


def test_streams_and_graphs():
    h, w, b, labels, dl = (t.cuda() for t in _general(333, 256, 3000, 0.5, True, 7))
    loss, lse = bb.bb_linear_ce_fwd(h, w, b, labels)
    want = bb.bb_linear_ce_bwd(h, w, b, labels, lse, dl)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    l2, s2 = bb.bb_linear_ce_fwd(h, w, b, labels, stream=side)
    g2 = bb.bb_linear_ce_bwd(h, w, b, labels, s2, dl, stream=side)
    side.synchronize()
    assert torch.equal(l2, loss) and all(torch.equal(x, y) for x, y in zip(g2, want))
    # a captured step: new labels, another number of rows with one, replayed
    ws = [_ws(333, 256, 3000, p) for p in (0, 1)]
    lab = labels.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gl, gs = bb.bb_linear_ce_fwd(h, w, b, lab, workspace=ws[0])
        gg = bb.bb_linear_ce_bwd(h, w, b, lab, gs, dl, workspace=ws[1])
    for new in (labels, labels.flip(0), torch.full_like(labels, -1), labels.abs() % 3000):
        lab.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        el, es = bb.bb_linear_ce_fwd(h, w, b, new)
        eg = bb.bb_linear_ce_bwd(h, w, b, new, es, dl)
        assert torch.equal(gl, el) and all(torch.equal(x, y) for x, y in zip(gg, eg))


def _guarded(shape, dtype):
    """A tensor between two guards of 4 KB, and a check that they are intact."""
    n = int(np.prod(shape))
    item = torch.empty(0, dtype=dtype).element_size()
    raw = torch.full((8192 + n * item,), 0x5A, dtype=torch.uint8, device="cuda")
    ok = lambda: bool((raw[:4096] == 0x5A).all() and (raw[4096 + n * item:] == 0x5A).all())
    return raw[4096:4096 + n * item].view(dtype).view(shape), ok


@pytest.mark.parametrize("N,D,V,share", [(5, 72, 131, 0.6), (128, 328, 1001, 1.0),
                                         (301, 136, 777, 0.5), (512, 64, 256, 1.0)])
def test_nothing_is_written_outside_the_buffers(N, D, V, share):
    h, w, b, labels, dl = (t.cuda() for t in _general(N, D, V, share, True, N))
    shapes = dict(loss=((N,), torch.float32), lse=((N,), torch.float32), dh=((N, D), torch.bfloat16),
                  dw=((V, D), torch.bfloat16), dbias=((V,), torch.float32),
                  wf=((bb.bb_linear_ce_workspace_size(N, D, V, 0),), torch.uint8),
                  wb=((bb.bb_linear_ce_workspace_size(N, D, V, 1),), torch.uint8))
    t = {n: _guarded(*v) for n, v in shapes.items()}
    keep = [x.clone() for x in (h, w, b, labels, dl)]
    bb.bb_linear_ce_fwd(h, w, b, labels, loss=t["loss"][0], lse=t["lse"][0], workspace=t["wf"][0])
    bb.bb_linear_ce_bwd(h, w, b, labels, t["lse"][0], dl, dh=t["dh"][0], dw=t["dw"][0],
                        dbias=t["dbias"][0], workspace=t["wb"][0])
    torch.cuda.synchronize()
    assert all(ok() for _, ok in t.values())
    assert all(torch.equal(x, y) for x, y in zip(keep, (h, w, b, labels, dl)))
    loss, lse = bb.bb_linear_ce_fwd(h, w, b, labels)
    assert torch.equal(loss, t["loss"][0]) and torch.equal(lse, t["lse"][0])


def test_workspace_aligned_to_16_bytes_only():
    h, w, b, labels, dl = (t.cuda() for t in _general(90, 128, 1000, 0.8, True, 5))
    loss, lse = bb.bb_linear_ce_fwd(h, w, b, labels)
    want = bb.bb_linear_ce_bwd(h, w, b, labels, lse, dl)
    for off in (16, 240, 272):
        ws = [torch.full((bb.bb_linear_ce_workspace_size(90, 128, 1000, p) + off,), 0xFF,
                         dtype=torch.uint8, device="cuda")[off:] for p in (0, 1)]
        got = bb.bb_linear_ce_fwd(h, w, b, labels, workspace=ws[0])
        assert torch.equal(got[0], loss) and torch.equal(got[1], lse)
        got = bb.bb_linear_ce_bwd(h, w, b, labels, lse, dl, workspace=ws[1])
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert bb.bb_attn_check_status(ws[1]) == 0
