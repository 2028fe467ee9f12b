"""The operators around the attention at the largest sizes that they accept,
and called from several host threads at once."""

import threading

import pytest
import torch

from block_sparse_long_bwd_b200 import binding as bb
from test_gpu_linear_ce import _check_general, _general

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,D,V,share", [(3, 65536, 300, 1.0), (100, 65536, 513, 0.9),
                                         (300, 65536, 257, 0.7), (1100, 8200, 1001, 0.9),
                                         (200, 8192, 3001, 1.0)])
def test_wide_rows(N, D, V, share):
    h, w, b, labels, dl = _general(N, D, V, share, True, N + D)
    c = lambda t: t.cuda()
    loss, lse = bb.bb_linear_ce_fwd(c(h), c(w), c(b), c(labels))
    grads = bb.bb_linear_ce_bwd(c(h), c(w), c(b), c(labels), lse, c(dl))
    _check_general(h, w, b, labels, dl, loss, lse, grads)


@pytest.mark.parametrize("N,V,labelled", [(3, 1 << 24, 3), (70, 1 << 24, 70), (200, 1 << 24, 150),
                                          (1 << 20, 130, 1 << 20), (1 << 20, 513, 40)])
def test_most_rows_and_words(N, V, labelled):
    """Every logit is 0 (h uses features that w leaves at zero): the forward's
    lse is log V, and with lse = 0 the gradients are sums of integers whose
    partial sums stay below 2^24, exact."""
    D = 64
    g = torch.Generator(device="cuda").manual_seed(V)
    h = torch.zeros(N, D, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    h[:, :32] = torch.randint(-2, 3, (N, 32), generator=g, device="cuda").bfloat16()
    w[:, 32:] = torch.randint(-2, 3, (V, 32), generator=g, device="cuda").bfloat16()
    labels = torch.full((N,), -1, dtype=torch.int32, device="cuda")
    on = torch.randperm(N, generator=g, device="cuda")[:labelled].sort().values
    labels[on] = torch.randint(0, V, (labelled,), generator=g, device="cuda", dtype=torch.int32)
    labels[on[0]], labels[on[-1]] = 0, V - 1
    lab = labels[on].long()
    ws = [torch.full((bb.bb_linear_ce_workspace_size(N, D, V, p),), 0xFF, dtype=torch.uint8,
                     device="cuda") for p in (0, 1)]
    loss, lse = bb.bb_linear_ce_fwd(h, w, None, labels, workspace=ws[0])
    assert bb.bb_attn_check_status(ws[0]) == 0
    ref = torch.tensor(float(V), dtype=torch.float64).log().item()
    # V terms of 1 are summed exactly up to 2^24; the logarithm leaves 2^-22
    assert ((lse[on].double() - ref).abs() <= 2.0**-22 * ref + 2.0**-23).all()
    assert torch.equal(loss, lse) and not loss[labels < 0].any()
    dl = torch.ones(N, device="cuda")
    dh, dw, db = bb.bb_linear_ce_bwd(h, w, torch.zeros(V, device="cuda"), labels,
                                     torch.zeros(N, device="cuda"), dl, workspace=ws[1])
    assert bb.bb_attn_check_status(ws[1]) == 0
    want = torch.zeros(N, D, dtype=torch.float64, device="cuda")
    want[on] = w.sum(0, dtype=torch.float64) - w[lab].double()
    assert torch.equal(dh, want.float().bfloat16())
    H = h[on].double()
    full = H.sum(0).expand(V, D).clone().index_add_(0, lab, -H)
    assert torch.equal(dw, full.float().bfloat16())
    count = torch.full((V,), float(labelled), dtype=torch.float64, device="cuda")
    assert torch.equal(db, count.index_add_(0, lab, -torch.ones_like(lab, dtype=torch.float64))
                       .float())


def test_several_host_threads():
    """Four threads, each with its own stream, inputs and sizes, at once: the
    bits of one at a time."""
    cases = []
    for i, (N, D, V) in enumerate(((40, 128, 900), (100, 264, 2001), (700, 64, 1500),
                                   (1500, 200, 700))):
        h, w, b, labels, dl = (t.cuda() for t in _general(N, D, V, 0.9, True, i))
        q, k = (torch.randn(2, 3, N, 64, device="cuda").bfloat16() for _ in range(2))
        cases.append((h, w, b, labels, dl, q, k, bb.make_qk_desc(2, 3, N, torch.bfloat16)))

    def step(case, stream):
        h, w, b, labels, dl, q, k, desc = case
        x = bb.bb_dropout_fwd(h, h, 0.1, 5, 1, stream=stream)
        loss, lse = bb.bb_linear_ce_fwd(x, w, b, labels, stream=stream)
        out = bb.bb_linear_ce_bwd(x, w, b, labels, lse, dl, stream=stream)
        qk = bb.bb_qk_norm_rope_fwd(desc, q, k, None, None, stream=stream)
        return (x, loss, lse, *out, *qk,
                *bb.bb_qk_norm_rope_bwd(desc, q, k, None, None, None, *qk, stream=stream))

    want = [step(c, None) for c in cases]
    torch.cuda.synchronize()
    got, errors = [None] * len(cases), []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            for _ in range(20):
                got[i] = step(cases[i], stream)
            stream.synchronize()
        except Exception as e:  # reported by the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
