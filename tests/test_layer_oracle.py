"""Pins of the oracle of the operators around the attention: output dropout
against the generator's bytes written out one by one, the norm with rotation
and the vocabulary cross entropy against torch fp64 autograd of a separate
formulation and central differences."""

import numpy as np
import pytest
import torch

import oracle


def test_out_dropout_bytes_one_by_one():
    seed, site, rate = 0xFEDCBA9876543210, 7, 0.3
    for start, n in ((0, 40), (5, 27), ((1 << 36) - 8, 24), (1 << 40, 17)):
        keep = oracle.out_dropout_keep(seed, site, rate, n, start)
        for k in range(n):
            i = start + k
            w = oracle.philox4x32_10((i >> 4 & 0xFFFFFFFF, i >> 36, site, 0xFFFFFFFF),
                                     (seed & 0xFFFFFFFF, seed >> 32))
            raw = b"".join(int(x).to_bytes(4, "little") for x in w)
            assert keep[k] == (raw[i & 15] >= oracle.dropout_threshold(rate)), (start, k)


def test_out_dropout_mean_and_rate():
    """Kept share within 5 standard deviations of the rounded rate, and the
    sum unbiased by its scale."""
    n, rate = 1 << 16, 0.1
    keep = oracle.out_dropout_keep(11, 0, rate, n)
    p = 1 - oracle.dropout_threshold(rate) / 256
    assert abs(keep.mean() - p) < 5 * np.sqrt(p * (1 - p) / n)
    y = oracle.out_dropout(np.ones(n), np.full(n, 2.0), rate, 11, 0)
    assert np.array_equal(y, np.where(keep, 2.0 + 1.0 / p, 2.0))
    assert np.array_equal(oracle.out_dropout(np.arange(9.0), None, 0.0, 5, 1), np.arange(9.0))


def _torch_qk(x, gamma, pos, eps, theta, rot, interleaved):
    """The rotation as a complex product, the norm by torch's own functions."""
    n = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps) * gamma
    f = torch.tensor(theta, dtype=torch.float64) ** (
        -torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    turn = torch.polar(torch.ones((), dtype=torch.float64), pos.double()[:, None, :, None] * f)
    r = n[..., :rot]
    if interleaved:
        z = torch.view_as_complex(r.unflatten(-1, (rot // 2, 2)).contiguous()) * turn
        r = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(r[..., : rot // 2].contiguous(), r[..., rot // 2:].contiguous()) * turn
        r = torch.cat([z.real, z.imag], -1)
    return torch.cat([r, n[..., rot:]], -1)


@pytest.mark.parametrize("rot,interleaved", [(8, False), (8, True), (4, False), (6, True), (2, False)])
def test_qk_matches_autograd(rot, interleaved):
    g = torch.Generator().manual_seed(rot)
    x = torch.randn((2, 3, 5, 8), generator=g, dtype=torch.float64, requires_grad=True)
    gamma = torch.rand(8, generator=g, dtype=torch.float64, requires_grad=True)
    dy = torch.randn((2, 3, 5, 8), generator=g, dtype=torch.float64)
    pos = torch.randint(-9, 1000, (2, 5), generator=g)
    y = _torch_qk(x, gamma, pos, 1e-5, 500.0, rot, interleaved)
    y.backward(dy)
    args = (1e-5, 500.0, rot, interleaved)
    got = oracle.qk_norm_rope(x.detach(), gamma.detach(), pos, *args)
    assert np.abs(got - y.detach().numpy()).max() < 1e-12
    dx, dg = oracle.qk_norm_rope_backward(x.detach(), gamma.detach(), pos, dy, *args)
    assert np.abs(dx - x.grad.numpy()).max() < 1e-11
    assert np.abs(dg - gamma.grad.numpy()).max() < 1e-11


def test_qk_keeps_the_norm_and_finite_differences():
    r = np.random.default_rng(3)
    x, dy = r.standard_normal((1, 1, 2, 8)), r.standard_normal((1, 1, 2, 8))
    args = (1e-6, 100.0, 8, False)
    y = oracle.qk_norm_rope(x, None, None, *args)
    assert np.allclose((y**2).mean(-1), 1.0, atol=1e-4)  # a rotation keeps the RMS
    dx, _ = oracle.qk_norm_rope_backward(x, None, None, dy, *args)
    for k in range(16):
        e = np.zeros(16)
        e[k] = 1e-6
        e = e.reshape(x.shape)
        f = [(oracle.qk_norm_rope(x + s * e, None, None, *args) * dy).sum() for s in (1, -1)]
        assert abs((f[0] - f[1]) / 2e-6 - dx.reshape(-1)[k]) < 1e-7


@pytest.mark.parametrize("N,D,V,bias", [(5, 4, 7, True), (1, 3, 1, False), (4, 6, 11, True)])
def test_linear_ce_matches_torch_and_differences(N, D, V, bias):
    g = torch.Generator().manual_seed(N * 10 + V)
    h = torch.randn((N, D), generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn((V, D), generator=g, dtype=torch.float64, requires_grad=True)
    b = torch.randn(V, generator=g, dtype=torch.float64, requires_grad=True) if bias else None
    labels = torch.randint(0, V, (N,), generator=g)
    labels[N // 2] = -100 if N > 1 else labels[0]
    up = torch.rand(N, generator=g, dtype=torch.float64)
    z = torch.nn.functional.linear(h, w, b)
    loss = torch.nn.functional.cross_entropy(z, labels, reduction="none", ignore_index=-100)
    loss.backward(up)
    hd, wd, bd = (None if t is None else t.detach().numpy() for t in (h, w, b))
    got, lse = oracle.linear_ce(hd, wd, bd, labels.numpy())
    assert np.abs(got - loss.detach().numpy()).max() < 1e-12
    grads = oracle.linear_ce_backward(hd, wd, bd, labels.numpy(), lse, up.numpy())
    for want, have in zip((h, w, b), grads):
        if want is not None:
            assert np.abs(have - want.grad.numpy()).max() < 1e-12
    for k in range(min(6, V * D)):
        e = np.zeros(V * D)
        e[k] = 1e-6
        f = [(oracle.linear_ce(hd, wd + s * e.reshape(V, D), bd, labels.numpy())[0]
              * up.numpy()).sum() for s in (1, -1)]
        assert abs((f[0] - f[1]) / 2e-6 - grads[1].reshape(-1)[k]) < 1e-8


def test_linear_ce_rows_without_a_label_and_masked_words():
    h = np.array([[1.0, 2.0], [np.nan, np.inf], [0.5, -1.0]])
    w = np.array([[1.0, 0.0], [0.0, 1.0], [1.0, 1.0]])
    bias = np.array([0.0, -np.inf, 0.0])  # the second word is excluded
    loss, lse = oracle.linear_ce(h, w, bias, [2, -1, 3])
    assert np.array_equal(loss[1:], [0, 0]) and np.array_equal(lse[1:], [0, 0])
    assert abs(lse[0] - np.log(np.exp(1.0) + np.exp(3.0))) < 1e-15
    dh, dw, db = oracle.linear_ce_backward(h, w, bias, [2, -1, 3], lse, np.ones(3))
    assert np.isfinite(dh).all() and np.isfinite(dw).all() and not dh[1:].any()
    assert db[1] == 0 and not dw[1].any() and abs(db.sum()) < 1e-15
