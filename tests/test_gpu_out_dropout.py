"""GPU parity of the output dropout against the fp64 oracle.

Tolerance, from the arithmetic: the scale 256 / (256 - thr) is rounded to
fp32 (2^-24 relative), the product and the sum are one fused operation
rounded to fp32, and the result is rounded once to the dtype: an element is
off by at most eps / 2 of its value (bf16 2^-8, fp32 2^-24) plus
2^-23 (|x| scale + |residual|)."""

import numpy as np
import pytest
import torch

import oracle
from block_sparse_long_bwd_b200 import binding as bb

pytestmark = pytest.mark.gpu
SEED = 0xFEDCBA9876543210


def _np(t):
    return t.double().cpu().numpy()


def _check(got, x, residual, rate, seed, site):
    ref = oracle.out_dropout(_np(x), None if residual is None else _np(residual), rate, seed, site)
    mag = np.abs(_np(x)) * oracle.dropout_scale(rate)
    if residual is not None:
        mag = mag + np.abs(_np(residual))
    err = np.abs(_np(got) - ref)
    tol = torch.finfo(got.dtype).eps / 2 * np.abs(ref) + 2.0**-23 * mag
    assert (err <= tol).all(), (err - tol).max()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [1, 15, 16, 17, 4096, 256 * 16 + 1, 100003])
@pytest.mark.parametrize("residual", [True, False])
def test_forward_and_backward(n, dtype, residual):
    g = torch.Generator().manual_seed(n)
    x, r, d = (torch.randn(n, generator=g).to(dtype).cuda() for _ in range(3))
    r = r if residual else None
    # The element behind the last stays as it was.
    buf = torch.full((n + 1,), 7.0, dtype=dtype, device="cuda")
    bb.bb_dropout_fwd(x, r, 0.1, SEED, 3, out=buf[:n])
    assert buf[n].item() == 7.0
    _check(buf[:n], x, r, 0.1, SEED, 3)
    _check(bb.bb_dropout_bwd(d, 0.1, SEED, 3), d, None, 0.1, SEED, 3)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tensors_aligned_to_16_bytes_only(dtype):
    """Every mixture of 16- and 32-byte alignment gives the same bits."""
    n, off = 5003, 16 // torch.finfo(dtype).bits * 8
    g = torch.Generator().manual_seed(4)
    base = [torch.randn(n, generator=g).to(dtype).cuda() for _ in range(2)]
    want = bb.bb_dropout_fwd(base[0], base[1], 0.1, 8)
    for which in range(8):
        t = []
        for k in range(3):
            buf = torch.empty(n + off, dtype=dtype, device="cuda")
            t.append(buf[off:] if which >> k & 1 else buf[:n])
        t[0].copy_(base[0])
        t[1].copy_(base[1])
        assert torch.equal(bb.bb_dropout_fwd(t[0], t[1], 0.1, 8, out=t[2]), want), which


@pytest.mark.parametrize("rate", [0.0, 0.001, 0.5, 255 / 256])
def test_rates(rate):
    x = torch.randn(3, 5, 771, device="cuda")
    _check(bb.bb_dropout_fwd(x, None, rate, 1, 0), x, None, rate, 1, 0)


def test_seed_and_site_give_other_decisions():
    one = torch.ones(65536, device="cuda")
    got = [bb.bb_dropout_fwd(one, None, 0.5, s, t) for s, t in ((1, 0), (1, 1), (2, 0), (1 << 63, 0))]
    for i in range(4):
        for j in range(i):
            assert 0.4 < (got[i] != got[j]).float().mean().item() < 0.6


def test_gradient_is_the_forwards_derivative():
    """The forward is linear in x: <dout, f(x) - f(0)> = <dx, x> in 64 bits
    (fp32 tensors: both sides within 2^-23 of the sum of magnitudes)."""
    x, d, r = (torch.randn(40001, device="cuda") for _ in range(3))
    dx = bb.bb_dropout_bwd(d, 0.25, 5, 2)
    y = bb.bb_dropout_fwd(x, None, 0.25, 5, 2)
    a, b = (d.double() * y.double()).sum(), (dx.double() * x.double()).sum()
    assert abs(a - b) <= 2.0**-22 * (d.double() * y.double()).abs().sum()
    # and the residual's derivative is dout itself: y rises with it one to one
    assert torch.equal(bb.bb_dropout_fwd(x, r, 0.25, 5, 2) == r, y == 0)


def test_dropped_infinities_and_nans_leave_no_trace():
    x = torch.full((4096,), float("nan"), device="cuda")
    x[::2] = float("inf")
    y = bb.bb_dropout_fwd(x, torch.ones_like(x), 0.5, 9, 0).cpu().numpy()
    keep = oracle.out_dropout_keep(9, 0, 0.5, 4096)
    assert (y[~keep] == 1.0).all() and not np.isfinite(y[keep]).any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_in_place(dtype):
    x, r = (torch.randn(12345, device="cuda").to(dtype) for _ in range(2))
    want = bb.bb_dropout_fwd(x, r, 0.1, 4)
    a, b = x.clone(), r.clone()
    assert torch.equal(bb.bb_dropout_fwd(a, r, 0.1, 4, out=a), want)
    assert torch.equal(bb.bb_dropout_fwd(x, b, 0.1, 4, out=b), want)
    d = x.clone()
    assert torch.equal(bb.bb_dropout_bwd(d, 0.1, 4, dx=d), bb.bb_dropout_bwd(x, 0.1, 4))


def test_side_stream_and_graph():
    x = torch.randn(1 << 20, device="cuda")
    want = bb.bb_dropout_fwd(x, x, 0.1, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = bb.bb_dropout_fwd(x, x, 0.1, 4, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bb.bb_dropout_fwd(x, x, 0.1, 4, out=out)
    x.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, bb.bb_dropout_fwd(x, x, 0.1, 4))


def test_elements_past_32_bits():
    n = (1 << 32) + 37
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    y = bb.bb_dropout_fwd(x, None, 0.25, 12, 1, out=x)
    for start in (0, (1 << 32) - 512):
        m = min(1024, n - start)
        want = oracle.out_dropout_keep(12, 1, 0.25, m, start)
        assert np.array_equal(y[start:start + m].float().cpu().numpy() != 0, want)
