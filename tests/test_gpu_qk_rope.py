"""GPU parity of the per-head norm with the rotary rotation against the fp64
oracle.

Tolerance, from the arithmetic.  Forward: y = r (x gamma_a cos - x' gamma_b
sin).  The sum of 64 squares takes 8 fused steps and 3 adds (11 x 2^-24,
halved by the root), rsqrtf is within 2 units (2^-22), the angle within
pi 2^-24, cos and sin within 2 units, the products one rounding each: below
2^-19 of |u_a| + |u_b| <= 2 max|u| together; the result is rounded once to
the dtype (eps / 2 of its value).  Backward, with v = gamma g and n = x r:
dx = r (v - n mean(v n)) is within 2^-18 of r (max|v| + max|n| mean|v n|) by
the same count (g carries the rotation's error, the mean 11 more roundings).
dgamma is a sum of fp32 terms of relative error 2^-19, added in a tree whose
longest path has at most 200 adds here: 2^-16 sum |g n| bounds both."""

import numpy as np
import pytest
import torch

import oracle
from block_sparse_long_bwd_b200 import binding as bb

pytestmark = pytest.mark.gpu


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _inputs(B, H, L, dtype, seed, gammas=True, pos=None):
    g = torch.Generator().manual_seed(seed)
    t = [(1.5 * torch.randn((B, H, L, 64), generator=g)).to(dtype).cuda() for _ in range(4)]
    gam = [(1 + 0.3 * torch.randn(64, generator=g)).cuda() if gammas else None for _ in range(2)]
    return t, gam, pos


def _check_fwd(y, x, gamma, pos, args):
    ref = oracle.qk_norm_rope(_np(x), _np(gamma), pos, *args)
    u = oracle.qk_norm_rope(_np(x), _np(gamma), pos, args[0], args[1], 0, False)
    tol = (torch.finfo(y.dtype).eps / 2 * np.abs(ref)
           + 2.0**-18 * np.abs(u).max(-1, keepdims=True))
    err = np.abs(_np(y) - ref)
    assert (err <= tol).all(), (err - tol).max()


def _check_bwd(dx, dgamma, x, gamma, pos, dy, args):
    x64, gam = _np(x), np.ones(64) if gamma is None else _np(gamma)
    ref, refg = oracle.qk_norm_rope_backward(x64, gam, pos, _np(dy), *args)
    g, _ = oracle.qk_norm_rope_backward(np.full_like(x64, 0.0), None, pos, _np(dy), 1.0, *args[1:])
    r = 1 / np.sqrt((x64**2).mean(-1, keepdims=True) + args[0])
    v, n = gam * g, x64 * r
    m = r * (np.abs(v).max(-1, keepdims=True)
             + np.abs(n).max(-1, keepdims=True) * np.abs(v * n).mean(-1, keepdims=True))
    tol = torch.finfo(dx.dtype).eps / 2 * np.abs(ref) + 2.0**-18 * m
    err = np.abs(_np(dx) - ref)
    assert (err <= tol).all(), (err - tol).max()
    errg = np.abs(_np(dgamma) - refg)
    assert (errg <= 2.0**-16 * np.abs(g * n).sum((0, 1, 2))).all(), errg.max()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,H,L,rot,inter", [
    (1, 1, 1, 64, False), (1, 12, 1, 64, True), (2, 3, 31, 64, False), (1, 2, 33, 32, False),
    (3, 1, 45, 16, False), (1, 4, 17, 48, False), (2, 2, 19, 24, False), (1, 3, 29, 2, False),
    (1, 3, 29, 62, True), (2, 5, 40, 0, False), (2, 12, 257, 64, False), (1, 16, 130, 64, True)])
def test_forward_and_backward(B, H, L, rot, inter, dtype):
    t, gam, _ = _inputs(B, H, L, dtype, L + rot)
    pos = torch.randint(-5000, 200000, (B, L), generator=torch.Generator().manual_seed(L),
                        dtype=torch.int32)
    for p in (None, pos):
        desc = bb.make_qk_desc(B, H, L, dtype, eps=1e-6, theta=10000.0, rot_dim=rot,
                               interleaved=inter)
        args = (float(np.float32(1e-6)), 10000.0, rot, inter)
        pc, pn = (None, None) if p is None else (p.cuda(), p.numpy())
        y = bb.bb_qk_norm_rope_fwd(desc, t[0], t[1], *gam, pc)
        for i in range(2):
            _check_fwd(y[i], t[i], gam[i], pn, args)
        out = bb.bb_qk_norm_rope_bwd(desc, t[0], t[1], *gam, pc, t[2], t[3])
        for i in range(2):
            _check_bwd(out[i], out[2 + i], t[i], gam[i], pn, t[2 + i], args)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,H,L,rot,inter", [
    (2, 5, 2111, 16, True), (1, 1, 19001, 64, False), (1, 3, 9500, 62, False),
    (1, 4, 6400, 64, True), (3, 7, 1100, 64, False)])
def test_a_block_walks_heads_of_both(B, H, L, rot, inter, dtype):
    """Enough tokens that a block's range of heads runs over several of them,
    odd numbers of q's and on into k's.  (dgamma: 2^-16 as above; 594 token
    blocks are 19 adds in each of 32 partial sums.)"""
    t, gam, _ = _inputs(B, H, L, dtype, L)
    desc = bb.make_qk_desc(B, H, L, dtype, rot_dim=rot, interleaved=inter)
    args = (float(np.float32(1e-6)), 10000.0, rot, inter)
    y = bb.bb_qk_norm_rope_fwd(desc, t[0], t[1], *gam)
    out = bb.bb_qk_norm_rope_bwd(desc, t[0], t[1], *gam, None, t[2], t[3])
    for i in range(2):
        _check_fwd(y[i], t[i], gam[i], None, args)
        _check_bwd(out[i], out[2 + i], t[i], gam[i], None, t[2 + i], args)


def test_far_positions_and_other_options():
    """The angle is reduced exactly: the largest positions are as good as
    the first (the oracle's fp64 angle is within 2^31 2^-53 of exact)."""
    t, gam, _ = _inputs(1, 2, 6, torch.float32, 5, gammas=False)
    pos = torch.tensor([[0, 1, 2**31 - 1, -(2**31), 123456789, 2**24 + 1]], dtype=torch.int32)
    for theta, eps, rot, inter in ((10000.0, 0.0, 64, False), (500000.0, 1e-3, 64, True),
                                   (1.0, 1e-6, 20, False)):
        desc = bb.make_qk_desc(1, 2, 6, torch.float32, eps=eps, theta=theta, rot_dim=rot,
                               interleaved=inter)
        y = bb.bb_qk_norm_rope_fwd(desc, t[0], t[1], None, None, pos.cuda())
        _check_fwd(y[0], t[0], None, pos.numpy(), (float(np.float32(eps)), theta, rot, inter))


def test_gradient_against_differences():
    """<dy, y(x + h e) - y(x - h e)> / 2h in fp64 of the fp32 outputs: the
    outputs carry 2^-18 each, so with h = 2^-4 and 64 components the quotient
    is within 64 2^-18 / 2^-3 + the cubic term (h^2 times a third derivative
    below 40 for unit rows)."""
    t, gam, _ = _inputs(1, 1, 3, torch.float32, 8)
    desc = bb.make_qk_desc(1, 1, 3, torch.float32)
    dx = bb.bb_qk_norm_rope_bwd(desc, t[0], t[1], *gam, None, t[2], t[3])[0]
    h = 2.0**-4
    for j in (0, 7, 31, 32, 63):
        f = []
        for s in (h, -h):
            x = t[0].clone()
            x[..., j] += s
            y = bb.bb_qk_norm_rope_fwd(desc, x, t[1], *gam, None)[0]
            f.append((y.double() * t[2].double()).sum(-1))
        diff = (f[0] - f[1]) / (2 * h)
        assert (diff - dx[..., j].double()).abs().max().item() <= 64 * 2.0**-15 + 40 * h * h


def test_zero_rows_and_infinite_rows():
    """A row of zeros has outputs and gradients by eps alone; an infinity
    stays in its own row."""
    t, gam, _ = _inputs(1, 2, 8, torch.float32, 6)
    t[0][0, 0, 3] = 0.0
    t[0][0, 1, 5, 9] = float("inf")
    desc = bb.make_qk_desc(1, 2, 8, torch.float32)
    y = bb.bb_qk_norm_rope_fwd(desc, t[0], t[1], *gam)[0]
    assert (y[0, 0, 3] == 0).all()
    dq = bb.bb_qk_norm_rope_bwd(desc, t[0], t[1], *gam, None, t[2], t[3])[0]
    ok = torch.ones(1, 2, 8, dtype=torch.bool)
    ok[0, 1, 5] = False
    assert torch.isfinite(y[ok.cuda()]).all() and torch.isfinite(dq[ok.cuda()]).all()


@pytest.mark.parametrize("rot", [64, 24])
def test_in_place_streams_and_graph(rot):
    B, H, L = 2, 4, 100
    t, gam, _ = _inputs(B, H, L, torch.bfloat16, 9)
    desc = bb.make_qk_desc(B, H, L, torch.bfloat16, rot_dim=rot)
    want = bb.bb_qk_norm_rope_fwd(desc, t[0], t[1], *gam)
    q, k = t[0].clone(), t[1].clone()
    bb.bb_qk_norm_rope_fwd(desc, q, k, *gam, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    wantb = bb.bb_qk_norm_rope_bwd(desc, t[0], t[1], *gam, None, t[2], t[3])
    a, b = t[2].clone(), t[3].clone()
    got = bb.bb_qk_norm_rope_bwd(desc, t[0], t[1], *gam, None, a, b, dq=a, dk=b)
    assert all(torch.equal(x, y) for x, y in zip(got, wantb))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = bb.bb_qk_norm_rope_bwd(desc, t[0], t[1], *gam, None, t[2], t[3], stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, wantb))
    # two captured calls share one workspace in order
    ws = torch.empty(bb.bb_qk_norm_rope_workspace_size(desc), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g1 = bb.bb_qk_norm_rope_bwd(desc, t[0], t[1], *gam, None, t[2], t[3], workspace=ws)
        g2 = bb.bb_qk_norm_rope_bwd(desc, t[1], t[0], *gam, None, t[3], t[2], workspace=ws)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(g1, wantb))
    assert torch.equal(g2[0], bb.bb_qk_norm_rope_bwd(desc, t[1], t[0], *gam, None, t[3], t[2])[0])


def test_offsets_past_32_bits():
    L = (1 << 25) + 9  # 64 L elements per head pass 2^31
    q = torch.zeros((1, 1, L, 64), dtype=torch.bfloat16, device="cuda")
    q[0, 0, -5:] = torch.randn(5, 64, generator=torch.Generator().manual_seed(1)).cuda()
    tail = q[:, :, -5:].clone()
    desc = bb.make_qk_desc(1, 1, L, torch.bfloat16)
    y = bb.bb_qk_norm_rope_fwd(desc, q, q, None, None)[0]
    pos = np.arange(L - 5, L)[None]
    _check_fwd(y[:, :, -5:], tail, None, pos, (float(np.float32(1e-6)), 10000.0, 64, False))
    del y
    dq = bb.bb_qk_norm_rope_bwd(desc, q, q, None, None, None, q, q)
    _check_bwd(dq[0][:, :, -5:], dq[2], tail, None, pos, tail,
               (float(np.float32(1e-6)), 10000.0, 64, False))
