"""The query/key norm and rotation where a block of the backward walks several
tiles of tokens (above 1024 x 32 of them) and several heads: partial sums of
the gamma gradients run over both.  Against the written-out formula in 64 bits
on the GPU; tolerances as in the other tests of the operator: forward and dx
2^-18 of the row's magnitudes beside the rounding, dgamma 2^-16 of sum |g n|
(two tiles x heads x 4 rows in a warp, 8 warps, then 1024 blocks in 32 sums of
32: below 200 additions on any path)."""

import pytest
import torch

from block_sparse_long_bwd_b200 import binding as bb

pytestmark = pytest.mark.gpu


def _rotation(L, rot, inter):
    """cos, sin [L, rot / 2] and the components of each pair."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    t = torch.arange(L, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (-2 * i / rot)
    j = torch.arange(rot // 2, device="cuda")
    return t.cos(), t.sin(), *((2 * j, 2 * j + 1) if inter else (j, j + rot // 2))


def _rotate(x, c, s, a, b):
    y = x.clone()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,H,L,rot,inter", [(2, 3, 20011, 64, False), (1, 2, 70001, 32, True),
                                             (3, 5, 11003, 20, False)])
def test_many_tiles_and_heads(B, H, L, rot, inter, dtype):
    g = torch.Generator(device="cuda").manual_seed(L)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    q, k, dq_out, dk_out = ((1.5 * r(B, H, L, 64)).to(dtype) for _ in range(4))
    gam = [1 + 0.3 * r(64) for _ in range(2)]
    eps = 2.0**-20
    desc = bb.make_qk_desc(B, H, L, dtype, eps=eps, rot_dim=rot, interleaved=inter)
    y = bb.bb_qk_norm_rope_fwd(desc, q, k, *gam)
    out = bb.bb_qk_norm_rope_bwd(desc, q, k, *gam, None, dq_out, dk_out)
    again = bb.bb_qk_norm_rope_bwd(desc, q, k, *gam, None, dq_out, dk_out)
    assert all(torch.equal(x, z) for x, z in zip(out, again))
    c, s, a, b = _rotation(L, rot, inter)
    half = torch.finfo(dtype).eps / 2
    for i, (x, dy) in enumerate(((q, dq_out), (k, dk_out))):
        x64, gm = x.double(), gam[i].double()
        rr = (x64.square().mean(-1, keepdim=True) + eps).rsqrt()
        u = gm * x64 * rr
        want = _rotate(u, c, s, a, b)
        tol = half * want.abs() + 2.0**-18 * u.abs().amax(-1, keepdim=True)
        assert ((y[i].double() - want).abs() <= tol).all()
        gg = _rotate(dy.double(), c, -s, a, b)
        n, v = x64 * rr, gm * gg
        want = rr * (v - n * (v * n).mean(-1, keepdim=True))
        m = rr * (v.abs().amax(-1, keepdim=True)
                  + n.abs().amax(-1, keepdim=True) * (v * n).abs().mean(-1, keepdim=True))
        assert ((out[i].double() - want).abs() <= half * want.abs() + 2.0**-18 * m).all()
        err = (out[2 + i].double() - (gg * n).sum((0, 1, 2))).abs()
        assert (err <= 2.0**-16 * (gg * n).abs().sum((0, 1, 2))).all()
