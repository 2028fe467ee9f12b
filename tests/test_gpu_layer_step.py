"""The operators around the attention in one training step, as a layer uses
them: projection -> query/key norm and rotation -> block-sparse attention ->
output projection -> dropout with the residual -> vocabulary cross entropy,
and all of it backward (the projections' own gradients are plain products
here).  Compared with torch fp64 autograd of the same step written with dense
attention (four blocks: every block attends every other one).

Tolerance: a result has passed at most a dozen bf16 roundings, each at most
2^-8 of what it rounds; with unit gains between them (normalised rows,
softmax, weights of unit row norm) their sum stays below 12 2^-8 = 0.047 of
the result's 2-norm."""

import numpy as np
import pytest
import torch

import oracle
from block_sparse_long_bwd_b200 import binding as bb

pytestmark = pytest.mark.gpu
B, L, hidden, H, V, RATE, SEED, SITE = 2, 256, 256, 4, 777, 0.1, 77, 5
D = H * 64
TOL = 12 * 2.0**-8


def _inputs():
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g)
    t = dict(x=r(B, L, hidden).bfloat16(), w_qkv=(r(3 * D, hidden) / hidden**0.5).bfloat16(),
             w_o=(r(hidden, D) / D**0.5).bfloat16(), gq=1 + 0.2 * r(64), gk=1 + 0.2 * r(64),
             w=(r(V, hidden) / hidden**0.5).bfloat16(), bias=0.3 * r(V))
    labels = torch.randint(0, V, (B * L,), generator=g)
    labels[torch.rand(B * L, generator=g) < 0.6] = -100  # masked-token training
    return t, labels.to(torch.int32)


class Step:
    """The step on the GPU with its buffers, as a user's program keeps them."""

    def __init__(self, t, labels):
        self.t = {n: v.cuda() for n, v in t.items()}
        self.labels = labels.cuda()
        self.att = bb.Attention(B, H, L, 64, 3, torch.bfloat16)
        self.desc = bb.make_qk_desc(B, H, L, torch.bfloat16)
        self.ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        self.dloss = torch.full((B * L,), 1.0 / int((labels >= 0).sum()), device="cuda")

    def run(self):
        t = self.t
        q, k, v = bb.bb_qkv_proj(t["x"], t["w_qkv"], None, H, self.ws)
        qr, kr = bb.bb_qk_norm_rope_fwd(self.desc, q, k, t["gq"], t["gk"])
        o, lse_a = self.att.forward(qr, kr, v)
        y = bb.bb_out_proj(o, t["w_o"], None, self.ws)
        h = bb.bb_dropout_fwd(y, t["x"], RATE, SEED, SITE)
        h2 = h.view(B * L, hidden)
        loss, lse = bb.bb_linear_ce_fwd(h2, t["w"], t["bias"], self.labels)
        dh, dw, db = bb.bb_linear_ce_bwd(h2, t["w"], t["bias"], self.labels, lse, self.dloss)
        dh = dh.view(B, L, hidden)
        dy = bb.bb_dropout_bwd(dh, RATE, SEED, SITE)
        do = (dy @ t["w_o"]).view(B, L, H, 64).transpose(1, 2).contiguous()
        dqr, dkr, dv = self.att.backward(qr, kr, v, o, lse_a, do)
        dq, dk, dgq, dgk = bb.bb_qk_norm_rope_bwd(self.desc, q, k, t["gq"], t["gk"], None, dqr, dkr)
        dqkv = torch.cat([z.transpose(1, 2).reshape(B, L, D) for z in (dq, dk, dv)], -1)
        dx = dh.float() + (dqkv @ t["w_qkv"]).float()
        return dict(loss=loss, dw=dw, dbias=db, dgq=dgq, dgk=dgk, dx=dx)


def _reference(t, labels):
    p = {n: v.double().requires_grad_() for n, v in t.items()}
    q, k, v = (z.view(B, L, H, 64).transpose(1, 2)
               for z in (p["x"] @ p["w_qkv"].t()).split(D, -1))
    ang = torch.arange(L, dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(32, dtype=torch.float64) / 32)
    turn = torch.polar(torch.ones_like(ang), ang)

    def norm_rope(z, gamma):
        u = z / torch.sqrt(z.pow(2).mean(-1, keepdim=True) + 1e-6) * gamma
        c = torch.complex(u[..., :32], u[..., 32:]) * turn
        return torch.cat([c.real, c.imag], -1)

    s = norm_rope(q, p["gq"]) @ norm_rope(k, p["gk"]).transpose(-1, -2) / 8
    o = (s.softmax(-1) @ v).transpose(1, 2).reshape(B, L, D)
    keep = torch.from_numpy(oracle.out_dropout_keep(SEED, SITE, RATE, B * L * hidden))
    y = o @ p["w_o"].t()
    h = p["x"] + y * keep.view(y.shape) * oracle.dropout_scale(RATE)
    z = h.view(B * L, hidden) @ p["w"].t() + p["bias"]
    loss = torch.nn.functional.cross_entropy(z, labels.long(), reduction="none",
                                             ignore_index=-100)
    loss.sum().div(int((labels >= 0).sum())).backward()
    return dict(loss=loss.detach(), dw=p["w"].grad, dbias=p["bias"].grad, dgq=p["gq"].grad,
                dgk=p["gk"].grad, dx=p["x"].grad)


def test_training_step_matches_autograd():
    t, labels = _inputs()
    got, want = Step(t, labels).run(), _reference(t, labels)
    for n in want:
        g, r = got[n].double().cpu(), want[n]
        assert torch.isfinite(g).all(), n
        off = ((g - r).norm() / r.norm()).item()
        assert off <= TOL, (n, off)


def test_captured_step_replays_the_same_bits():
    """The whole step in a graph, replayed after eager steps and on new
    inputs: the eager step's bits."""
    t, labels = _inputs()
    step = Step(t, labels)
    eager = step.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step.run()
    for scale in (1.0, -0.5):
        step.t["x"].copy_((t["x"].float() * scale).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        got = {n: v.clone() for n, v in out.items()}
        eager = step.run()
        for n in eager:
            assert torch.equal(got[n], eager[n]), (n, scale)


def test_two_streams_at_once():
    """Two steps of the loss in flight on two streams, each with its own
    workspace, beside the attention on a third: the bits of one at a time."""
    t, labels = _inputs()
    g = torch.Generator().manual_seed(9)
    hs = [torch.randn(n, hidden, generator=g).bfloat16().cuda() for n in (100, 1500)]
    labs = [torch.randint(0, V, (x.shape[0],), generator=g, dtype=torch.int32).cuda() for x in hs]
    w, bias = t["w"].cuda(), t["bias"].cuda()
    step = Step(t, labels)

    def ce(i, stream=None):
        loss, lse = bb.bb_linear_ce_fwd(hs[i], w, bias, labs[i], stream=stream)
        return (loss,) + bb.bb_linear_ce_bwd(hs[i], w, bias, labs[i], lse, lse, stream=stream)

    want = [ce(0), ce(1)]
    alone = step.run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [ce(i, streams[i]) for i in (0, 1)]
        both = step.run()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
        assert all(torch.equal(both[n], alone[n]) for n in alone)


def test_binding_refuses_wrong_shapes_and_types():
    x = torch.zeros(4, 8, device="cuda")
    with pytest.raises(ValueError):
        bb.bb_dropout_fwd(x, torch.zeros(8, 4, device="cuda"), 0.1, 0)
    with pytest.raises(ValueError):
        bb.bb_dropout_fwd(x.half(), None, 0.1, 0)
    with pytest.raises(ValueError):
        bb.bb_dropout_fwd(x.t(), None, 0.1, 0)
    with pytest.raises(ValueError):
        bb.bb_dropout_bwd(x, 0.1, 0, dx=torch.zeros(4, 8, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(bb.BBError):
        bb.bb_dropout_fwd(x, None, 1.0, 0)
    h = torch.zeros(6, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(9, 64, device="cuda", dtype=torch.bfloat16)
    lab = torch.zeros(6, device="cuda", dtype=torch.int32)
    with pytest.raises(ValueError):
        bb.bb_linear_ce_fwd(h, w, None, lab.long())
    with pytest.raises(ValueError):
        bb.bb_linear_ce_fwd(h, w[:, :32].contiguous(), None, lab)
    with pytest.raises(ValueError):
        bb.bb_linear_ce_fwd(h, w, torch.zeros(8, device="cuda"), lab)
    with pytest.raises(bb.BBError) as e:
        bb.bb_linear_ce_fwd(h, w, None, lab, workspace=torch.zeros(64, dtype=torch.uint8,
                                                                  device="cuda"))
    assert e.value.code == bb.BB_ERR_WORKSPACE
    with pytest.raises(bb.BBError) as e:
        bb.bb_linear_ce_fwd(h[:, :60].contiguous(), w[:, :60].contiguous(), None, lab)
    assert e.value.code == -2
    assert np.isfinite(bb.bb_linear_ce_fwd(h, w, None, lab)[0].cpu().numpy()).all()
