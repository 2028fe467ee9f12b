"""Measured cases of the operators around the block-sparse attention.

Three operators of an encoder layer's training step:

* dropout: counter-based dropout of a layer's output, with the residual added
  in the same pass; the keep decisions are drawn again in the backward.
* qk_norm_rope: RMS norm of each head's queries and keys and the rotary
  position rotation, between the Q/K/V projection and the attention.
* linear_ce: softmax cross entropy of a vocabulary projection, without the
  logits in memory, with its gradients.

``run`` computes an operator with elementary torch operations, or, where
``own`` is true, with the library's kernels; ``exact`` computes it in 64 bits.
"""

import math

import numpy as np
import torch

own = False

THETA = 10000.0
EPS = 1e-6
SEED = 0x5EED0123456789AB

# Philox4x32-10: multipliers and key increments.
PHILOX_M = (0xD2511F53, 0xCD9E8D57)
PHILOX_W = (0x9E3779B9, 0xBB67AE85)
LOW32 = 0xFFFFFFFF

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # A handful of tokens through one layer's output dropout: the cost of a call.
        dict(name="dropout_fwd_16_tokens", op="dropout_fwd", B=1, L=16, hidden=768, dtype="bf16",
             rate=0.1, residual=True, site=3),
        # The output dropout and residual of a BigBird-large training batch.
        dict(name="dropout_fwd_large", op="dropout_fwd", B=4, L=4096, hidden=1024, dtype="bf16",
             rate=0.1, residual=True, site=0),
        # Gradient through dropout, fp32, a ragged batch of an odd width.
        dict(name="dropout_bwd_odd_f32", op="dropout_bwd", B=3, L=4001, hidden=771, dtype="f32",
             rate=0.25, residual=False, site=1),
        # One token's queries and keys (a single decoding step).
        dict(name="qk_fwd_one_token", op="qk_fwd", B=1, H=12, L=1, dtype="bf16", rot_dim=64,
             interleaved=False, packed=False),
        # BigBird-large training batch, forward.
        dict(name="qk_fwd_large", op="qk_fwd", B=4, H=16, L=4096, dtype="bf16", rot_dim=64,
             interleaved=False, packed=False),
        # BigBird-base training batch of packed documents, gradients.
        dict(name="qk_bwd_packed", op="qk_bwd", B=8, H=12, L=4096, dtype="bf16", rot_dim=64,
             interleaved=False, packed=True),
        # fp32, an odd length, adjacent pairs on half of the head.
        dict(name="qk_bwd_odd_f32", op="qk_bwd", B=1, H=12, L=5003, dtype="f32", rot_dim=32,
             interleaved=True, packed=False),
        # Scoring a few tokens: bound by reading the vocabulary's weights.
        dict(name="ce_fwd_13_rows", op="ce_fwd", N=13, hidden=768, V=30011, labelled=13, bias=True,
             weighted=False),
        # Masked-language-model evaluation: a batch of 4 x 4096 tokens, 15 % with a label.
        dict(name="ce_fwd_mlm", op="ce_fwd", N=16384, hidden=1024, V=50021, labelled=2458,
             bias=True, weighted=False),
        # Gradients of a small fine-tuning batch, odd sizes, weighted rows.
        dict(name="ce_bwd_77_rows", op="ce_bwd", N=77, hidden=776, V=30011, labelled=70, bias=True,
             weighted=True),
        # Gradients at BigBird-base width, every token labelled.
        dict(name="ce_bwd_base", op="ce_bwd", N=4096, hidden=768, V=32000, labelled=4096,
             bias=False, weighted=False),
        # A whole training step of the loss at BigBird-large width: loss, then all gradients.
        dict(name="ce_train_large", op="ce_train", N=8192, hidden=1024, V=50021, labelled=8192,
             bias=True, weighted=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dropout_fwd", "dropout_bwd", "qk_fwd", "qk_bwd", "ce_fwd", "ce_bwd",
                     "ce_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("dropout"):
        tokens = _log(rng, 1, 16384)
        B = rng.choice([1, 1, 2, 3, 4])
        return dict(op=op, B=B, L=max(1, tokens // B), hidden=rng.randint(64, 1024), dtype=dtype,
                    rate=rng.choice([0.05, 0.1, 0.25, 0.5]),
                    residual=op == "dropout_fwd" and rng.random() < 0.7, site=rng.randint(0, 48))
    if op.startswith("qk"):
        tokens = _log(rng, 1, 32768)
        B = rng.choice([1, 1, 2, 3, 4, 8])
        rot = rng.choice([64, 64, 64, 32, 16, 2 * rng.randint(1, 32)])
        return dict(op=op, B=B, H=rng.randint(1, 12 if dtype == "bf16" else 6),
                    L=max(1, tokens // B), dtype=dtype, rot_dim=rot,
                    interleaved=rng.random() < 0.4, packed=rng.random() < 0.5)
    N = _log(rng, 1, 8192)
    return dict(op=op, N=N, hidden=8 * rng.randint(8, 128), V=_log(rng, 500, 50000),
                labelled=max(1, int(N * rng.choice([1.0, 1.0, 0.5, 0.15]))),
                bias=rng.random() < 0.5, weighted=rng.random() < 0.5)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    op = case["op"]
    s = dict(case, seed=(SEED + 1000003 * seed) % 2**64)
    if op.startswith("dropout"):
        shape, dt = (case["B"], case["L"], case["hidden"]), DTYPES[case["dtype"]]
        s["x"] = randn(*shape).to(dt)
        s["residual_in"] = randn(*shape).to(dt) if case["residual"] else None
        return s
    if op.startswith("qk"):
        B, H, L, dt = case["B"], case["H"], case["L"], DTYPES[case["dtype"]]
        for n in ("q", "k"):
            s[n] = (1.5 * randn(B, H, L, 64)).to(dt)
            s["g" + n] = 1.0 + 0.2 * randn(64)
            if op == "qk_bwd":
                s["d" + n] = randn(B, H, L, 64).to(dt)
        s["positions"] = None
        if case["packed"]:
            # Documents of random lengths, each counted from 0.
            start = torch.rand((B, L), generator=g, device="cuda") < 4.0 / L
            start[:, 0] = True
            at = torch.arange(L, device="cuda").expand(B, L)
            s["positions"] = (at - torch.where(start, at, 0).cummax(1).values).to(torch.int32)
        return s
    N, hidden, V, lab = case["N"], case["hidden"], case["V"], case["labelled"]
    # A partly trained model: each row leans towards its label by a varying amount.
    w = (0.05 * randn(V, hidden)).to(torch.bfloat16)
    true = torch.randint(0, V, (N,), generator=g, device="cuda")
    lean = 12.0 * torch.rand((N, 1), generator=g, device="cuda") / hidden**0.5
    h = randn(N, hidden) + lean * (20.0 * w[true].float())
    s["h"], s["w"] = h.to(torch.bfloat16), w
    s["bias_in"] = 0.5 * randn(V) if case["bias"] else None
    rows = torch.randperm(N, generator=g, device="cuda")[:lab]
    labels = torch.full((N,), -100, device="cuda")
    labels[rows] = true[rows]
    s["labels"] = labels.to(torch.int32)
    each = torch.rand(N, generator=g, device="cuda") + 0.5 if case["weighted"] else 1.0
    s["dloss"] = torch.full((N,), 1.0 / lab, device="cuda") * each
    if op == "ce_bwd":
        s["lse"] = torch.zeros(N, device="cuda")
        for part in rows.split(2048):
            z = s["h"][part].float() @ w.float().t()
            z = z if s["bias_in"] is None else z + s["bias_in"]
            s["lse"][part] = z.double().logsumexp(1).float()
    return s


# ---- plain forms ----------------------------------------------------------


def _mul32(a, m):
    """High and low words of a * m; a holds 32-bit values in int64."""
    lo, hi = (a & 0xFFFF) * m, (a >> 16) * m
    return (hi + (lo >> 16)) >> 16, ((hi << 16) + lo) & LOW32


def _keep(s, n):
    """Keep decisions of elements 0 .. n - 1: one Philox call for 16 elements."""
    g = torch.arange((n + 15) // 16, device="cuda")
    c = [g & LOW32, g >> 32, torch.full_like(g, s["site"]), torch.full_like(g, LOW32)]
    k0, k1 = s["seed"] & LOW32, s["seed"] >> 32
    for _ in range(10):
        h0, l0 = _mul32(c[0], PHILOX_M[0])
        h1, l1 = _mul32(c[2], PHILOX_M[1])
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
        k0, k1 = (k0 + PHILOX_W[0]) & LOW32, (k1 + PHILOX_W[1]) & LOW32
    words = torch.stack(c, dim=1)
    shifts = torch.arange(0, 32, 8, device="cuda")
    return ((words[:, :, None] >> shifts) & 255).reshape(-1)[:n] >= _threshold(s["rate"])


def _threshold(rate):
    return math.floor(256 * rate + 0.5)


def _dropout(s):
    x = s["x"].float()
    keep = _keep(s, x.numel()).view(x.shape)
    y = torch.where(keep, x * (256.0 / (256 - _threshold(s["rate"]))), 0.0)
    if s["residual_in"] is not None:
        y = y + s["residual_in"].float()
    return y.to(s["x"].dtype)


def _angles(s):
    """cos and sin of each token's angles, [B or 1, 1, L, rot_dim / 2]; the angle in 64 bits."""
    L, rot = s["L"], s["rot_dim"]
    pos = s["positions"]
    pos = torch.arange(L, device="cuda")[None] if pos is None else pos
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    a = (pos.double()[:, :, None] * THETA ** (-2.0 * i / rot))[:, None]
    return a.cos().float(), a.sin().float()


def _rotate(x, cos, sin, rot, interleaved):
    r, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = r[..., : rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([r, rest], dim=-1)


def _qk_fwd(s, x, gamma, cos, sin):
    f = x.float()
    n = f * (f.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return _rotate(n * gamma, cos, sin, s["rot_dim"], s["interleaved"]).to(x.dtype)


def _qk_bwd(s, x, gamma, dy, cos, sin):
    f = x.float()
    r = (f.square().mean(-1, keepdim=True) + EPS).rsqrt()
    n = f * r
    g = _rotate(dy.float(), cos, -sin, s["rot_dim"], s["interleaved"])
    dgamma = (g * n).double().sum((0, 1, 2)).float()
    dn = g * gamma
    dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    return dx.to(x.dtype), dgamma


def _logits(s, rows):
    z = s["h"][rows].float() @ s["w"].float().t()
    return z if s["bias_in"] is None else z + s["bias_in"]


def _ce_fwd(s):
    N, rows = s["N"], (s["labels"] >= 0).nonzero()[:, 0]
    z = _logits(s, rows)
    m = z.amax(1, keepdim=True)
    lse = m[:, 0] + (z - m).exp().sum(1).log()
    at = z.gather(1, s["labels"][rows].long()[:, None])[:, 0]
    zero = torch.zeros(N, device="cuda")
    return zero.index_put((rows,), lse - at), zero.index_put((rows,), lse)


def _ce_bwd(s, lse):
    rows = (s["labels"] >= 0).nonzero()[:, 0]
    h, w = s["h"], s["w"]
    dz = (_logits(s, rows) - lse[rows, None]).exp()
    dz[torch.arange(rows.numel(), device="cuda"), s["labels"][rows].long()] -= 1.0
    dz *= s["dloss"][rows, None]
    dh = torch.zeros(h.shape, device="cuda").index_put((rows,), dz @ w.float())
    dw = dz.t() @ h[rows].float()
    out = {"dh": dh.to(h.dtype), "dw": dw.to(w.dtype)}
    if s["bias_in"] is not None:
        out["dbias"] = dz.sum(0)
    return out


def _run_plain(s):
    op = s["op"]
    if op.startswith("dropout"):
        return _dropout(s)
    if op.startswith("qk"):
        cos, sin = _angles(s)
        if op == "qk_fwd":
            return [_qk_fwd(s, s["q"], s["gq"], cos, sin), _qk_fwd(s, s["k"], s["gk"], cos, sin)]
        dq, dgq = _qk_bwd(s, s["q"], s["gq"], s["dq"], cos, sin)
        dk, dgk = _qk_bwd(s, s["k"], s["gk"], s["dk"], cos, sin)
        return [dq, dk, dgq, dgk]
    if op == "ce_fwd":
        loss, lse = _ce_fwd(s)
        return {"loss": loss, "lse": lse}
    if op == "ce_bwd":
        return _ce_bwd(s, s["lse"])
    loss, lse = _ce_fwd(s)
    return {"loss": loss, "lse": lse, **_ce_bwd(s, lse)}


# ---- the library's calls ---------------------------------------------------


def _run_own(s):
    from block_sparse_long_bwd_b200 import binding as bb

    op = s["op"]
    if op == "dropout_fwd":
        return bb.bb_dropout_fwd(s["x"], s["residual_in"], s["rate"], s["seed"], s["site"])
    if op == "dropout_bwd":
        return bb.bb_dropout_bwd(s["x"], s["rate"], s["seed"], s["site"])
    if op.startswith("qk"):
        desc = bb.make_qk_desc(s["B"], s["H"], s["L"], s["q"].dtype, eps=EPS, theta=THETA,
                               rot_dim=s["rot_dim"], interleaved=s["interleaved"])
        if op == "qk_fwd":
            return bb.bb_qk_norm_rope_fwd(desc, s["q"], s["k"], s["gq"], s["gk"], s["positions"])
        return bb.bb_qk_norm_rope_bwd(desc, s["q"], s["k"], s["gq"], s["gk"], s["positions"],
                                      s["dq"], s["dk"])
    out = {}
    lse = s.get("lse")
    if op != "ce_bwd":
        out["loss"], lse = bb.bb_linear_ce_fwd(s["h"], s["w"], s["bias_in"], s["labels"])
        out["lse"] = lse
    if op != "ce_fwd":
        dh, dw, dbias = bb.bb_linear_ce_bwd(s["h"], s["w"], s["bias_in"], s["labels"], lse,
                                            s["dloss"])
        out |= {"dh": dh, "dw": dw} | ({} if dbias is None else {"dbias": dbias})
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op = case["op"]
    if op.startswith("dropout"):
        n = case["B"] * case["L"] * case["hidden"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * size * (3 if case["residual"] else 2), "flops": 2 * n}
    if op.startswith("qk"):
        n = 2 * case["B"] * case["H"] * case["L"] * 64
        size = 2 if case["dtype"] == "bf16" else 4
        pos = 4 * case["B"] * case["L"] if case["packed"] else 0
        if op == "qk_fwd":
            return {"bytes": 2 * n * size + pos + 512, "flops": 8 * n}
        return {"bytes": 3 * n * size + pos + 1024, "flops": 16 * n}
    # Rows without a label are neither read nor multiplied.
    N, D, V, lab = case["N"], case["hidden"], case["V"], case["labelled"]
    vb = 4 * V if case["bias"] else 0
    read = 2 * lab * D + 2 * V * D + vb + 4 * N
    grads = 2 * N * D + 2 * V * D + vb
    if op == "ce_fwd":
        return {"bytes": read + 8 * N, "flops": 2.0 * lab * D * V}
    if op == "ce_bwd":
        return {"bytes": read + 8 * N + grads, "flops": 6.0 * lab * D * V}
    return {"bytes": read + 12 * N + grads, "flops": 6.0 * lab * D * V}


# ---- 64 bits ---------------------------------------------------------------


def _exact_keep(seed, site, thr, n):
    """The keep decisions with numpy's 64-bit products."""
    g = np.arange((n + 15) // 16, dtype=np.uint64)
    low, s32 = np.uint64(LOW32), np.uint64(32)
    x0, x1 = g & low, g >> s32
    x2, x3 = np.full_like(g, site), np.full_like(g, LOW32)
    for r in range(10):
        key0 = np.uint64((seed + r * PHILOX_W[0]) & LOW32)
        key1 = np.uint64(((seed >> 32) + r * PHILOX_W[1]) & LOW32)
        a, b = x0 * np.uint64(PHILOX_M[0]), x2 * np.uint64(PHILOX_M[1])
        x0, x1, x2, x3 = (b >> s32) ^ x1 ^ key0, b & low, (a >> s32) ^ x3 ^ key1, a & low
    words = np.stack([x0, x1, x2, x3], axis=1).astype("<u4")
    return torch.from_numpy(words.view(np.uint8).reshape(-1)[:n] >= thr)


def _exact_qk(s, x, gamma, dy):
    """y, or with dy the gradients: each head's norm and rotation as one matrix per token,
    y = R diag(gamma) x / rms(x), differentiated by the product rule."""
    L, rot = s["L"], s["rot_dim"]
    pos = s["positions"]
    pos = torch.arange(L, device="cuda")[None] if pos is None else pos
    R = torch.zeros((*pos.shape, 64, 64), dtype=torch.float64, device="cuda")
    for j in range(64):
        R[..., j, j] = 1.0
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + rot // 2)
        angle = pos.double() * math.pow(THETA, -2.0 * i / rot)
        R[..., a, a] = R[..., b, b] = torch.cos(angle)
        R[..., b, a] = torch.sin(angle)
        R[..., a, b] = -R[..., b, a]
    x, gamma = x.double(), gamma.double()
    rms = torch.sqrt((x * x).sum(-1, keepdim=True) / 64 + EPS)
    if dy is None:
        return torch.einsum("blij,bhlj->bhli", R.expand(x.shape[0], L, 64, 64), gamma * x / rms)
    back = torch.einsum("blij,bhli->bhlj", R.expand(x.shape[0], L, 64, 64), dy.double())
    dgamma = (back * x / rms).sum((0, 1, 2))
    inner = (back * gamma * x).sum(-1, keepdim=True)
    return back * gamma / rms - x * inner / (64 * rms**3), dgamma


def _exact_ce(s, grads, lse_in):
    N, D, V = s["N"], s["hidden"], s["V"]
    f64 = dict(dtype=torch.float64, device="cuda")
    loss, lse = torch.zeros(N, **f64), torch.zeros(N, **f64)
    dh, dw, db = torch.zeros((N, D), **f64), torch.zeros((V, D), **f64), torch.zeros(V, **f64)
    w = s["w"].double()
    for part in torch.arange(N, device="cuda")[s["labels"] >= 0].split(2048):
        h, lab = s["h"][part].double(), s["labels"][part].long()
        z = torch.einsum("nd,vd->nv", h, w)
        if s["bias_in"] is not None:
            z += s["bias_in"].double()
        lse[part] = torch.logsumexp(z, 1) if lse_in is None else lse_in[part].double()
        loss[part] = lse[part] - z[torch.arange(part.numel(), device="cuda"), lab]
        if grads:
            hot = torch.nn.functional.one_hot(lab, V)
            dz = (torch.exp(z - lse[part, None]) - hot) * s["dloss"][part, None].double()
            dh[part] = torch.einsum("nv,vd->nd", dz, w)
            dw += torch.einsum("nv,nd->vd", dz, h)
            db += dz.sum(0)
    out = {} if lse_in is not None else {"loss": loss, "lse": lse}
    if grads:
        out |= {"dh": dh, "dw": dw} | ({} if s["bias_in"] is None else {"dbias": db})
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("dropout"):
        x = s["x"].double().cpu()
        thr = int(case["rate"] * 256 + 0.5)
        keep = _exact_keep(s["seed"], case["site"], thr, x.numel()).view(x.shape)
        y = torch.where(keep, x / (1 - thr / 256), torch.zeros((), dtype=torch.float64))
        return y if s["residual_in"] is None else y + s["residual_in"].double().cpu()
    if op == "qk_fwd":
        return [_exact_qk(s, s["q"], s["gq"], None), _exact_qk(s, s["k"], s["gk"], None)]
    if op == "qk_bwd":
        dq, dgq = _exact_qk(s, s["q"], s["gq"], s["dq"])
        dk, dgk = _exact_qk(s, s["k"], s["gk"], s["dk"])
        return [dq, dk, dgq, dgk]
    return _exact_ce(s, op != "ce_fwd", s.get("lse"))
