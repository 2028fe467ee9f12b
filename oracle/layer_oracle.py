"""fp64 CPU oracle of the operators around the attention (test infrastructure
only): output dropout, the per-head norm with the rotary rotation, and the
vocabulary projection's softmax cross entropy, each with its gradient, by the
plain definition in NumPy.
"""

import math

import numpy as np

from .bigbird_oracle import dropout_scale, dropout_threshold, philox4x32_10


def _f64(x):
    return np.asarray(x, dtype=np.float64)


def out_dropout_keep(seed, site, rate, n, start=0):
    """bool [n] keep decisions of elements start .. start + n - 1: byte i & 15
    of the Philox4x32-10 call at counter (i >> 4 low, i >> 4 high, site,
    2^32 - 1) under the seed, kept when >= the rate's byte threshold."""
    i = np.arange(start, start + n, dtype=np.uint64)
    g0 = start >> 4
    g = np.arange(g0, ((start + n - 1) >> 4) + 1, dtype=np.uint64)
    low = np.uint64(0xFFFFFFFF)
    w = philox4x32_10((g & low, g >> np.uint64(32), np.uint64(site), low),
                      (seed & 0xFFFFFFFF, seed >> 32))
    words = np.stack([np.broadcast_to(x, g.shape).astype(np.uint64) for x in w], axis=1)
    j = i & np.uint64(15)
    word = words[(i >> np.uint64(4)).astype(np.int64) - g0, (j >> np.uint64(2)).astype(np.int64)]
    byte = (word >> (np.uint64(8) * (j & np.uint64(3)))) & np.uint64(255)
    return byte >= np.uint64(dropout_threshold(rate))


def out_dropout(x, residual, rate, seed, site):
    """(residual +) x / keep probability where kept, else (residual +) 0; the
    gradient of x is the same with x = dout and no residual."""
    x = _f64(x)
    keep = out_dropout_keep(seed, site, rate, x.size).reshape(x.shape)
    y = np.where(keep, x * dropout_scale(rate), 0.0)
    return y if residual is None else y + _f64(residual)


def _pairs(rot_dim, interleaved):
    for i in range(rot_dim // 2):
        yield i, *((2 * i, 2 * i + 1) if interleaved else (i, i + rot_dim // 2))


def _rotate(u, pos, theta, rot_dim, interleaved, sign):
    """u [B, H, L, d] rotated by sign times each token's angles; pos [B, L]."""
    y = u.copy()
    for i, a, b in _pairs(rot_dim, interleaved):
        t = pos.astype(np.float64)[:, None, :] * theta ** (-2.0 * i / rot_dim)
        c, s = np.cos(t), sign * np.sin(t)
        y[..., a] = u[..., a] * c - u[..., b] * s
        y[..., b] = u[..., b] * c + u[..., a] * s
    return y


def _positions(x, pos):
    B, _, L, _ = x.shape
    return np.broadcast_to(np.arange(L), (B, L)) if pos is None else np.asarray(pos)


def qk_norm_rope(x, gamma, pos, eps, theta, rot_dim, interleaved):
    """Rotated gamma * x / sqrt(mean(x^2) + eps) of x [B, H, L, d]."""
    x = _f64(x)
    g = np.ones(x.shape[-1]) if gamma is None else _f64(gamma)
    u = g * x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return _rotate(u, _positions(x, pos), theta, rot_dim, interleaved, 1.0)


def qk_norm_rope_backward(x, gamma, pos, dy, eps, theta, rot_dim, interleaved):
    """(dx, dgamma) for upstream dy.  With r = 1 / sqrt(mean(x^2) + eps) and
    g = R^T dy: dgamma = sum of g x r, and from dr/dx_j = -r^3 x_j / d,
    dx = gamma g r - x r^3 mean(gamma g x)."""
    x = _f64(x)
    gam = np.ones(x.shape[-1]) if gamma is None else _f64(gamma)
    g = _rotate(_f64(dy), _positions(x, pos), theta, rot_dim, interleaved, -1.0)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dx = gam * g * r - x * r**3 * (gam * g * x).mean(-1, keepdims=True)
    return dx, (g * x * r).sum((0, 1, 2))


def linear_ce(h, w, bias, labels):
    """(loss, lse) [N] of logits h w^T + bias: lse = log sum exp, loss = lse -
    logit of the label; rows whose label is outside [0, V) give 0 and 0."""
    h, w, labels = _f64(h), _f64(w), np.asarray(labels)
    loss, lse = np.zeros(len(h)), np.zeros(len(h))
    for n in range(len(h)):
        if 0 <= labels[n] < len(w):
            z = w @ h[n] + (0.0 if bias is None else _f64(bias))
            m = z.max()
            with np.errstate(invalid="ignore"):
                lse[n] = m + math.log(np.exp(z - m).sum()) if np.isfinite(m) else m
                loss[n] = lse[n] - z[labels[n]]
    return loss, lse


def linear_ce_backward(h, w, bias, labels, lse, dloss):
    """(dh, dw, dbias) for upstream dloss [N] and the forward's lse: per row
    with a label, dz = dloss (exp(z - lse) - onehot(label)); dh = dz w,
    dw = sum dz h, dbias = sum dz."""
    h, w, labels = _f64(h), _f64(w), np.asarray(labels)
    dh, dw, db = np.zeros_like(h), np.zeros_like(w), np.zeros(len(w))
    for n in range(len(h)):
        if 0 <= labels[n] < len(w):
            z = w @ h[n] + (0.0 if bias is None else _f64(bias))
            dz = np.exp(z - float(lse[n]))
            dz[labels[n]] -= 1.0
            dz *= float(dloss[n])
            dh[n] = dz @ w
            dw += np.outer(dz, h[n])
            db += dz
    return dh, dw, db
