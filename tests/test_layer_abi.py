"""Host-side checks of the operators around the attention that need no GPU:
every call refuses bad arguments before it touches a pointer or CUDA."""

import ctypes

import pytest
import torch

from block_sparse_long_bwd_b200 import binding as bb

P = 1 << 20  # a fake 16-byte aligned address, never dereferenced


def test_out_dropout_refusals():
    lib = bb.lib()
    f, b = lib.bb_dropout_fwd, lib.bb_dropout_bwd
    assert f(0, 1, 0.1, 0, 0, P, None, P, None) == -1        # no elements
    assert f(16, 2, 0.1, 0, 0, P, None, P, None) == -1       # dtype
    for rate in (1.0, -0.1, float("nan"), 255.6 / 256):
        assert f(16, 1, rate, 0, 0, P, None, P, None) == -1
        assert b(16, 1, rate, 0, 0, P, P, None) == -1
    assert f(16, 1, 0.1, 0, 0, None, None, P, None) == -1
    assert f(16, 1, 0.1, 0, 0, P, None, None, None) == -1
    assert f(16, 1, 0.1, 0, 0, P + 2, None, P, None) == -1
    assert f(16, 1, 0.1, 0, 0, P, P + 8, P, None) == -1
    assert f((1 << 42) + 1, 1, 0.1, 0, 0, P, None, P, None) == -2


def _qk(**kw):
    base = dict(B=2, H=3, L=50, dtype=bb.BB_BF16)
    base.update(kw)
    return bb.make_qk_desc(**base)


def test_qk_norm_rope_refusals():
    lib = bb.lib()
    bad = [(dict(B=0), -1), (dict(H=-1), -1), (dict(L=0), -1), (dict(dtype=5), -1),
           (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(rot_dim=65), -1),
           (dict(rot_dim=66), -1), (dict(rot_dim=-2), -1), (dict(rot_dim=7), -1),
           (dict(theta=0.5), -1), (dict(theta=float("inf")), -1), (dict(d=128), -2),
           (dict(H=40000), -2)]
    n = ctypes.c_size_t(0)
    for kw, code in bad:
        d = ctypes.byref(_qk(**kw))
        assert lib.bb_qk_norm_rope_workspace_size(d, ctypes.byref(n)) == code, kw
        assert lib.bb_qk_norm_rope_fwd(d, P, P, None, None, None, P, P, None) == code, kw
    d_ = _qk()
    d_.interleaved = 2
    assert lib.bb_qk_norm_rope_fwd(ctypes.byref(d_), P, P, None, None, None, P, P, None) == -1
    assert lib.bb_qk_norm_rope_workspace_size(ctypes.byref(_qk()), None) == -1
    assert lib.bb_qk_norm_rope_workspace_size(None, ctypes.byref(n)) == -1
    assert bb.bb_qk_norm_rope_workspace_size(_qk(rot_dim=0, theta=0.0)) > 0  # theta unused
    d, size = ctypes.byref(_qk()), bb.bb_qk_norm_rope_workspace_size(_qk())
    for i in (0, 1, 5, 6):
        a = [P, P, None, None, None, P, P]
        a[i] = None
        assert lib.bb_qk_norm_rope_fwd(d, *a, None) == -1
    for i in range(7):
        a = [P] * 7
        a[i] = P + 4
        assert lib.bb_qk_norm_rope_fwd(d, *a, None) == -1
    good = [P] * 12
    assert lib.bb_qk_norm_rope_bwd(d, *good, size - 1, None) == -4
    for i, code in ((0, -1), (5, -1), (6, -1), (7, -1), (8, -1), (11, -4)):
        a = list(good)
        a[i] = None
        assert lib.bb_qk_norm_rope_bwd(d, *a, size, None) == code, i


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(16)
    with pytest.raises(ValueError):
        bb.bb_dropout_fwd(x, None, 0.1, 0)
    with pytest.raises(ValueError):
        bb.bb_dropout_bwd(x, 0.1, 0)
    q = torch.zeros((2, 3, 50, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bb.bb_qk_norm_rope_fwd(_qk(), q, q, None, None)


def test_linear_ce_refusals():
    lib = bb.lib()
    n = ctypes.c_size_t(0)
    size = lib.bb_linear_ce_workspace_size
    for args, code in (((0, 64, 10), -1), ((5, 0, 10), -1), ((5, 64, 0), -1), ((-1, 64, 10), -1),
                       ((5, 60, 10), -2), ((5, 56, 10), -2), ((5, 65544, 10), -2),
                       ((1 << 25, 64, 10), -2), ((5, 64, 1 << 25), -2),
                       ((1 << 24, 64, 1 << 24), -2)):
        assert size(*args, 0, ctypes.byref(n)) == code, args
        assert lib.bb_linear_ce_fwd(*args, P, P, P, P, P, P, P, 1 << 40, None) == code
        assert lib.bb_linear_ce_bwd(*args, P, P, P, P, P, P, P, P, P, P, 1 << 40, None) == code
    assert size(5, 64, 10, 2, ctypes.byref(n)) == -1
    assert size(5, 64, 10, 0, None) == -1
    dims = (100, 128, 1000)
    f, b = (bb.bb_linear_ce_workspace_size(*dims, p) for p in (0, 1))
    good = [P] * 7
    assert lib.bb_linear_ce_fwd(*dims, *good, f - 1, None) == -4
    for i, code in ((0, -1), (1, -1), (3, -1), (4, -1), (5, -1), (6, -4)):
        a = list(good)
        a[i] = None
        assert lib.bb_linear_ce_fwd(*dims, *a, f, None) == code, i
        a[i] = P + 4
        assert lib.bb_linear_ce_fwd(*dims, *a, f, None) == -1, i
    good = [P] * 10
    assert lib.bb_linear_ce_bwd(*dims, *good, b - 1, None) == -4
    for i, code in ((0, -1), (1, -1), (3, -1), (4, -1), (5, -1), (6, -1), (7, -1), (9, -4)):
        a = list(good)
        a[i] = None
        assert lib.bb_linear_ce_bwd(*dims, *a, b, None) == code, i
        a[i] = P + 4
        assert lib.bb_linear_ce_bwd(*dims, *a, b, None) == -1, i


def test_linear_ce_workspace_is_bounded_by_a_piece():
    """The backward's workspace holds one piece of the vocabulary (256 MiB of
    dz at most), not the N x V logits."""
    N, D, V = 32768, 1024, 200000
    need = bb.bb_linear_ce_workspace_size(N, D, V, 1)
    # dz of a piece, packed rows, fp32 dh, and the dbias sums of a piece
    assert need < (256 << 20) + N * D * 2 + N * D * 4 + N // 128 * 8192 * 4 + (4 << 20)
    assert need < N * V * 2 // 10
    assert bb.bb_status_str(bb.BB_ERR_BAD_LABEL) != bb.bb_status_str(42)
