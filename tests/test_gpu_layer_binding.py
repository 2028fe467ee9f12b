"""The binding's checks of the cross entropy's status word on the GPU."""

import pytest
import torch

from block_sparse_long_bwd_b200 import binding as bb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [7, 300])
def test_a_label_outside_the_vocabulary_raises_where_asked(N):
    D, V = 64, 500
    g = torch.Generator().manual_seed(N)
    h = torch.randn(N, D, generator=g).bfloat16().cuda()
    w = torch.randn(V, D, generator=g).bfloat16().cuda()
    labels = torch.randint(-1, V, (N,), generator=g, dtype=torch.int32).cuda()
    dl = torch.ones(N, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    loss, lse = bb.bb_linear_ce_fwd(h, w, None, labels)
    grads = bb.bb_linear_ce_bwd(h, w, None, labels, lse, dl)
    for stream in (None, side):
        kw = dict(stream=stream, check=True)
        got = bb.bb_linear_ce_fwd(h, w, None, labels, **kw)
        assert torch.equal(got[0], loss) and torch.equal(got[1], lse)
        got = bb.bb_linear_ce_bwd(h, w, None, labels, lse, dl, **kw)
        assert torch.equal(got[0], grads[0]) and torch.equal(got[1], grads[1])
        bad = labels.clone()
        bad[N // 2] = V
        torch.cuda.synchronize()
        for call in (lambda: bb.bb_linear_ce_fwd(h, w, None, bad, **kw),
                     lambda: bb.bb_linear_ce_bwd(h, w, None, bad, lse, dl, **kw)):
            with pytest.raises(bb.BBError) as e:
                call()
            assert e.value.code == bb.BB_ERR_BAD_LABEL
        bb.bb_linear_ce_fwd(h, w, None, bad, stream=stream)  # not asked: no wait, no error
    torch.cuda.synchronize()
