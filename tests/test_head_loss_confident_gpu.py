"""GPU tests of the head loss's gradients of rows that the model predicts well:
p - 1 at the label is small against p, so that a probability rounded to bf16
before the subtraction would lose it."""
import numpy as np
import pytest
import torch

import qlora_fine_tuning_blockwise_amd as q
from head_confident import confident
from oracle import close
from test_row_ops_gpu import BF16, DEV, F32, check, say, strided

pytestmark = pytest.mark.gpu

ALL = (0.9, 0.99, 0.999, 1 - 2.0 ** -12)


def _norm(a):
    return np.sqrt((a * a).sum(1))


# One pass over W, few rows with a product behind them, tiles; W in place and
# copied (a width of no whole steps), and in two pieces. With a larger vocabulary the
# bound of its sum of exponentials grows, and the likeliest labels are left out.
@pytest.mark.parametrize("M,V,K,targets", [
    (1, 300, 512, ALL[3:]), (1, 300, 64, ALL[:1]), (16, 300, 512, ALL), (16, 512, 100, ALL), (9, 400, 4160, ALL),
    (40, 512, 512, ALL), (64, 300, 100, ALL), (300, 512, 512, ALL), (300, 400, 100, ALL), (300, 33000, 72, ALL[:2])])
@pytest.mark.parametrize("kind", [BF16, F32], ids=["bf16", "f32"])
def test_head_loss_gradient_of_likely_labels(M, V, K, targets, kind):
    scale = 0.5
    say("head likely labels", M, V, K, kind)
    x, W, labels, dloss = confident(M, V, K, targets, scale, M + V + K)
    xv, _ = strided(torch.from_numpy(x).to(BF16), 8)
    Wv, _ = strided(torch.from_numpy(W).to(BF16), 3 if K % 32 else 0)
    ids, d = torch.from_numpy(labels).to(DEV), torch.from_numpy(dloss).to(DEV)
    stats = torch.empty(2, M, device=DEV)
    q.qlora_head_loss_fwd(xv, Wv, ids, scale=scale, stats_out=stats)
    dX, dW = q.qlora_head_loss_bwd(xv, Wv, ids, d, stats, scale=scale, dx_dtype=kind, grad_dtype=kind)
    (wX, eX), (wW, eW) = close.head_loss_bwd(x, W, labels, dloss, scale, 3 if kind == F32 else 1, exact_logits=True)
    # A bound as large as the gradient would let anything pass.
    assert (_norm(eX) < _norm(wX) / 16).all()
    check(dX, wX, eX, "dX")
    check(dW, wW, eW, "dW")
    got = dX.double().cpu().numpy()
    assert (_norm(got - wX) <= _norm(wX) / 16).all()
    for m in ({}, {"want_dw": False}):
        again, _ = q.qlora_head_loss_bwd(xv, Wv, ids, d, stats, scale=scale, dx_dtype=kind, grad_dtype=kind, **m)
        assert torch.equal(again, dX)
    _, alone = q.qlora_head_loss_bwd(xv, Wv, ids, d, stats, scale=scale, grad_dtype=kind, want_dx=False)
    assert torch.equal(alone, dW)
