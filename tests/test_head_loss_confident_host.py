"""The bound of dX in oracle/close.py on rows whose label is likely, on the CPU:
the arithmetic that keeps the label's probability out of the rounded ones lies
within it, one that rounds it with the others and subtracts 1 afterwards does not."""
import numpy as np
import pytest

from head_confident import bf16, confident
from oracle import close

TARGETS = (0.9, 0.99, 0.999, 1 - 2.0 ** -12)


@pytest.mark.parametrize("M,V,K", [(16, 300, 64), (40, 512, 100)])
def test_bound_sees_a_rounded_label(M, V, K):
    scale = 0.5
    x, W, labels, dloss = confident(M, V, K, TARGETS, scale, M)
    (want, err), _ = close.head_loss_bwd(x, W, labels, dloss, scale, exact_logits=True)
    z = scale * x.astype(np.float64) @ W.T.astype(np.float64)
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    at = np.arange(M), labels
    for m in range(M):  # near what was asked for, in the distance from 1
        assert abs((1 - p[m, labels[m]]) / (1 - TARGETS[m % 4]) - 1) < 0.2
    # the gradient by its own formula
    hot = np.zeros_like(p)
    hot[at] = 1
    f = (dloss * scale)[:, None].astype(np.float64)
    assert np.allclose(want, f * ((p - hot) @ W), rtol=1e-12, atol=0)
    # A bound as large as the gradient would let anything pass.
    norm = lambda a: np.sqrt((a * a).sum(1))  # noqa: E731
    assert (norm(err) < norm(want) / 16).all()
    rest = p[at] - 1
    apart = p.copy()
    apart[at] = 0
    good = f * (bf16(apart) @ W.astype(np.float64) + rest[:, None] * W[labels])
    assert (np.abs(good - want) <= err).all()
    bad = f * (bf16(p) @ W.astype(np.float64) - W[labels])
    likely = [m for m in range(M) if m % 4 >= 2]  # 0.999 becomes 1
    assert (norm(bad - want)[likely] > norm(want)[likely] / 2).all()
    assert (np.abs(bad - want) > err).any(1)[likely].all()
