"""Inputs of the vocabulary head's loss whose labels have a given probability,
for the tests of the gradient of rows that the model predicts well."""
import numpy as np
import torch

STEP = 0.25  # of W's entries, +-STEP


def bf16(a):
    """To bf16 and back, to nearest even."""
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16).float().numpy()


def _probability(z, label):
    z = z - z.max()
    return np.exp(z[label]) / np.exp(z).sum()


def confident(M, V, K, targets, scale, seed):
    """x, W (fp32 values that bf16 holds), labels, dloss: row m's label has nearly
    the probability targets[m % len(targets)]. W's entries are +-1/4 and a row of x
    is a multiple c of its label's signs, so that every product and every partial sum
    of a logit is a whole number, K at most, times c / 4: c has 8 bits, K at most 13,
    and with a power of two for the scale fp32 holds each logit exactly."""
    assert K <= 8192 and np.frexp(scale)[0] == 0.5
    g = np.random.default_rng(seed)
    W = np.where(g.random((V, K)) < 0.5, -STEP, STEP).astype(np.float32)
    labels = g.permutation(V)[:M] if M <= V else g.integers(0, V, M)
    signs = np.sign(W[labels])
    agree = (signs.astype(np.float64) @ W.T.astype(np.float64)) * scale  # logits for c = 1
    c = np.empty(M, np.float32)
    for m in range(M):
        lo, hi = 0.0, 400.0 / (abs(scale) * STEP * K)
        for _ in range(60):
            mid = (lo + hi) / 2
            lo, hi = (mid, hi) if _probability(mid * agree[m], labels[m]) < targets[m % len(targets)] else (lo, mid)
        c[m] = bf16(np.array([lo]))[0]
    dloss = ((0.5 + g.random(M)) / M).astype(np.float32)
    return signs * c[:, None], W, labels, dloss
