"""The operators that close a training step (the norm behind a residual
addition, the loss of the vocabulary head, the clipping of the gradients'
global norm) in 64 bits, with numpy alone, each from its formula, with the
bound of the error that the library's arithmetic may make of them.

`err` counts roundings as oracle/rows.py does: u = 2^-24 for each in fp32, and
2^-8 relative for one to bf16. What the output's own type rounds away is not
part of it.
"""
from __future__ import annotations

import numpy as np

from oracle import rows
from oracle.rows import U

E4M3_MAX = 448.0
BF16 = 2.0 ** -8  # half a step, relative


# ------------------------------------------------- norm behind an addition
def add_norm_fwd(h, gamma, beta, eps, center, depth=None):
    """Of the sum h as it is kept (rounded): y, err, stats, err, and the scales
    of 8-bit codes and their err."""
    y, err, stats, e_stats = rows.norm_fwd(h, gamma, beta, eps, center, depth)
    a = np.abs(y)
    scales = a.max(1) / E4M3_MAX
    e_scales = err.max(1) / E4M3_MAX + 2 * U * scales
    return y, err, stats, e_stats, scales, e_scales


def codes_err(y, err, scales, e_scales):
    """What code * scale (as exact numbers) may be off y by: half a step of
    E4M3, 2^-4 of a value and 2^-10 of the scale below its normal numbers, of a
    value that has the errors of y and of two roundings, and the scale's own
    error, to which a code of at most 448 is proportional."""
    size = np.abs(y) + err
    code = np.minimum(size / np.maximum(scales, 1e-300)[:, None], E4M3_MAX)
    return (err + 3 * U * size + np.maximum(2.0 ** -4 * size, 2.0 ** -10 * scales[:, None])
            + (code + 1) * e_scales[:, None] * (1 + 2.0 ** -4))


def add_norm_bwd(dY, dH, h, gamma, eps, center, depth=None, rows_depth=None):
    (dX, err), dg, db = rows.norm_bwd(dY, h, gamma, eps, center, depth, rows_depth)
    if dH is not None:
        dX = dX + dH.astype(np.float64)
        err = err + U * np.abs(dX)
    return (dX, err), dg, db


# ----------------------------------------------------- clipping of gradients
def grad_norm(grads, max_norm):
    """norm, factor. Both are rounded to fp32 once (the sums are in 64 bits)."""
    norm = float(np.sqrt(sum(float((g.astype(np.float64) ** 2).sum()) for g in grads)))
    return norm, (max_norm / norm if norm > max_norm else norm / norm if np.isnan(norm) else 1.0)


# ------------------------------------------------------ loss of the head
def _logits(x, W, scale):
    """Logits and the error of their fp32 sums: a matrix instruction adds 8 to 16
    products and then the sum so far, so that a term passes at most K / 8 + 16
    additions, of which each may be off by a whole step (2 u)."""
    x, W = x.astype(np.float64), W.astype(np.float64)
    K = x.shape[1]
    z = scale * (x @ W.T)
    e = abs(scale) * (2 * U * (K / 8 + 16)) * (np.abs(x) @ np.abs(W).T) + 2 * U * np.abs(z)
    return z, e


def _softmax(z, e):
    """max, log of the sum taken from it, probabilities; the error of the
    logarithm, and the relative one of a probability."""
    V = z.shape[1]
    m = z.max(1, keepdims=True)
    a = z - m
    w = np.exp(a)
    total = w.sum(1, keepdims=True)
    L = np.log(total)
    p = w / total
    e_m = e.max(1, keepdims=True)
    # an exponential is off by its argument's error: the logits', the product
    # with log2(e) (two roundings of |a|) and three of its own; the sum of V of
    # them by at most V / 16 + 64 additions in a tile, a wave and over the tiles
    rel = e + e_m + U * (3 * np.abs(a) + 4)
    e_L = (p * rel).sum(1, keepdims=True) + U * (min(V, V / 16 + 64) + 2 * np.abs(L) + 4)
    return m, L, p, e_m, e_L, rel


def _live(labels, V):
    labels = np.asarray(labels, np.int64)
    live = (labels >= 0) & (labels < V)
    return live, np.where(live, labels, 0)


def head_loss_fwd(x, W, labels, scale=1.0):
    """loss, err, stats, err of the stats."""
    live, ids = _live(labels, W.shape[0])
    with np.errstate(invalid="ignore"):
        z, e = _logits(np.where(live[:, None], x, 0.0), W, scale)
        m, L, _, e_m, e_L, _ = _softmax(z, e)
    at, e_at = np.take_along_axis(z, ids[:, None], 1), np.take_along_axis(e, ids[:, None], 1)
    loss = (L + (m - at))[:, 0]
    err = (e_L + e_m + e_at + U * (np.abs(m - at) + np.abs(L)) * 2)[:, 0]
    stats = np.concatenate([m, L], 1).T * live
    return np.where(live, loss, 0.0), err * live, stats, np.concatenate([e_m, e_L], 1).T * live


def head_loss_bwd(x, W, labels, dloss, scale=1.0, terms=1, exact_logits=False):
    """(dX, err), (dW, err), for statistics as an fp32 forward gives them. terms:
    into how many bf16 numbers a probability (for dX) and a logit's gradient (for
    dW) are split before the matrix products: 1 for bf16 outputs, 3 for fp32. The
    label's own probability is not split for dX: p - 1 and its product are fp32.
    exact_logits: inputs whose logits and all of their partial sums fp32 holds."""
    V, K = W.shape
    live, ids = _live(labels, V)
    live = live & (np.asarray(dloss) != 0)
    xs = np.where(live[:, None], x, 0.0).astype(np.float64)
    W = W.astype(np.float64)
    M = xs.shape[0]
    z, e = _logits(xs, W, scale)
    if exact_logits:
        e = np.zeros_like(e)
    m, L, p, e_m, e_L, rel = _softmax(z, e)
    f = np.where(live, dloss.astype(np.float64) * scale, 0.0)[:, None]
    lost = BF16 ** terms
    # The hardware's exponential, its product with exp(-L), and a bf16 part of
    # it are zero below 2^-126: at most 2^-126 is lost of each.
    e_p = p * (rel + e_L + 4 * U) + 3 * 2.0 ** -126
    hot = np.zeros_like(p)
    hot[np.arange(M), ids] = 1.0
    # sums of fp32 products in the matrix units, as the logits', and over pieces
    adds = lambda n: 2 * U * (n * terms / 8 + 64)  # noqa: E731
    others = np.where(hot > 0, 0.0, p)
    rest = np.take_along_axis(p - hot, ids[:, None], 1)
    dX = f * (others @ W + rest * W[ids])
    # What is rounded before the products is all but the label's entry; at the
    # label the probability's own error remains, and the subtraction's.
    e_dX = np.abs(f) * ((e_p + np.where(hot > 0, 0.0, p + e_p) * (lost + adds(V))) @ np.abs(W)
                        + 3 * U * (np.abs(others @ W) + np.abs(rest * W[ids]))) + 2 * U * np.abs(dX)
    d = f * (p - hot)
    e_d = np.abs(f) * (e_p + U * np.abs(p - hot)) + 2 * U * np.abs(d)
    dW = d.T @ xs
    e_dW = (e_d + np.abs(d) * (lost + adds(M))).T @ np.abs(xs)
    return (dX, e_dX), (dW, e_dW)
