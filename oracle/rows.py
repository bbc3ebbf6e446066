"""The row operators (token embedding, norm, distillation from a teacher's top
logits) and their gradients in 64 bits, with numpy alone, each from its
formula, and with the bound of the error that fp32 arithmetic may make of
them.

Every function that returns (values, err) counts in `err` the roundings of an
fp32 evaluation, u = 2^-24 each: a sum of terms a_i with at most h additions
between a term and the result is off by at most h u sum |a_i| (to first
order; `h` is given by the caller or taken as the count of terms), and an
error of an operand is carried to the result by the derivative. What the
output's own type rounds away is not part of `err`.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24


# ------------------------------------------------------------------ embedding
def embed_fwd(W, ids, scale):
    ids = np.asarray(ids, np.int64)
    live = (ids >= 0) & (ids < W.shape[0])
    out = np.zeros((ids.size, W.shape[1]))
    out[live] = scale * W[ids[live]].astype(np.float64)
    return out, U * np.abs(out)


def embed_bwd(dY, ids, V, scale, dW=None, h=None):
    """dW given: the gradient is added to it. h: additions between a token's
    row and its sum (default: as many as the id has tokens)."""
    ids = np.asarray(ids, np.int64)
    live = (ids >= 0) & (ids < V)
    out = np.zeros((V, dY.shape[1]))
    size = np.zeros((V, dY.shape[1]))
    rows = dY[live].astype(np.float64)
    np.add.at(out, ids[live], scale * rows)
    np.add.at(size, ids[live], np.abs(scale * rows))
    count = np.bincount(ids[live], minlength=V)[:, None]
    err = U * ((count if h is None else np.minimum(count, h)) + 1) * size
    if dW is not None:
        out = out + dW
        err = err + U * np.where(count > 0, np.abs(out), 0.0)
    return out, err


# ----------------------------------------------------------------------- norm
def _stats(x, eps, center, h):
    """Mean, rstd and xh of the rows, and bounds of the errors of the mean
    (absolute), of rstd (relative) and of xh (absolute)."""
    x = x.astype(np.float64)
    N = x.shape[1]
    mean = x.mean(1, keepdims=True) if center else np.zeros((x.shape[0], 1))
    d = x - mean
    var = (d * d).mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt(var + eps)
    xh = d * rstd
    # sum and product with 1/N (itself rounded)
    e_mean = (h + 2) * U * np.abs(x).mean(1, keepdims=True) if center else np.zeros_like(mean)
    # The variance around a mean that is off by e is larger by e^2; each
    # deviation is rounded once, its square is summed with h additions, then
    # the product with 1/N, the sum with eps, the root and the division.
    share = var / (var + eps)
    e_rstd = 0.5 * ((h + 6) * U * share + (e_mean * rstd) ** 2) + 4 * U
    e_xh = rstd * e_mean + np.abs(xh) * (e_rstd + 2 * U)
    return mean, rstd, xh, e_mean, e_rstd, e_xh


def norm_fwd(x, gamma, beta, eps, center, h=None):
    h = x.shape[1] if h is None else h
    g = 1.0 if gamma is None else gamma.astype(np.float64)
    b = 0.0 if beta is None else beta.astype(np.float64)
    mean, rstd, xh, e_mean, e_rstd, e_xh = _stats(x, eps, center, h)
    y = xh * g + b
    err = np.abs(g) * e_xh + U * (np.abs(xh * g) + np.abs(y))
    stats = np.concatenate([mean, rstd], 1).T
    e_stats = np.concatenate([e_mean + U * np.abs(mean), rstd * e_rstd], 1).T
    return y, err, stats, e_stats


def norm_bwd(dY, x, gamma, eps, center, h=None, hm=None):
    """(dX, err), (dgamma, err), (dbeta, err). hm: additions between a row and
    the sums over the rows (default: as many as there are rows)."""
    h = x.shape[1] if h is None else h
    M = x.shape[0] if hm is None else min(hm, x.shape[0])
    dY = dY.astype(np.float64)
    _, rstd, xh, _, e_rstd, e_xh = _stats(x, eps, center, h)
    g = dY if gamma is None else dY * gamma.astype(np.float64)
    c1 = g.mean(1, keepdims=True) if center else np.zeros_like(rstd)
    c2 = (g * xh).mean(1, keepdims=True)
    dX = rstd * (g - c1 - xh * c2)
    e_c1 = (h + 3) * U * np.abs(g).mean(1, keepdims=True) if center else 0.0
    e_c2 = (h + 4) * U * np.abs(g * xh).mean(1, keepdims=True) + (np.abs(g) * e_xh).mean(1, keepdims=True)
    parts = np.abs(g) + np.abs(c1) + np.abs(xh * c2)
    err = rstd * (e_c1 + np.abs(xh) * e_c2 + e_xh * np.abs(c2) + 4 * U * parts) \
        + np.abs(dX) * (e_rstd + 2 * U)
    dg = dY * xh
    e_dg = (np.abs(dY) * e_xh).sum(0) + (M + 1) * U * np.abs(dg).sum(0)
    return (dX, err), (dg.sum(0), e_dg), (dY.sum(0), M * U * np.abs(dY).sum(0))


# --------------------------------------------------------------- distillation
def _teacher(ids, t, V, T):
    ids = np.asarray(ids, np.int64)
    t = t.astype(np.float64)
    live = (ids >= 0) & (ids < V) & ~(t == -np.inf)
    some = live.any(1)
    a = np.where(live, t, -np.inf) / T
    top = np.where(some, a.max(1), 0.0)[:, None]
    a = np.where(live, a - top, 0.0)
    total = np.log(np.where(some, np.where(live, np.exp(a), 0.0).sum(1), 1.0))[:, None]
    logp = a - total
    k = ids.shape[1]
    p = np.where(live, np.exp(logp), 0.0)
    # the exponents' own roundings, the sum over k and its logarithm
    e_logp = U * (2 * np.abs(a) + np.abs(total) + np.abs(logp) + k + 8
                  + 2 * (p * np.abs(a)).sum(1, keepdims=True))
    return np.where(live, ids, 0), live, some, p, logp, e_logp


def _student(z, T, h):
    z = z.astype(np.float64)
    m = z.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        a = (z - m) / T
    w = np.exp(a)
    total = w.sum(1, keepdims=True)
    L = np.log(total)
    far = np.where(w > 0, w * np.abs(np.where(w > 0, a, 0.0)), 0.0).sum(1, keepdims=True) / total
    e_L = U * (h + 8 + 4 * far + 2 * np.abs(L))
    return m, a, L, e_L


def distill_fwd(z, ids, t, T, h=None):
    """loss, err, stats, err of the stats."""
    V = z.shape[1]
    h = V if h is None else h
    ids, live, some, p, logp, e_logp = _teacher(ids, t, V, T)
    with np.errstate(invalid="ignore", divide="ignore"):
        m, a, L, e_L = _student(np.where(some[:, None], z, 0.0), T, h)
        at = np.take_along_axis(a, ids, 1)
        diff = logp - (at - L)
        use = p > 0
        terms = np.where(use, p * np.where(use, diff, 0.0), 0.0)
        loss = T * T * terms.sum(1)
        fin = np.where(np.isfinite(at), np.abs(at), 0.0)
        fd = np.where(np.isfinite(diff), np.abs(diff), 0.0)
        e = p * (e_logp + e_L + U * (2 * fin + 2 * fd + np.abs(L))) \
            + p * fd * (e_logp + 4 * U + ids.shape[1] * U)
    err = T * T * e.sum(1) + 4 * U * np.where(np.isfinite(loss), np.abs(loss), 0.0)
    stats = np.concatenate([m, L], 1).T * some
    return np.where(some, loss, 0.0), err * some, stats, np.concatenate([0 * m, e_L], 1).T * some


def distill_bwd(z, ids, t, dloss, T, h=None):
    """Gradient and err, for statistics as an fp32 forward gives them."""
    V = z.shape[1]
    h = V if h is None else h
    given = ids
    ids, live, some, p, logp, e_logp = _teacher(ids, t, V, T)
    some = some & (dloss != 0)
    with np.errstate(invalid="ignore", divide="ignore"):
        m, a, L, e_L = _student(np.where(some[:, None], z, 0.0), T, h)
        q = np.exp(a - L)
        e_q = q * (e_L + U * (4 * np.where(q > 0, np.abs(a), 0.0) + 3 * np.abs(L) + 6))
    taken = np.zeros_like(q)
    e_p = np.zeros_like(q)
    rows = np.broadcast_to(np.arange(z.shape[0])[:, None], given.shape)
    np.add.at(taken, (rows[live], ids[live]), p[live])
    np.add.at(e_p, (rows[live], ids[live]), (p * (e_logp + (4 + given.shape[1]) * U))[live])
    s = (dloss.astype(np.float64) * T)[:, None]
    out = np.where(some[:, None], s * (q - taken), 0.0)
    err = np.abs(s) * (e_q + e_p + 2 * U * np.abs(q - taken)) + 2 * U * np.abs(out)
    return out, np.where(some[:, None], err, 0.0)
