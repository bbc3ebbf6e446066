"""CPU tests of the inputs and tolerances that the GPU tests of single terms
use: one term lost, or counted twice, at any of their places leaves at least
twice the tolerance."""
import numpy as np
import pytest

from oracle import rows
from row_ops_edges import (distill_case, distill_depth, embed_case, embed_depth, norm_case, norm_depth,
                           norm_rows_depth, rows_case, tolerance)

EPS32, EPS16 = 2.0 ** -23, 2.0 ** -7
NORM_WIDTHS = [5, 9, 64, 511, 513, 1027, 2049, 4101, 8193, 16381, 16384]
VOCABULARIES = [300, 8193, 65473, 65474, 70003, 200000]


def caught(got, want, err, eps):
    """Whether a wrong result is beyond twice the tolerance in some place of
    every row."""
    off = np.abs(got - want) > 2 * tolerance(want, err, eps)
    return off.reshape(off.shape[0], -1).any(1).all()


@pytest.mark.parametrize("N", NORM_WIDTHS)
@pytest.mark.parametrize("center", [True, False])
def test_a_term_of_a_normed_row(N, center):
    x, dY, at = norm_case(N, N)
    r, h, eps = np.arange(len(at)), norm_depth(N), 1e-5
    y, err, stats, e_stats = rows.norm_fwd(x, None, None, eps, center, h)
    (dX, eX), _, _ = rows.norm_bwd(dY, x, None, eps, center, h)
    x64, big = x.astype(np.float64), x[r, at].astype(np.float64)
    mean, rstd = stats[0], stats[1]
    xh = (x64 - mean[:, None]) * rstd[:, None]
    for times in (-1, 1):   # lost, counted twice
        m2 = mean + times * big / N if center else mean
        d2 = x64 - m2[:, None]
        var = ((d2 * d2).sum(1) + times * d2[r, at] ** 2) / N
        s2 = 1 / np.sqrt(var + eps)
        assert caught(s2[:, None], rstd[:, None], e_stats[1][:, None], EPS32)
        assert not center or caught(m2[:, None], mean[:, None], e_stats[0][:, None], EPS32)
        for e in (EPS32, EPS16):
            assert caught(d2 * s2[:, None], y, err, e)
        # the sums of the backward, with the statistics given
        g = dY.astype(np.float64)
        c1 = ((g.sum(1) + times * g[r, at]) / N if center else 0 * mean)[:, None]
        c2 = (((g * xh).sum(1) + times * (g * xh)[r, at]) / N)[:, None]
        c1r, c2r = (g.mean(1) if center else 0 * mean)[:, None], (g * xh).mean(1)[:, None]
        for a, b in ((c1, c2r), (c1r, c2)):
            if not center and a is c1:
                continue
            for e in (EPS32, EPS16):
                assert caught(rstd[:, None] * (g - a - xh * b), dX, eX, e)


@pytest.mark.parametrize("V", VOCABULARIES)
@pytest.mark.parametrize("T", [1.0, 2.0])
def test_a_term_of_the_logits(V, T):
    z, ids, t, at = distill_case(V, T, V)
    loss, err, stats, e_stats = rows.distill_fwd(z, ids, t, T, distill_depth(V))
    z64, r = z.astype(np.float64), np.arange(at.size)
    w = np.exp((z64 - stats[0][:, None]) / T)
    for times in (-1, 1):
        L = np.log(w.sum(1) + times * w[r, at])
        assert caught(L[:, None], stats[1][:, None], e_stats[1][:, None], EPS32)
        assert caught((loss + T * T * (L - stats[1]))[:, None], loss[:, None], err[:, None], EPS32)


@pytest.mark.parametrize("M", [600, 5000, 9000])
def test_a_token_of_a_shared_id(M):
    dY, at = embed_case(M, M)
    want, err = rows.embed_bwd(dY, np.full(M, 2), 4, 0.7, h=embed_depth(M, M))
    for times in (-1, 1):
        off = want[2] + times * 0.7 * dY[at, np.arange(len(at))]
        assert caught(off[:, None], want[2][:, None], err[2][:, None], EPS32)


@pytest.mark.parametrize("M,N", [(4133, 64), (1061, 2000), (549, 4000), (293, 16381)])
def test_a_row_of_the_sums_over_rows(M, N):
    x, dY, at = rows_case(M, N, M)
    _, (dg, eg), (db, eb) = rows.norm_bwd(dY, x, None, 1e-5, True, norm_depth(N), norm_rows_depth(M, N))
    n = min(N, 4 * len(at))
    j = np.arange(n)
    m = np.array(at)[j % len(at)]
    _, _, stats, _ = rows.norm_fwd(x, None, None, 1e-5, True)
    xh = (x[m, j] - stats[0][m]) * stats[1][m]
    for times in (-1, 1):
        assert caught((dg[j] + times * dY[m, j] * xh)[:, None], dg[j][:, None], eg[j][:, None], EPS32)
        assert caught((db[j] + times * dY[m, j])[:, None], db[j][:, None], eb[j][:, None], EPS32)
