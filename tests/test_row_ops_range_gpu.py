"""The norm over the range of values that its declaration names, at the widths
where the sum of a row's squares leaves fp32 first."""
import numpy as np
import pytest
import torch

import qlora_fine_tuning_blockwise_amd as q
from oracle import rows
from test_row_ops_gpu import BF16, DEV, F32, check, host, randn, say

pytestmark = pytest.mark.gpu

WIDTHS = [1, 3, 4, 255, 256, 257, 1000, 4096, 5000, 16384]


def both_ways(x, dY, gamma, eps, center):
    kind = q.NORM_LAYER if center else q.NORM_RMS
    stats = torch.empty(2, x.shape[0], device=DEV)
    y = q.qlora_norm_fwd(x.to(DEV), gamma.to(DEV), eps=eps, norm=kind, stats_out=stats)
    want, err, wstats, e_stats = rows.norm_fwd(host(x), host(gamma), None, eps, center)
    check(y, want, err, "y")
    check(stats, wstats, e_stats, "stats")
    (wX, eX), (wg, eg), _ = rows.norm_bwd(host(dY), host(x), host(gamma), eps, center)
    for given in (stats, None):
        dX, dg, _ = q.qlora_norm_bwd(dY.to(DEV), x.to(DEV), gamma.to(DEV), eps=eps, norm=kind, stats=given)
        check(dX, wX, eX, "dX")
        check(dg, wg, eg, "dgamma")


def rows_of_size(g, N, size, dtype):
    """Rows whose values all have nearly that size, of either sign; the second
    one has a mean of that size as well and deviations of a quarter."""
    sign = np.where(g.random((2, N)) < 0.5, -1.0, 1.0)
    x = size * sign * (1.0 - 0.25 * g.random((2, N)))
    x[1] = size * (0.7 + 0.25 * g.random(N))
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_norm_of_rows_up_to_the_stated_size(N, dtype):
    """Values next to 2^60: N of their squares pass 2^128 from 256 columns on."""
    g = np.random.default_rng(N)
    for center in (True, False):
        if center and N == 1:
            continue   # a deviation of zero, whatever the value
        say("norm large", N, dtype, center)
        x = rows_of_size(g, N, 2.0 ** 60 * 0.999, dtype)
        dY = randn(g, (2, N), dtype)
        gamma = randn(g, N, F32, 0.3, 1.0)
        both_ways(x, dY, gamma, 1e-5, center)


@pytest.mark.parametrize("N", WIDTHS[1:])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_norm_without_eps_down_to_the_stated_size(N, dtype):
    """eps = 0 and deviations next to 2^-50, the smallest that it takes."""
    g = np.random.default_rng(N)
    for center in (True, False):
        say("norm small", N, dtype, center)
        x = rows_of_size(g, N, 2.0 ** -48, dtype)
        dY = randn(g, (2, N), dtype)
        gamma = randn(g, N, F32, 0.3, 1.0)
        both_ways(x, dY, gamma, 0.0, center)


# --------------------------------------------------------------- distillation
U = 2.0 ** -24


@pytest.mark.parametrize("V", [5000, 130000])
@pytest.mark.parametrize("T", [1.0, 2.0])
def test_distill_gradient_of_a_nearly_even_row(V, T):
    """Logits within one temperature of the largest, so that q is about 1 / V:
    with m and L as given, q may be off by the roundings of (z - m) log2(e) /
    (2 T) (its factor's |d / T| / 2, its own 0.7), twice the root's exponential
    (one step of a value from 0.6 to 1: 1.7 each), exp(-L) (2) and the three
    products (1 each), whatever L is: nine times 2^-24 with |d / T| <= 1."""
    say("distill even", V, T)
    g = np.random.default_rng(V)
    M = 6
    z = (16.0 - T * g.random((M, V))).astype(np.float32)   # z - m is exact
    ids = np.full((M, 1), V - 1)
    z64, m = z.astype(np.float64), z.max(1).astype(np.float64)
    L = np.log(np.exp((z64 - m[:, None]) / T).sum(1)).astype(np.float32)
    stats = torch.from_numpy(np.stack([m.astype(np.float32), L])).to(DEV)
    dz = q.qlora_distill_bwd(torch.from_numpy(z).to(DEV), torch.from_numpy(ids).to(DEV),
                             torch.zeros(M, 1, device=DEV), torch.ones(M, device=DEV), stats, temperature=T)
    want = T * np.exp((z64 - m[:, None]) / T - L.astype(np.float64)[:, None])
    off = np.abs(dz.double().cpu().numpy()[:, :-1] / want[:, :-1] - 1.0).max()
    assert off <= 9 * U, off / U


@pytest.mark.parametrize("k", [8, 64, 1000])
def test_distill_loss_of_a_far_student(k):
    """A student that gives every entry of the teacher the same q: the loss is
    sum p log p - log q, and what p's sum misses of one counts log q times.
    Rounding errors taken as independent have a root mean square of 2^-24 /
    sqrt(3) of the value at most. With p as exponentials over their sum, p's sum
    is off by the roundings of that sum (at most k / 64 of them and 6, fewer
    count as its parts are smaller), the loss by as many and by the one of log q:
    with the three largest of each sum counted in full, sqrt(3 + 3 + 1) of them,
    1.6 times 2^-24 of log q over the rows."""
    say("distill far", k)
    g = np.random.default_rng(k)
    M, V = 2000, 1200
    z = np.full((M, V), 0.0, np.float32)
    z[:, 1100:] = 64.0 + 16 * g.random((M, 1))       # log q of the others: that and log 100
    ids = np.stack([g.permutation(1100)[:k] for _ in range(M)])
    t = (3 * g.standard_normal((M, k))).astype(np.float32)
    loss = q.qlora_distill_fwd(torch.from_numpy(z).to(DEV), torch.from_numpy(ids).to(DEV),
                               torch.from_numpy(t).to(DEV))
    p = np.exp(t - t.max(1, keepdims=True).astype(np.float64))
    p /= p.sum(1, keepdims=True)
    far = z[:, 1100].astype(np.float64) + np.log(100.0)
    want = (p * np.log(p)).sum(1) + far
    off = (loss.double().cpu().numpy() - want) / far
    say("off", k, np.sqrt((off * off).mean()) / U, np.abs(off).max() / U)
    assert np.sqrt((off * off).mean()) <= 1.6 * U
