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
