"""GPU tests of the row operators' loops: more rows, pieces, sums and runs than
one round of workgroups (or lanes) takes, for each loop that a kernel has."""
import math

import numpy as np
import pytest
import torch

import qlora_fine_tuning_blockwise_amd as q
from oracle import rows
from row_ops_edges import distill_depth, embed_depth, norm_depth
from test_row_ops_gpu import BF16, DEV, F32, check, host, norm_inputs, randn, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N", [(13000, 500), (7000, 1000), (6500, 2000), (3300, 4000), (3100, 8000),
                                 (600, 16381)])
@pytest.mark.parametrize("x_dtype,y_dtype", [(BF16, BF16), (F32, F32)])
def test_norm_forward_takes_further_rows(M, N, x_dtype, y_dtype):
    """At least two rows for each workgroup (or wave, up to 1024 columns), some
    of them a third."""
    x, _, gamma, beta = norm_inputs(M, N, M, x_dtype, y_dtype, F32)
    for center in (True, False):
        say("norm rows", M, N, x_dtype, center)
        stats = torch.full((2, M), math.nan, device=DEV)
        y = torch.full((M, N), math.nan, dtype=y_dtype, device=DEV)
        q.qlora_norm_fwd(x.to(DEV), gamma.to(DEV), beta.to(DEV), y=y, stats_out=stats,
                         norm=q.NORM_LAYER if center else q.NORM_RMS)
        want, err, wstats, e_stats = rows.norm_fwd(host(x), host(gamma), host(beta), 1e-5, center,
                                                   norm_depth(N))
        check(y, want, err, "y")
        check(stats, wstats, e_stats, "stats")


def test_embed_forward_takes_further_tokens():
    """More than 65536 workgroups of one wide row, and of four narrow ones."""
    for M, V, D in ((65700, 777, 1030), (262400, 777, 24)):
        say("embed rows", M, V, D)
        g = torch.Generator(device=DEV).manual_seed(D)
        W = torch.randn(V, D, generator=g, device=DEV).to(BF16)
        ids = torch.randint(-1, V + 1, (M,), generator=g, device=DEV)
        out = torch.full((M, D), math.nan, device=DEV)
        q.qlora_embed_fwd(W, ids, scale=1.3, out=out)
        live = (ids >= 0) & (ids < V)
        # one product of two fp32 values, rounded once
        want = torch.where(live[:, None], W[ids.clamp(0, V - 1)].float() * np.float32(1.3).item(), 0.0)
        assert torch.equal(out, want)


@pytest.mark.parametrize("M,V,D,run", [(40000, 1300, 9, 33), (4096, 400, 20, 17), (1 << 17, 300, 3, 700),
                                       ((1 << 17) + 5000, 900, 5, 0), (1 << 20, 70000, 2, 0)])
@pytest.mark.parametrize("ids_dtype", [torch.int32, torch.int64])
def test_embed_gradient_of_many_sums_and_runs(M, V, D, run, ids_dtype):
    """More sums that pass a tile's end than the joining launch has workgroups
    for, more than 64 runs to search (from 131073 tokens on), and the most
    tokens that a call takes."""
    say("embed sums", M, V, D, run, ids_dtype)
    g = np.random.default_rng(M + D)
    if run:
        ids = g.permutation(np.arange(M) // run)
    else:
        ids = np.minimum(np.exp(g.random(M) * np.log(V + 1)).astype(np.int64) - 1, V)
        ids[g.random(M) < 0.05] = -1
    ids = torch.from_numpy(ids).to(ids_dtype)
    dY = randn(g, (M, D))
    dW = q.qlora_embed_bwd(dY.to(DEV), ids.to(DEV), V, scale=0.7)
    live = host(ids)
    most = int(np.bincount(live[(live >= 0) & (live < V)]).max())
    want, err = rows.embed_bwd(host(dY), live, V, float(np.float32(0.7)), h=embed_depth(M, most))
    check(dW, want, err, "dW")


def test_distill_takes_further_pieces():
    """More pieces of long rows than workgroups, in both directions, and more
    rows than the finishing launch has workgroups: 8.7 GB of logits."""
    M, V, k = 65600, 66000, 3
    say("distill pieces")
    g = torch.Generator(device=DEV).manual_seed(1)
    z = torch.empty(M, V, dtype=BF16, device=DEV)
    for a in range(0, M, 8192):
        z[a:a + 8192] = torch.randn(z[a:a + 8192].shape, generator=g, device=DEV)
    ids = torch.randint(0, V, (M, k), generator=g, device=DEV)
    ids[5::1000] = -1
    t = torch.randn(M, k, generator=g, device=DEV)
    dl = 0.5 + torch.rand(M, generator=g, device=DEV)
    loss = torch.full((M,), math.nan, device=DEV)
    stats = torch.full((2, M), math.nan, device=DEV)
    q.qlora_distill_fwd(z, ids, t, temperature=2.0, loss=loss, stats_out=stats)
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(stats).all())
    dz = torch.full((M, V), math.nan, dtype=BF16, device=DEV)
    q.qlora_distill_bwd(z, ids, t, dl, stats, temperature=2.0, dlogits=dz)
    for a in range(0, M, 8192):
        assert bool(torch.isfinite(dz[a:a + 8192]).all())
    h = distill_depth(V)
    # items are (row, piece) in order: rows around the places where a round of
    # 65536 workgroups ends, with three pieces, five, and one
    at = sorted({0, 5, 13106, 13107, 13108, 21844, 21845, 21846, 26214, 26215, 43690, 43691, 43692,
                 65535, 65536, 65537, 65598, 65599})
    for m in at:
        r = slice(m, m + 1)
        want, err, wstats, e_stats = rows.distill_fwd(host(z[r]), host(ids[r]), host(t[r]), 2.0, h)
        check(loss[r], want, err, f"loss {m}")
        check(stats[:, r], wstats, e_stats, f"stats {m}")
        want, err = rows.distill_bwd(host(z[r]), host(ids[r]), host(t[r]), host(dl[r]), 2.0, h)
        check(dz[r], want, err, f"dlogits {m}")


def test_distill_takes_further_short_rows():
    """One piece a row, more rows than workgroups, entries of 64-bit ids up to
    the most that a row may have."""
    M, V, k = 66000, 70, 1024
    say("distill short rows")
    g = np.random.default_rng(2)
    z, t = randn(g, (M, V), BF16, 2.0), randn(g, (M, k), BF16)
    ids = torch.from_numpy(g.integers(-2, V + 2, (M, k)))
    dl = randn(g, M)
    stats = torch.empty(2, M, device=DEV)
    args = (z.to(DEV), ids.to(DEV), t.to(DEV))
    loss = q.qlora_distill_fwd(*args, stats_out=stats)
    dz = q.qlora_distill_bwd(*args, dl.to(DEV), stats, grad_dtype=F32)
    for a in (0, 20000, 65500):
        r = slice(a, a + 500)
        want, err, wstats, e_stats = rows.distill_fwd(host(z[r]), host(ids[r]), host(t[r]), 1.0,
                                                      distill_depth(V))
        check(loss[r], want, err, "loss")
        check(stats[:, r], wstats, e_stats, "stats")
        want, err = rows.distill_bwd(host(z[r]), host(ids[r]), host(t[r]), host(dl[r]), 1.0,
                                     distill_depth(V))
        check(dz[r], want, err, "dlogits")
