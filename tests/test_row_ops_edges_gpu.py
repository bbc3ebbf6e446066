"""GPU tests of the row operators in which one term at a border of a vector, a
round, a tile or a workgroup decides the result (row_ops_edges.py), with error
bounds of the kernels' own depths of summation."""
import math

import numpy as np
import pytest
import torch

import qlora_fine_tuning_blockwise_amd as q
from oracle import rows
from row_ops_edges import (distill_case, distill_depth, embed_case, embed_depth, norm_case, norm_depth,
                           norm_rows_depth, rows_case)
from test_row_ops_edges_host import NORM_WIDTHS, VOCABULARIES
from test_row_ops_gpu import BF16, DEV, F32, check, host, say, strided

pytestmark = pytest.mark.gpu

CODES = [(x, y, d) for x in (BF16, F32) for y in (BF16, F32) for d in (BF16, F32)]


@pytest.mark.parametrize("N", NORM_WIDTHS + [1, 3, 8, 512, 1024, 2048, 4096, 8192])
@pytest.mark.parametrize("center", [True, False])
def test_a_term_of_a_normed_row(N, center):
    if N < 5:
        x, dY = np.full((2, N), 1.5, np.float32), np.ones((2, N), np.float32)
    else:
        x, dY, _ = norm_case(N, N)
    kind, h = (q.NORM_LAYER if center else q.NORM_RMS), norm_depth(N)
    M = x.shape[0]
    for x_dtype, y_dtype in ((BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)):
        say("norm edge", N, center, x_dtype, y_dtype)
        xt, dt = torch.from_numpy(x).to(x_dtype), torch.from_numpy(dY).to(y_dtype)
        xv, _ = strided(xt, 1, lead=1)
        dv, _ = strided(dt, 2, lead=0)
        stats = torch.empty(2, M, device=DEV)
        y = q.qlora_norm_fwd(xv, norm=kind, y_dtype=y_dtype, stats_out=stats)
        want, err, wstats, e_stats = rows.norm_fwd(host(xt), None, None, 1e-5, center, h)
        check(y, want, err, "y")
        check(stats, wstats, e_stats, "stats")
        (wX, eX), _, _ = rows.norm_bwd(host(dt), host(xt), None, 1e-5, center, h)
        for d_dtype in (BF16, F32):
            for given in (stats, None):
                dX, _, _ = q.qlora_norm_bwd(dv, xv, norm=kind, stats=given, dx_dtype=d_dtype,
                                            want_dgamma=False, want_dbeta=False)
                check(dX, wX, eX, f"dX {d_dtype}")


@pytest.mark.parametrize("N", [64, 1000, 2000, 4000, 8000, 16381])
@pytest.mark.parametrize("i", range(8))
def test_every_type_build_of_the_norm_gradient(N, i):
    """All types of x, dY and dX at every count of threads a row has, with more
    rows than the workgroups hold at once (and, at the end, fewer)."""
    x_dtype, y_dtype, d_dtype = CODES[i]
    M = {64: 4133, 1000: 2085, 2000: 1061, 4000: 549, 8000: 293, 16381: 293}[N]
    center = (i + N // 1000) % 2 == 0
    say("norm types", M, N, x_dtype, y_dtype, d_dtype, center)
    x, dY, _ = rows_case(M, N, M)
    xt, dt = torch.from_numpy(x).to(x_dtype), torch.from_numpy(dY).to(y_dtype)
    gamma = torch.from_numpy(1 + 0.3 * np.random.default_rng(i).standard_normal(N).astype(np.float32))
    dX, dg, db = q.qlora_norm_bwd(dt.to(DEV), xt.to(DEV), gamma.to(DEV),
                                  norm=q.NORM_LAYER if center else q.NORM_RMS, dx_dtype=d_dtype)
    (wX, eX), (wg, eg), (wb, eb) = rows.norm_bwd(host(dt), host(xt), host(gamma), 1e-5, center,
                                                 norm_depth(N), norm_rows_depth(M, N))
    check(dX, wX, eX, "dX")
    check(dg, wg, eg, "dgamma")
    check(db, wb, eb, "dbeta")


@pytest.mark.parametrize("V", VOCABULARIES)
@pytest.mark.parametrize("z_dtype", [BF16, F32])
@pytest.mark.parametrize("extra,lead", [(None, 0), (0, 0), (1, 1), (5, 3)])
def test_a_term_of_the_logits(V, z_dtype, extra, lead):
    """extra None: rows that begin on a line, each border at its round place."""
    if extra is None:
        extra = -V % 64
    T = 2.0 if V % 2 else 1.0
    say("distill edge", V, z_dtype, extra, lead)
    z, ids, t, at = distill_case(V, T, V)
    zt = torch.from_numpy(z).to(z_dtype)
    M = zt.shape[0]
    zv, _ = strided(zt, extra, lead)
    gv, gbuf = strided(torch.zeros(M, V, dtype=F32 if V % 2 else z_dtype), extra, lead)
    stats = torch.empty(2, M, device=DEV)
    args = (zv, torch.from_numpy(ids).to(DEV), torch.from_numpy(t).to(DEV))
    loss = q.qlora_distill_fwd(*args, temperature=T, stats_out=stats)
    q.qlora_distill_bwd(*args, torch.ones(M, device=DEV), stats, temperature=T, dlogits=gv)
    torch.cuda.synchronize()
    h = distill_depth(V)
    want, err, wstats, e_stats = rows.distill_fwd(host(zt), ids, t, T, h)
    check(loss, want, err, "loss")
    check(stats, wstats, e_stats, "stats")
    wz, ez = rows.distill_bwd(host(zt), ids, t, np.ones(M), T, h)
    check(gv, wz, ez, "dlogits")
    assert int(torch.isnan(gbuf).sum()) == gbuf.numel() - M * V


@pytest.mark.parametrize("M", [20, 32, 33, 600, 4096, 5000, 9000])
@pytest.mark.parametrize("y_dtype,grad_dtype", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
def test_a_token_of_a_shared_id(M, y_dtype, grad_dtype):
    say("embed edge", M, y_dtype, grad_dtype)
    dY, _ = embed_case(M, M)
    dt = torch.from_numpy(dY).to(y_dtype)
    dv, _ = strided(dt, 1, lead=1)
    ids = np.full(M, 2)
    dW = q.qlora_embed_bwd(dv, torch.from_numpy(ids).to(DEV), 4, scale=0.7, grad_dtype=grad_dtype)
    want, err = rows.embed_bwd(host(dt), ids, 4, float(np.float32(0.7)), h=embed_depth(M, M))
    check(dW, want, err, "dW")


def test_a_token_of_many_ids():
    """Sums that begin and end anywhere in a tile, each held to its own depth."""
    g = np.random.default_rng(4)
    for M, V in ((4000, 90), (6000, 40), (20000, 300), (21000, 300)):
        say("embed edge ids", M, V)
        ids = g.integers(0, V, M)
        dY = g.standard_normal((M, 12)).astype(np.float32)
        dW = q.qlora_embed_bwd(torch.from_numpy(dY).to(DEV), torch.from_numpy(ids).to(DEV), V)
        most = int(np.bincount(ids).max())
        want, err = rows.embed_bwd(dY, ids, V, 1.0, h=embed_depth(M, most))
        check(dW, want, err, "dW")
        assert math.isfinite(float(dW.abs().max()))
