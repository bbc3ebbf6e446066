"""GPU tests of the row operators (embedding, norm, distillation) against
their 64-bit forms: |got - want| <= err + half a step of the output's type,
where err is the bound of fp32 arithmetic that oracle/rows.py derives for the
values at hand."""
import math

import numpy as np
import pytest
import torch

import qlora_fine_tuning_blockwise_amd as q
from oracle import rows
from qlora_fine_tuning_blockwise_amd import _lib

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F32, BF16 = torch.float32, torch.bfloat16


def say(*a):
    print(*a, flush=True)


def host(t):
    return t.detach().float().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def check(got, want, err, name):
    """Half a step of the output's type is eps / 2 relative to the value (for
    bf16 and fp32, whose smallest normal is 2^-126, half of the smallest
    subnormal below it)."""
    eps = torch.finfo(got.dtype).eps
    low = 2.0 ** -126 * eps
    g = got.detach().double().cpu().numpy()
    assert g.shape == want.shape, (name, g.shape, want.shape)
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(g), np.isnan(want)), f"{name}: NaN elsewhere"
    assert np.array_equal(g[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)]), f"{name}: infinities"
    with np.errstate(invalid="ignore"):
        off = np.abs(g - want)[fin]
        tol = (np.broadcast_to(err, want.shape) + 0.5 * eps * (np.abs(want) + err) + low)[fin]
    bad = off > tol
    if bad.any():
        i = int(np.argmax(off - tol))
        raise AssertionError(f"{name}: {bad.sum()} of {bad.size} beyond the bound, worst "
                             f"{off[i]:.3e} against {tol[i]:.3e}")


def randn(g, shape, dtype=F32, scale=1.0, shift=0.0):
    return torch.from_numpy((g.standard_normal(shape) * scale + shift).astype(np.float32)).to(dtype)


def strided(t, extra, lead=0):
    """A device view with t's values whose rows lie `extra` elements apart more
    than their width, starting `lead` elements into the buffer; and the buffer,
    whose other elements are NaN."""
    M, N = t.shape
    buf = torch.full((lead + M * (N + extra),), math.nan, dtype=t.dtype, device=DEV)
    view = buf[lead:].view(M, N + extra)[:, :N]
    view.copy_(t)
    return view, buf


# ----------------------------------------------------------------------- norm
NORM_SHAPES = [(1, 1), (2, 3), (1, 7), (3, 8), (5, 64), (2, 511), (3, 512), (3, 513), (2, 1024),
               (2, 1025), (1, 2047), (3, 2048), (2, 2049), (1, 4096), (3, 4101), (2, 8192),
               (2, 8193), (1, 16384), (2, 16381), (300, 100), (1000, 65), (523, 1030)]


def norm_inputs(M, N, seed, x_dtype, y_dtype, w_dtype):
    g = np.random.default_rng(seed)
    x = randn(g, (M, N), scale=1.5, shift=0.4) * torch.from_numpy(
        np.exp(0.5 * g.standard_normal((M, 1))).astype(np.float32))
    return (x.to(x_dtype), randn(g, (M, N), y_dtype), randn(g, N, w_dtype, 0.3, 1.0),
            randn(g, N, w_dtype, 0.2))


@pytest.mark.parametrize("i,shape", list(enumerate(NORM_SHAPES)))
@pytest.mark.parametrize("center", [True, False])
def test_norm_forward(i, shape, center):
    M, N = shape
    types = [(BF16, BF16, BF16), (F32, BF16, F32), (BF16, F32, F32), (F32, F32, BF16)]
    x_dtype, y_dtype, w_dtype = types[(i + center) % 4]
    say("norm fwd", M, N, center, x_dtype, y_dtype, w_dtype)
    x, _, gamma, beta = norm_inputs(M, N, 10 + i, x_dtype, y_dtype, w_dtype)
    gamma = None if i % 5 == 4 else gamma
    beta = None if i % 3 == 2 else beta
    xv, _ = strided(x, i % 4, lead=i % 3)
    yv, ybuf = strided(torch.zeros(M, N, dtype=y_dtype), (i + 1) % 3, lead=i % 2)
    stats = torch.empty(2, M, device=DEV)
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    out = q.qlora_norm_fwd(xv, dev(gamma), dev(beta), eps=1e-5,
                           norm=q.NORM_LAYER if center else q.NORM_RMS, y=yv, stats_out=stats)
    torch.cuda.synchronize()
    assert out is yv
    want, err, wstats, e_stats = rows.norm_fwd(host(x), None if gamma is None else host(gamma),
                                               None if beta is None else host(beta), 1e-5, center)
    check(yv, want, err, "y")
    check(stats, wstats, e_stats, "stats")
    assert int(torch.isnan(ybuf).sum()) == ybuf.numel() - M * N  # nothing else was written


@pytest.mark.parametrize("i,shape", list(enumerate(NORM_SHAPES)))
@pytest.mark.parametrize("center", [True, False])
def test_norm_backward(i, shape, center):
    M, N = shape
    types = [(BF16, BF16, BF16), (F32, BF16, F32), (BF16, F32, F32), (F32, F32, BF16),
             (BF16, BF16, F32)]
    x_dtype, y_dtype, d_dtype = types[(i + center) % 5]
    say("norm bwd", M, N, center, x_dtype, y_dtype, d_dtype)
    x, dY, gamma, _ = norm_inputs(M, N, 40 + i, x_dtype, y_dtype, BF16)
    gamma = None if i % 5 == 4 else gamma
    xv, _ = strided(x, i % 3, lead=i % 2)
    dv, _ = strided(dY, (i + 1) % 4, lead=i % 3)
    stats = None
    if i % 2:
        stats = torch.empty(2, M, device=DEV)
        q.qlora_norm_fwd(xv, norm=q.NORM_LAYER if center else q.NORM_RMS, stats_out=stats)
    kw = dict(eps=1e-5, norm=q.NORM_LAYER if center else q.NORM_RMS, stats=stats, dx_dtype=d_dtype,
              grad_dtype=F32 if i % 4 else BF16)
    gd = None if gamma is None else gamma.to(DEV)
    dX, dg, db = q.qlora_norm_bwd(dv, xv, gd, **kw)
    torch.cuda.synchronize()
    (wX, eX), (wg, eg), (wb, eb) = rows.norm_bwd(host(dY), host(x),
                                                 None if gamma is None else host(gamma), 1e-5, center)
    check(dX, wX, eX, "dX")
    check(dg, wg, eg, "dgamma")
    check(db, wb, eb, "dbeta")
    # each output alone has the bits of the call that asks for all
    for want in ((True, False, False), (False, True, False), (False, False, True)):
        got = q.qlora_norm_bwd(dv, xv, gd, want_dx=want[0], want_dgamma=want[1], want_dbeta=want[2], **kw)
        for a, b, w in zip(got, (dX, dg, db), want):
            assert (a is None) == (not w) and (a is None or torch.equal(a, b))


def test_norm_many_rows_of_a_long_batch():
    """More rows than workgroups times row groups: every loop runs."""
    for M, N in ((9000, 48), (1500, 1500)):
        say("norm rows", M, N)
        x, dY, gamma, beta = norm_inputs(M, N, 5, F32, F32, F32)
        y = q.qlora_norm_fwd(x.to(DEV), gamma.to(DEV), beta.to(DEV))
        dX, dg, db = q.qlora_norm_bwd(dY.to(DEV), x.to(DEV), gamma.to(DEV))
        torch.cuda.synchronize()
        want, err, _, _ = rows.norm_fwd(host(x), host(gamma), host(beta), 1e-5, True)
        check(y, want, err, "y")
        (wX, eX), (wg, eg), (wb, eb) = rows.norm_bwd(host(dY), host(x), host(gamma), 1e-5, True)
        check(dX, wX, eX, "dX")
        check(dg, wg, eg, "dgamma")
        check(db, wb, eb, "dbeta")


def test_norm_of_awkward_rows():
    """A large mean against the deviation, constant rows, tiny and huge rows;
    a row that holds NaN or infinity spoils itself alone."""
    g = np.random.default_rng(3)
    x = randn(g, (8, 700))
    x[0] += 1000.0
    x[1] = 3.25
    x[2] = 0.0
    x[3] *= 1e-18
    x[4] *= 1e15
    x[6, 699] = math.nan
    x[7, 0] = math.inf
    dY, gamma = randn(g, (8, 700)), randn(g, 700, shift=1.0)
    for center in (True, False):
        say("norm awkward", center)
        kind = q.NORM_LAYER if center else q.NORM_RMS
        y = q.qlora_norm_fwd(x.to(DEV), gamma.to(DEV), norm=kind)
        dX, dg, _ = q.qlora_norm_bwd(dY.to(DEV), x.to(DEV), gamma.to(DEV), norm=kind)
        torch.cuda.synchronize()
        want, err, _, _ = rows.norm_fwd(host(x)[:6], host(gamma), None, 1e-5, center)
        check(y[:6], want, err, "y")
        (wX, eX), _, _ = rows.norm_bwd(host(dY)[:6], host(x)[:6], host(gamma), 1e-5, center)
        check(dX[:6], wX, eX, "dX")
        assert torch.isnan(y[6]).all() and torch.isnan(dX[6]).all() and torch.isnan(dX[7]).any()
        assert torch.isnan(dg).any()


def test_norm_with_no_eps():
    """eps = 0: the workgroups' row groups that have no row add nothing."""
    x, dY, gamma, _ = norm_inputs(3, 100, 6, F32, F32, F32)
    for center in (True, False):
        dX, dg, db = q.qlora_norm_bwd(dY.to(DEV), x.to(DEV), gamma.to(DEV), eps=0.0,
                                      norm=q.NORM_LAYER if center else q.NORM_RMS)
        (wX, eX), (wg, eg), (wb, eb) = rows.norm_bwd(host(dY), host(x), host(gamma), 0.0, center)
        check(dX, wX, eX, "dX")
        check(dg, wg, eg, "dgamma")
        check(db, wb, eb, "dbeta")


def test_norm_without_rows():
    dX, dg, db = q.qlora_norm_bwd(torch.empty(0, 70, device=DEV), torch.empty(0, 70, device=DEV),
                                  grad_dtype=BF16)
    assert dX.shape == (0, 70) and not dg.any() and not db.any()
    assert q.qlora_norm_fwd(torch.empty(0, 70, device=DEV)).shape == (0, 70)


def test_norm_gradient_by_differences():
    """The GPU's gradient along a direction against the central difference of
    the 64-bit forward, whose own error is below 1e-7 of it."""
    g = np.random.default_rng(8)
    M, N = 4, 300
    x, dY, gamma, d = randn(g, (M, N), shift=0.3), randn(g, (M, N)), randn(g, N, shift=1.0), \
        g.standard_normal((M, N))
    dX, _, _ = q.qlora_norm_bwd(dY.to(DEV), x.to(DEV), gamma.to(DEV))

    def f(v):
        return (rows.norm_fwd(v, host(gamma), None, 1e-5, True)[0] * host(dY)).sum()
    h, x64 = 1e-5, host(x).astype(np.float64)
    want = (f(x64 + h * d) - f(x64 - h * d)) / (2 * h)
    (wX, eX), _, _ = rows.norm_bwd(host(dY), host(x), host(gamma), 1e-5, True)
    tol = ((eX + 2.0 ** -24 * np.abs(wX)) * np.abs(d)).sum() + 1e-6 * abs(want)
    assert abs((host(dX) * d).sum() - want) <= tol


# ------------------------------------------------------------------ embedding
@pytest.mark.parametrize("M,V,D", [(1, 1, 1), (3, 5, 7), (17, 100, 8), (5, 9, 513), (70, 300, 1024),
                                   (33, 50, 1027), (2000, 999, 40), (9, 3, 5000)])
@pytest.mark.parametrize("w_dtype,out_dtype,ids_dtype", [
    (BF16, BF16, torch.int64), (F32, BF16, torch.int32), (BF16, F32, torch.int32), (F32, F32, torch.int64)])
def test_embed_forward(M, V, D, w_dtype, out_dtype, ids_dtype):
    say("embed fwd", M, V, D, w_dtype, out_dtype, ids_dtype)
    g = np.random.default_rng(M + D)
    W = randn(g, (V, D), w_dtype)
    ids = torch.from_numpy(g.integers(-1, V + 1, M)).to(ids_dtype)
    if ids_dtype == torch.int64 and M > 2:
        ids[1] = 1 << 32   # outside, though its low half is the row 0
    Wv, _ = strided(W, M % 3, lead=M % 2)
    ov, obuf = strided(torch.zeros(M, D, dtype=out_dtype), V % 3, lead=1)
    q.qlora_embed_fwd(Wv, ids.to(DEV), scale=1.3, out=ov)
    torch.cuda.synchronize()
    want, err = rows.embed_fwd(host(W), host(ids), np.float32(1.3).astype(np.float64))
    check(ov, want, err, "out")
    assert int(torch.isnan(obuf).sum()) == obuf.numel() - M * D


def embed_case(M, V, D, y_dtype, grad_dtype, ids, scale=0.7, extra=1, accumulate=False):
    g = np.random.default_rng(M * 7 + D)
    dY = randn(g, (M, D), y_dtype)
    live = (ids >= 0) & (ids < V)
    dv, _ = strided(dY, extra, lead=extra)
    dv[torch.from_numpy(~live).to(DEV)] = math.nan   # rows without an id are not read
    idt = torch.from_numpy(ids).to(DEV)
    old = None
    dW = None
    if accumulate:
        dW = randn(g, (V, D), grad_dtype).to(DEV)
        old = host(dW).astype(np.float64)
    got = q.qlora_embed_bwd(dv, idt, V, scale=scale, grad_dtype=grad_dtype,
                            dW=None if dW is None else dW.clone(), accumulate=accumulate)
    again = q.qlora_embed_bwd(dv, idt, V, scale=scale, grad_dtype=grad_dtype,
                              dW=None if dW is None else dW.clone(), accumulate=accumulate)
    torch.cuda.synchronize()
    want, err = rows.embed_bwd(host(dY), ids, V, float(np.float32(scale)), old)
    check(got, want, err, "dW")
    assert torch.equal(got, again)   # the order of a sum does not depend on the launch
    if accumulate:
        still = np.setdiff1d(np.arange(V), ids)
        assert torch.equal(got[still], dW[still])


@pytest.mark.parametrize("M,V,D", [(1, 1, 1), (1, 3, 3), (2, 5, 7), (5, 100, 8), (37, 20, 65),
                                   (64, 9, 513), (511, 300, 40), (513, 300, 40), (700, 50, 1027),
                                   (4096, 700, 24), (4097, 700, 24), (13001, 5000, 17)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_backward(M, V, D, accumulate):
    say("embed bwd", M, V, D, accumulate)
    g = np.random.default_rng(M)
    ids = np.minimum(np.exp(g.random(M) * np.log(V + 1)).astype(np.int64) - 1, V)  # V: outside
    ids[g.random(M) < 0.1] = -1
    embed_case(M, V, D, BF16 if M % 2 else F32, F32 if D % 2 else BF16, ids, accumulate=accumulate)
    embed_case(M, V, D, F32 if M % 2 else BF16, BF16 if D % 2 else F32, ids.astype(np.int32),
               accumulate=accumulate)


@pytest.mark.parametrize("M", [1, 4, 5, 40, 600, 5000, 9000])
def test_embed_backward_of_one_id(M):
    """All tokens, or all but the ends, share an id: sums over many tiles."""
    say("embed bwd one id", M)
    ids = np.full(M, 2, np.int64)
    embed_case(M, 4, 530, BF16, F32, ids)
    ids[0], ids[-1] = 3, 0
    embed_case(M, 4, 530, F32, F32, ids, extra=0)
    ids[:] = -5
    embed_case(M, 4, 12, F32, BF16, ids)


def test_embed_backward_tiles_end_where_ids_do():
    """Runs of equal ids that end on, before and after the tiles' borders."""
    for M in (64, 2048, 4800):
        for run in (4, 15, 16, 17, 31, 32, 33, 64):
            say("embed bwd runs", M, run)
            ids = np.arange(M) // run
            embed_case(M, M // run + 1, 9, F32, F32, np.random.default_rng(run).permutation(ids))


def test_embed_backward_without_tokens():
    for dt in (F32, BF16):
        dW = q.qlora_embed_bwd(torch.empty(0, 33, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV),
                               7, grad_dtype=dt)
        assert dW.shape == (7, 33) and not dW.any()


@pytest.mark.parametrize("M", [9, 4500])
@pytest.mark.parametrize("V,D,dtype", [(1, 1, BF16), (7, 1, BF16), (8, 1, BF16), (3, 3, F32), (31, 1, BF16),
                                       (33, 1, F32), (1023, 9, BF16), (1025, 4, F32), (2049, 513, BF16)])
def test_embed_backward_fills_the_table(M, V, D, dtype):
    """Rows without a token become zero to the last element whatever part of
    the zeros each launch writes, and what lies behind the table stays."""
    say("embed bwd fill", M, V, D, dtype)
    ids = torch.full((M,), V - 1, dtype=torch.int64, device=DEV)
    ids[1:] = -1
    dY = torch.ones(M, D, device=DEV)
    whole = torch.full((V * D + 64,), math.nan, dtype=dtype, device=DEV)
    dW = whole[:V * D].view(V, D)
    q.qlora_embed_bwd(dY, ids, V, scale=3.0, dW=dW)
    torch.cuda.synchronize()
    assert not dW[:-1].any() and bool((dW[-1] == 3.0).all())
    assert bool(whole[V * D:].isnan().all())


# --------------------------------------------------------------- distillation
def distill_inputs(M, V, k, seed, z_dtype, t_dtype, ids_dtype):
    g = np.random.default_rng(seed)
    z = randn(g, (M, V), z_dtype, 2.5)
    t = randn(g, (M, k), t_dtype, 2.0, 3.0)
    ids = g.integers(0, V, (M, k))
    for m in range(M):
        if m % 3 == 0 and k <= V:
            ids[m] = g.permutation(V)[:k]   # distinct, as a top-k gives them
    if M > 1:
        ids[1] = -1                          # nothing live: the row is empty
        z[1] = math.nan
    if M > 2 and k > 1:
        ids[2, k // 2:] = V                  # padded entries
        t[2, 0] = -math.inf
    dl = g.standard_normal(M).astype(np.float32)
    if M > 4:
        dl[3] = 0.0
        z[4, V // 2] = -math.inf
        ids[4] = np.where(ids[4] == V // 2, -1, ids[4])
    return z, torch.from_numpy(ids).to(ids_dtype), t, torch.from_numpy(dl)


DISTILL = [(1, 1, 1), (1, 7, 3), (2, 8, 20), (5, 257, 16), (6, 2048, 64), (3, 8193, 100),
           (2, 70003, 300), (1, 200000, 1024), (9, 1000, 1), (1100, 300, 8)]


@pytest.mark.parametrize("i,shape", list(enumerate(DISTILL)))
@pytest.mark.parametrize("z_dtype", [BF16, F32])
def test_distill(i, shape, z_dtype):
    M, V, k = shape
    T = (1.0, 2.0, 0.7)[i % 3]
    t_dtype = F32 if i % 2 else BF16
    ids_dtype = torch.int64 if i % 4 < 2 else torch.int32
    g_dtype = z_dtype if i % 3 else (F32 if z_dtype == BF16 else BF16)
    say("distill", M, V, k, T, z_dtype, t_dtype, ids_dtype, g_dtype)
    z, ids, t, dl = distill_inputs(M, V, k, 70 + i, z_dtype, t_dtype, ids_dtype)
    zv, _ = strided(z, i % 3, lead=(i + 1) % 2)
    idd, td = ids.to(DEV), t.to(DEV)
    stats = torch.empty(2, M, device=DEV)
    loss = q.qlora_distill_fwd(zv, idd, td, temperature=T, stats_out=stats)
    gv, gbuf = strided(torch.zeros(M, V, dtype=g_dtype), (i + 1) % 3, lead=i % 2)
    q.qlora_distill_bwd(zv, idd, td, dl.to(DEV), stats, temperature=T, dlogits=gv)
    torch.cuda.synchronize()
    T64 = float(np.float32(T))
    want, err, wstats, e_stats = rows.distill_fwd(host(z), host(ids), host(t), T64)
    check(loss, want, err, "loss")
    check(stats, wstats, e_stats, "stats")
    wz, ez = rows.distill_bwd(host(z), host(ids), host(t), host(dl), T64)
    check(gv, wz, ez, "dlogits")
    assert int(torch.isnan(gbuf).sum()) == gbuf.numel() - M * V


def test_distill_of_masked_logits():
    """Vocabulary entries masked by -infinity or the type's lowest value, whole
    rows of the lowest value, and a live entry that the student has ruled out."""
    V, k = 300, 4
    for dt in (BF16, F32):
        low = torch.finfo(dt).min
        g = np.random.default_rng(5)
        z = randn(g, (6, V), dt)
        z[0, 100:] = -math.inf
        z[1, :200] = low
        z[2] = low                        # uniform
        z[3, 7] = -math.inf               # the teacher names it: loss +inf
        z[4] = 1e4 * z[4]
        z[5, 0] = 300.0
        ids = torch.tensor([[1, 2, 3, 4], [250, 260, 299, 200], [0, 9, 100, 299], [6, 7, 8, 9],
                            [0, 1, 2, 3], [5, 5, 0, 0]])
        t = randn(g, (6, k))
        say("distill masked", dt)
        for T in (1.0, 4.0, 0.5):
            stats = torch.empty(2, 6, device=DEV)
            args = (z.to(DEV), ids.to(DEV), t.to(DEV))
            loss = q.qlora_distill_fwd(*args, temperature=T, stats_out=stats)
            dz = q.qlora_distill_bwd(*args, torch.ones(6, device=DEV), stats, temperature=T,
                                     grad_dtype=F32)
            torch.cuda.synchronize()
            want, err, _, _ = rows.distill_fwd(host(z), host(ids), host(t), T)
            assert want[3] == np.inf
            check(loss, want, err, "loss")
            wz, ez = rows.distill_bwd(host(z), host(ids), host(t), np.ones(6), T)
            check(dz, wz, ez, "dlogits")


@pytest.mark.parametrize("size,T", [(30.0, 1.0), (1e5, 1.0), (1e5, 2.0 ** -20), (1e9, 0.01),
                                    (1e20, 1.0), (1e30, 2.0 ** 20)])
def test_distill_of_large_logits(size, T):
    """Logits whose quotients by the temperature are far beyond the range of an
    exponential, with their largest entries close together."""
    g = np.random.default_rng(21)
    M, V, k = 5, 3000, 6
    z = randn(g, (M, V), F32, size)
    top = z.max(dim=1, keepdim=True).values
    for j in range(4):   # near the largest: steps of about T
        z[:, 7 + j] = torch.nextafter(top[:, 0] - j * T, torch.tensor(0.0))
    ids = torch.tensor([[7, 8, 9, 10, 0, 2999]] * M)
    t = randn(g, (M, k), F32, T)
    stats = torch.empty(2, M, device=DEV)
    args = (z.to(DEV), ids.to(DEV), t.to(DEV))
    loss = q.qlora_distill_fwd(*args, temperature=T, stats_out=stats)
    dz = q.qlora_distill_bwd(*args, torch.ones(M, device=DEV), stats, temperature=T)
    torch.cuda.synchronize()
    want, err, wstats, e_stats = rows.distill_fwd(host(z), host(ids), host(t), T)
    check(loss, want, err, "loss")
    check(stats, wstats, e_stats, "stats")
    wz, ez = rows.distill_bwd(host(z), host(ids), host(t), np.ones(M), T)
    check(dz, wz, ez, "dlogits")


def test_distill_spreads_nan_by_row():
    z, t = torch.zeros(4, 50), torch.zeros(4, 3)
    ids = torch.tensor([[0, 1, 2]] * 4)
    z[0, 40] = math.nan
    t[1, 1] = math.nan
    z[2, 3] = math.inf
    stats = torch.empty(2, 4, device=DEV)
    args = (z.to(DEV), ids.to(DEV), t.to(DEV))
    loss = host(q.qlora_distill_fwd(*args, stats_out=stats))
    dz = host(q.qlora_distill_bwd(*args, torch.ones(4, device=DEV), stats))
    assert np.isnan(loss[:3]).all() and np.isfinite(loss[3])
    assert np.isnan(dz[0]).all() and np.isnan(dz[1, :3]).all() and np.isfinite(dz[3]).all()


def test_distill_gradient_by_differences():
    g = np.random.default_rng(9)
    M, V, k, T = 3, 200, 10, 2.0
    z, ids, t, _ = distill_inputs(M, V, k, 4, F32, F32, torch.int64)
    z[1] = randn(g, V)
    w, d = g.standard_normal(M).astype(np.float32), g.standard_normal((M, V))
    stats = torch.empty(2, M, device=DEV)
    args = (z.to(DEV), ids.to(DEV), t.to(DEV))
    q.qlora_distill_fwd(*args, temperature=T, stats_out=stats)
    dz = q.qlora_distill_bwd(*args, torch.from_numpy(w).to(DEV), stats, temperature=T)

    def f(v):
        return (rows.distill_fwd(v, host(ids), host(t), T)[0] * w).sum()
    h, z64 = 1e-5, host(z).astype(np.float64)
    want = (f(z64 + h * d) - f(z64 - h * d)) / (2 * h)
    wz, ez = rows.distill_bwd(host(z), host(ids), host(t), w, T)
    tol = ((ez + 2.0 ** -24 * np.abs(wz)) * np.abs(d)).sum() + 1e-6 * abs(want)
    assert abs((host(dz) * d).sum() - want) <= tol


# ------------------------------------------------------------ far addresses
def test_offsets_past_32_bits():
    """Rows that lie past 2^32 bytes and 2^31 elements in their buffers: a table
    of 4.9 GB and its gradient, and views of two rows 2^31 + 24 elements apart."""
    g = np.random.default_rng(12)
    V, D = 600_000, 4096
    say("far table")
    table = torch.empty(V, D, dtype=BF16, device=DEV)
    ids = torch.tensor([V - 1, 0, V - 2, V - 1, V], device=DEV)
    W = randn(g, (2, D), BF16)
    table[0], table[V - 2:] = W[0].to(DEV), W.to(DEV)
    out = q.qlora_embed_fwd(table, ids)
    assert torch.equal(out[0], W[1].to(DEV)) and torch.equal(out[1], W[0].to(DEV))
    assert torch.equal(out[2], W[0].to(DEV)) and not out[4].any()
    dY = randn(g, (5, D), BF16)
    dW = q.qlora_embed_bwd(dY.to(DEV), ids, V, dW=table)
    want, err = rows.embed_bwd(host(dY), np.array([2, 0, 1, 2, 3]), 3, 1.0)
    check(dW[[0, V - 2, V - 1]], want, err, "dW")
    assert not dW[1:V - 2].any()
    del table, dW
    say("far rows")
    ld = (1 << 31) + 24
    buf = torch.empty(ld + 4096, dtype=BF16, device=DEV)

    def far(t):
        v = buf.as_strided(t.shape, (ld, 1))
        v.copy_(t)
        return v
    x, dy = randn(g, (2, 1000), BF16), randn(g, (2, 1000), BF16)
    y = q.qlora_norm_fwd(far(x))
    want, err, _, _ = rows.norm_fwd(host(x), None, None, 1e-5, True)
    check(y, want, err, "y")
    dX, _, _ = q.qlora_norm_bwd(dy.to(DEV), far(x))
    (wX, eX), _, _ = rows.norm_bwd(host(dy), host(x), None, 1e-5, True)
    check(dX, wX, eX, "dX")
    top, t = torch.tensor([[3, 999], [0, 1]]), randn(g, (2, 2))
    stats = torch.empty(2, 2, device=DEV)
    loss = q.qlora_distill_fwd(far(x), top.to(DEV), t.to(DEV), stats_out=stats)
    want, err, _, _ = rows.distill_fwd(host(x), host(top), host(t), 1.0)
    check(loss, want, err, "loss")
    got = q.qlora_distill_bwd(x.to(DEV), top.to(DEV), t.to(DEV), torch.ones(2, device=DEV), stats,
                              dlogits=buf.as_strided((2, 1000), (ld, 1)))
    want, err = rows.distill_bwd(host(x), host(top), host(t), np.ones(2), 1.0)
    check(got, want, err, "dlogits")
    dW = q.qlora_embed_bwd(far(dy), torch.tensor([1, 1], device=DEV), 2)
    want, err = rows.embed_bwd(host(dy), np.array([1, 1]), 2, 1.0)
    check(dW, want, err, "dW")


def test_many_rows():
    """More rows than a launch has workgroups: every kernel's loop over rows."""
    M, g = 70001, np.random.default_rng(13)
    say("many rows")
    z, t = randn(g, (M, 24), BF16), randn(g, (M, 3))
    ids = torch.from_numpy(g.integers(-1, 24, (M, 3)))
    dl = torch.from_numpy(g.standard_normal(M).astype(np.float32))
    stats = torch.empty(2, M, device=DEV)
    args = (z.to(DEV), ids.to(DEV), t.to(DEV))
    loss = q.qlora_distill_fwd(*args, stats_out=stats)
    dz = q.qlora_distill_bwd(*args, dl.to(DEV), stats, grad_dtype=F32)
    want, err, _, _ = rows.distill_fwd(host(z), host(ids), host(t), 1.0)
    check(loss, want, err, "loss")
    want, err = rows.distill_bwd(host(z), host(ids), host(t), host(dl), 1.0)
    check(dz, want, err, "dlogits")
    W = randn(g, (50, 24), BF16)
    tok = torch.from_numpy(g.integers(-1, 51, M))
    out = q.qlora_embed_fwd(W.to(DEV), tok.to(DEV), out_dtype=F32)
    want, err = rows.embed_fwd(host(W), host(tok), 1.0)
    check(out, want, err, "out")
    dW = q.qlora_embed_bwd(z.to(DEV), tok.to(DEV), 50)
    want, err = rows.embed_bwd(host(z), host(tok), 50, 1.0)
    check(dW, want, err, "dW")
    # rows cut into more pieces than a launch has workgroups
    M, V = 9001, 70000
    z = torch.randn(M, V, device=DEV, dtype=BF16)
    ids, t = torch.randint(0, V, (M, 2), device=DEV), torch.randn(M, 2, device=DEV)
    stats = torch.empty(2, M, device=DEV)
    loss = q.qlora_distill_fwd(z, ids, t, stats_out=stats)
    dz = q.qlora_distill_bwd(z, ids, t, torch.ones(M, device=DEV), stats)
    for m in (0, 4500, 9000):
        r = slice(m, m + 1)
        want, err, _, _ = rows.distill_fwd(host(z[r]), host(ids[r]), host(t[r]), 1.0)
        check(loss[r], want, err, "loss")
        want, err = rows.distill_bwd(host(z[r]), host(ids[r]), host(t[r]), np.ones(1), 1.0)
        check(dz[r], want, err, "dlogits")


# ------------------------------------------------------------- a step of them
class Step:
    """Embedding, norm, a quantized linear layer with its adapter, a second one
    to the vocabulary, the distillation loss, and all gradients back to the
    table, as a training step runs them."""

    def __init__(self, M=40, V=520, D=256, k=12, seed=0):
        g = np.random.default_rng(seed)
        dev = lambda t: t.to(DEV)  # noqa: E731
        self.M, self.V, self.D, self.T = M, V, D, 2.0
        self.table = dev(randn(g, (V, D), BF16))
        self.ids = dev(torch.from_numpy(np.where(g.random(M) < 0.2, -1, g.integers(0, V, M))))
        self.gamma, self.beta = dev(randn(g, D, BF16, 0.2, 1.0)), dev(randn(g, D, BF16, 0.1))
        self.w1 = q.qlora_quantize_nf4_dq(dev(randn(g, (D, D), BF16, 0.06)))
        self.w2 = q.qlora_quantize_nf4_dq(dev(randn(g, (V, D), BF16, 0.06)))
        self.A1, self.B1 = dev(randn(g, (D, 16), BF16, 0.06)), dev(randn(g, (16, D), BF16, 0.05))
        self.A2, self.B2 = dev(randn(g, (D, 16), BF16, 0.06)), dev(randn(g, (16, V), BF16, 0.05))
        self.top_ids = dev(torch.from_numpy(g.integers(-1, V, (M, k))))
        self.top_ids[3] = -1
        self.top = dev(randn(g, (M, k), F32, 2.0))
        self.dloss = torch.full((M,), 1.0 / M, device=DEV)
        self.stats, self.lstats = torch.empty(2, M, device=DEV), torch.empty(2, M, device=DEV)

    def run(self):
        o = {}
        o["e"] = q.qlora_embed_fwd(self.table, self.ids, scale=2.0)
        o["h"] = q.qlora_norm_fwd(o["e"], self.gamma, self.beta, stats_out=self.stats)
        o["a"] = q.qlora_linear_fwd(self.w1, o["h"], self.A1, self.B1, 32.0, y_dtype=BF16)
        o["z"] = q.qlora_linear_fwd(self.w2, o["a"], self.A2, self.B2, 32.0, y_dtype=BF16)
        o["loss"] = q.qlora_distill_fwd(o["z"], self.top_ids, self.top, temperature=self.T,
                                        stats_out=self.lstats)
        o["dz"] = q.qlora_distill_bwd(o["z"], self.top_ids, self.top, self.dloss, self.lstats,
                                      temperature=self.T)
        o["da"], o["dA2"], o["dB2"] = q.qlora_linear_bwd(self.w2, o["a"], o["dz"], self.A2, self.B2,
                                                         32.0, dx_dtype=BF16)
        o["dh"], o["dA1"], o["dB1"] = q.qlora_linear_bwd(self.w1, o["h"], o["da"], self.A1, self.B1,
                                                         32.0)
        o["de"], o["dgamma"], o["dbeta"] = q.qlora_norm_bwd(o["dh"], o["e"], self.gamma,
                                                            stats=self.stats, dx_dtype=F32)
        o["dW"] = q.qlora_embed_bwd(o["de"], self.ids, self.V, scale=2.0)
        return o


def test_the_operators_together():
    """Every operator of a step against its 64-bit form on the values that the
    step gave it."""
    s = Step()
    o = s.run()
    torch.cuda.synchronize()
    ids = host(s.ids)
    want, err = rows.embed_fwd(host(s.table), ids, 2.0)
    check(o["e"], want, err, "embedding")
    want, err, _, _ = rows.norm_fwd(host(o["e"]), host(s.gamma), host(s.beta), 1e-5, True)
    check(o["h"], want, err, "norm")
    want, err, _, _ = rows.distill_fwd(host(o["z"]), host(s.top_ids), host(s.top), s.T)
    check(o["loss"], want, err, "loss")
    want, err = rows.distill_bwd(host(o["z"]), host(s.top_ids), host(s.top), host(s.dloss), s.T)
    check(o["dz"], want, err, "dlogits")
    (wX, eX), (wg, eg), (wb, eb) = rows.norm_bwd(host(o["dh"]), host(o["e"]), host(s.gamma), 1e-5, True)
    check(o["de"], wX, eX, "dX of the norm")
    check(o["dgamma"], wg, eg, "dgamma")
    check(o["dbeta"], wb, eb, "dbeta")
    want, err = rows.embed_bwd(host(o["de"]), ids, s.V, 2.0)
    check(o["dW"], want, err, "dW")
    # the table's step, as AdamW takes it
    p = s.table.float()
    m, v = torch.zeros_like(p), torch.zeros_like(p)
    q.qlora_adamw_step(p, o["dW"], m, v, 1, 1e-3)
    torch.cuda.synchronize()
    still = np.setdiff1d(np.arange(s.V), ids)
    assert torch.equal(p[still], s.table.float()[still]) and not torch.equal(p, s.table.float())


def test_a_captured_step_replays_with_the_same_bits():
    s = Step(M=33, V=1030, D=320, seed=3)
    want = {k: v.clone() for k, v in s.run().items()}
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        s.run()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = s.run()
    for replay in range(4):
        for t in o.values():
            t.fill_(-7.0)
        graph.replay()
        torch.cuda.synchronize()
        eager = s.run()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(o[k], want[k]) and torch.equal(eager[k], want[k]), (replay, k)


def test_two_streams_at_once():
    """Two independent steps on two streams, launched in turn without waits,
    and the stream argument in the place of the current stream."""
    a, b = Step(seed=1), Step(seed=2)
    wa = {k: v.clone() for k, v in a.run().items()}
    wb = {k: v.clone() for k, v in b.run().items()}
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(sa):
            oa = a.run()
        with torch.cuda.stream(sb):
            ob = b.run()
    torch.cuda.synchronize()
    for k in wa:
        assert torch.equal(oa[k], wa[k]) and torch.equal(ob[k], wb[k]), k
    e = q.qlora_embed_fwd(a.table, a.ids, scale=2.0, stream=sa)
    h = q.qlora_norm_fwd(e, a.gamma, a.beta, stream=sa)
    loss = q.qlora_distill_fwd(wa["z"], a.top_ids, a.top, temperature=2.0, stream=sb)
    dW = q.qlora_embed_bwd(wa["de"], a.ids, a.V, scale=2.0, stream=sb)
    torch.cuda.synchronize()
    assert torch.equal(h, wa["h"]) and torch.equal(loss, wa["loss"]) and torch.equal(dW, wa["dW"])


def test_a_short_workspace_is_refused():
    x = torch.zeros(4, 64, device=DEV)
    ids = torch.zeros(4, dtype=torch.int64, device=DEV)
    small = torch.empty(16, dtype=torch.uint8, device=DEV)
    for call in (lambda: q.qlora_norm_bwd(x, x, workspace=small),
                 lambda: q.qlora_embed_bwd(x, ids, 9, workspace=small),
                 lambda: q.qlora_distill_fwd(torch.zeros(1, 90000, device=DEV), ids[None], x[:1, :4].clone(),
                                             workspace=small)):
        with pytest.raises(RuntimeError):
            call()
    assert q.qlora_norm_bwd(x, x, want_dgamma=False, want_dbeta=False, workspace=small)[0].shape == (4, 64)
    assert _lib.load() is not None
