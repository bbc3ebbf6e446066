"""GPU tests of the vocabulary head's loss and its gradients against their
64-bit forms: |got - want| <= err + half a step of the output's type, where err
is the bound that oracle/close.py derives for the values at hand (the roundings
to bf16 that the products' operands take among them)."""
import math

import numpy as np
import pytest
import torch

import qlora_fine_tuning_blockwise_amd as q
from oracle import close
from test_row_ops_gpu import BF16, DEV, F32, check, host, randn, say, strided

pytestmark = pytest.mark.gpu

I32, I64 = torch.int32, torch.int64


def head_inputs(M, V, K, seed, dead=0.3, ids=I64, sigma=2.0):
    """Logits with a deviation of sigma, labels that the model favours, and a
    share of rows without a label (and with NaN for x), as a masked batch has."""
    g = np.random.default_rng(seed)
    W = randn(g, (V, K), BF16, sigma / math.sqrt(K))
    labels = g.integers(0, V, M)
    x = randn(g, (M, K)) + torch.from_numpy(g.uniform(0, 2, (M, 1)).astype(np.float32)) * W[labels].float()
    x = x.to(BF16)
    off = g.random(M) < dead
    if M > 1:
        off[0] = False
    else:
        off[:] = False
    labels = np.where(off, g.choice([-100, -1, V, 2 ** 31 - 1], M), labels)
    x[torch.from_numpy(off)] = math.nan
    dloss = (0.5 + g.random(M)).astype(np.float32) / M
    if M > 3:
        dloss[M // 2] = 0.0
    return x, W, torch.from_numpy(labels).to(ids), torch.from_numpy(dloss)


SHAPES = [(1, 1, 1), (1, 7, 3), (2, 255, 31), (3, 256, 32), (5, 257, 33), (17, 300, 64), (64, 511, 72),
          (65, 512, 96), (129, 1000, 128), (255, 513, 100), (256, 768, 160), (257, 511, 8), (300, 1500, 1027),
          (513, 777, 250), (700, 1030, 512)]


def forward(x, W, labels, scale, i):
    xv, xbuf = strided(x, (8 * (i % 3)) if i % 2 else i % 5, lead=i % 3)
    # In place (aligned rows) and copied (the others).
    Wv, wbuf = strided(W, (8 - W.shape[1] % 8) % 8 + 8 * (i % 2) if i % 3 else i % 5, lead=0 if i % 3 else i % 4)
    stats = torch.empty(2, x.shape[0], device=DEV)
    loss = q.qlora_head_loss_fwd(xv, Wv, labels.to(DEV), scale=scale, stats_out=stats)
    return xv, Wv, loss, stats


@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES)))
def test_head_loss_forward(i, shape):
    M, V, K = shape
    scale = (1.0, 0.5, -1.25)[i % 3]
    say("head fwd", M, V, K, scale)
    x, W, labels, _ = head_inputs(M, V, K, 200 + i, ids=(I32, I64)[i % 2])
    for k in range(4):
        _, _, loss, stats = forward(x, W, labels, scale, i + k)
        torch.cuda.synchronize()
        want, err, wstats, e_stats = close.head_loss_fwd(host(x), host(W), labels.numpy(), scale)
        check(loss, want, err, "loss")
        check(stats, wstats, e_stats, "stats")


@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES)))
@pytest.mark.parametrize("kind", [BF16, F32], ids=["bf16", "f32"])
def test_head_loss_backward(i, shape, kind):
    M, V, K = shape
    scale = (1.0, 0.5, -1.25)[i % 3]
    say("head bwd", M, V, K, kind)
    x, W, labels, dloss = head_inputs(M, V, K, 230 + i, ids=(I32, I64)[i % 2])
    xv, Wv, _, stats = forward(x, W, labels, scale, i)
    labels_d, dloss_d = labels.to(DEV), dloss.to(DEV)
    dXv, buf = strided(torch.zeros(M, K, dtype=kind), i % 3, lead=i % 2)
    dX, dW = q.qlora_head_loss_bwd(xv, Wv, labels_d, dloss_d, stats, scale=scale, dX=dXv, grad_dtype=kind)
    torch.cuda.synchronize()
    terms = 3 if kind == F32 else 1
    (wX, eX), (wW, eW) = close.head_loss_bwd(host(x), host(W), labels.numpy(), dloss.numpy(), scale, terms)
    check(dX, wX, eX, "dX")
    check(dW, wW, eW, "dW")
    assert int(torch.isnan(buf).sum()) == buf.numel() - M * K
    # each output alone has the same bits
    a, none = q.qlora_head_loss_bwd(xv, Wv, labels_d, dloss_d, stats, scale=scale, dx_dtype=kind, want_dw=False)
    assert none is None and torch.equal(a, dX)
    none, b = q.qlora_head_loss_bwd(xv, Wv, labels_d, dloss_d, stats, scale=scale, grad_dtype=kind, want_dx=False)
    assert none is None and torch.equal(b, dW)
    # added to what is there, with one rounding
    g = np.random.default_rng(i)
    old = randn(g, (V, K), kind, 0.01)
    acc = old.to(DEV)
    _, c = q.qlora_head_loss_bwd(xv, Wv, labels_d, dloss_d, stats, scale=scale, want_dx=False, dW=acc, accumulate=True)
    assert c is acc
    want = wW + host(old).astype(np.float64)
    check(acc, want, eW + 2.0 ** -24 * np.abs(want), "dW, accumulated")


@pytest.mark.parametrize("M,V,K", [(70, 70001, 40), (300, 33000, 72), (520, 40000, 64)])
def test_head_loss_in_pieces(M, V, K):
    """Vocabularies of several pieces. A row for each border of a tile and of a
    piece, whose label's neighbour there takes about half of the probability: one
    entry that is lost or counted twice cannot hide."""
    say("head pieces", M, V, K)
    x, W, labels, dloss = head_inputs(M, V, K, 7)
    at = sorted({p for w in (256, 512, 8192, 16384, 16640, 23552, 32768, 47104, V) for p in (w - 1, w, w + 1)
                 if p < V} | {0, 1, V - 2})
    scale = math.sqrt(K)
    W = (W * scale / 2).to(BF16)  # rows of a length near sqrt(K)
    for r, v in enumerate(at):
        x[r] = (W[v].float() * (14.0 / float((W[v].float() ** 2).sum()))).to(BF16)
        labels[r] = (v * 7 + 3) % V
    xv, Wv, loss, stats = forward(x, W, labels, 1.0, 1)
    want, err, wstats, e_stats = close.head_loss_fwd(host(x), host(W), labels.numpy())
    p_at = np.exp(host(x[:len(at)]).astype(np.float64) @ host(W).astype(np.float64).T)
    p_at = (p_at / p_at.sum(1, keepdims=True))[np.arange(len(at)), at]
    assert p_at.min() > 0.1
    check(loss, want, err, "loss")
    check(stats, wstats, e_stats, "stats")
    for kind in (BF16, F32):
        dX, dW = q.qlora_head_loss_bwd(xv, Wv, labels.to(DEV), dloss.to(DEV), stats, dx_dtype=kind, grad_dtype=kind)
        (wX, eX), (wW, eW) = close.head_loss_bwd(host(x), host(W), labels.numpy(), dloss.numpy(), 1.0,
                                                 3 if kind == F32 else 1)
        check(dX, wX, eX, "dX")
        check(dW, wW, eW, "dW")


@pytest.mark.parametrize("M", [1, 5, 40, 300])
def test_head_loss_of_rows_without_labels(M):
    x, W, _, _ = head_inputs(M, 600, 96, 3)
    x[:] = math.nan
    labels, dloss = torch.full((M,), -100), torch.ones(M)
    stats = torch.full((2, M), 5.0, device=DEV)
    args = x.to(DEV), W.to(DEV), labels.to(DEV)
    loss = q.qlora_head_loss_fwd(*args, stats_out=stats)
    assert not loss.any() and not stats.any()
    dX, dW = q.qlora_head_loss_bwd(*args, dloss.to(DEV), stats)
    assert dX.shape == (M, 96) and not dX.any() and dW.shape == (600, 96) and not dW.any()
    old = torch.full((600, 96), 2.0, device=DEV)
    q.qlora_head_loss_bwd(*args, dloss.to(DEV), stats, want_dx=False, dW=old, accumulate=True)
    assert bool((old == 2.0).all())


def test_head_loss_without_rows():
    x, W = torch.empty(0, 64, dtype=BF16, device=DEV), torch.zeros(30, 64, dtype=BF16, device=DEV)
    labels, none = torch.empty(0, dtype=I64, device=DEV), torch.empty(0, device=DEV)
    stats = torch.empty(2, 0, device=DEV)
    assert q.qlora_head_loss_fwd(x, W, labels, stats_out=stats).shape == (0,)
    dX, dW = q.qlora_head_loss_bwd(x, W, labels, none, stats, grad_dtype=F32)
    assert dX.shape == (0, 64) and not dW.any()
    old = torch.ones(30, 64, dtype=BF16, device=DEV)
    q.qlora_head_loss_bwd(x, W, labels, none, stats, dW=old, accumulate=True)
    assert bool((old == 1).all())


@pytest.mark.parametrize("M", [3, 270])
def test_head_loss_of_large_logits(M):
    """Logits in the hundreds, of which one stands far above the others, or none
    does; and NaN and infinity in a row of x, which stay in that row."""
    g = np.random.default_rng(4)
    V, K = 700, 64
    W = randn(g, (V, K), BF16)
    x = randn(g, (M, K), BF16, 30.0)
    x[1] = 0  # an even distribution
    labels = torch.from_numpy(g.integers(0, V, M))
    labels[0] = int((x[0].float() @ W.float().t()).argmax())
    dloss = torch.ones(M)
    stats = torch.empty(2, M, device=DEV)
    loss = q.qlora_head_loss_fwd(x.to(DEV), W.to(DEV), labels.to(DEV), stats_out=stats)
    want, err, wstats, e_stats = close.head_loss_fwd(host(x), host(W), labels.numpy())
    check(loss, want, err, "loss")
    check(stats, wstats, e_stats, "stats")
    dX, dW = q.qlora_head_loss_bwd(x.to(DEV), W.to(DEV), labels.to(DEV), dloss.to(DEV), stats, dx_dtype=F32,
                                   grad_dtype=F32)
    (wX, eX), (wW, eW) = close.head_loss_bwd(host(x), host(W), labels.numpy(), dloss.numpy(), 1.0, 3)
    check(dX, wX, eX, "dX")
    check(dW, wW, eW, "dW")
    bad = x.clone()
    bad[2, 5] = math.nan
    bad[0, 9] = math.inf
    got = q.qlora_head_loss_fwd(bad.to(DEV), W.to(DEV), labels.to(DEV), stats_out=stats)
    assert torch.isnan(got[2]) and not torch.isfinite(got[0])
    assert torch.equal(got[1], loss[1]) and torch.equal(got[3:], loss[3:])


def test_head_loss_gradient_by_differences():
    """Central differences of the loss along random directions, in inputs that
    are bf16 before and after the step (multiples of 2^-6 below 2). The
    difference's own error is of the third derivative, 2^-12 of terms of the
    derivative's size, and of the forward's roundings, 2^-20 over the step 2^-6:
    all below 2e-3 of the sum of the terms' sizes."""
    g = np.random.default_rng(11)
    M, V, K, step = 20, 300, 64, 2.0 ** -6
    grid = lambda shape: torch.from_numpy(g.integers(-32, 33, shape).astype(np.float32)) * step  # noqa: E731
    x, W = grid((M, K)), grid((V, K))
    labels, dloss = torch.from_numpy(g.integers(0, V, M)).to(DEV), randn(g, M).to(DEV)
    stats = torch.empty(2, M, device=DEV)

    def f(x_, W_):
        loss = q.qlora_head_loss_fwd(x_.to(BF16).to(DEV), W_.to(BF16).to(DEV), labels)
        return float((loss.double() * dloss.double()).sum())
    q.qlora_head_loss_fwd(x.to(BF16).to(DEV), W.to(BF16).to(DEV), labels, stats_out=stats)
    dX, dW = q.qlora_head_loss_bwd(x.to(BF16).to(DEV), W.to(BF16).to(DEV), labels, dloss, stats, dx_dtype=F32,
                                   grad_dtype=F32)
    for grad, other in ((dX.cpu().double(), False), (dW.cpu().double(), True)):
        d = torch.from_numpy(g.integers(-1, 2, tuple(grad.shape)).astype(np.float32))
        pair = [(x, W + s * step * d) if other else (x + s * step * d, W) for s in (1, -1)]
        want = (f(*pair[0]) - f(*pair[1])) / (2 * step)
        size = float((grad * d).abs().sum())
        assert abs(float((grad * d).sum()) - want) <= 2e-3 * size


def test_head_loss_repeats_its_bits():
    x, W, labels, dloss = (t.to(DEV) for t in head_inputs(600, 3001, 320, 12))
    stats = [torch.empty(2, 600, device=DEV) for _ in range(2)]
    losses = [q.qlora_head_loss_fwd(x, W, labels, stats_out=s) for s in stats]
    assert torch.equal(*losses) and torch.equal(*stats)
    (a, b), (c, d) = (q.qlora_head_loss_bwd(x, W, labels, dloss, stats[0]) for _ in range(2))
    assert torch.equal(a, c) and torch.equal(b, d)


def test_head_loss_refused():
    x, W, labels, dloss = (t.to(DEV) for t in head_inputs(8, 300, 64, 1))
    stats = torch.empty(2, 8, device=DEV)
    small = torch.empty(256, dtype=torch.uint8, device=DEV)
    with pytest.raises(RuntimeError):
        q.qlora_head_loss_fwd(x, W, labels, workspace=small)
    with pytest.raises(RuntimeError):
        q.qlora_head_loss_bwd(x, W, labels, dloss, stats, workspace=small)
    with pytest.raises(RuntimeError):
        q.qlora_head_loss_bwd(x, W, labels, dloss, stats, dX=x)
    with pytest.raises(RuntimeError):
        q.qlora_head_loss_bwd(x, W, labels, dloss, stats, dW=W)
    with pytest.raises(RuntimeError):
        q.qlora_head_loss_fwd(x, W, labels, scale=math.inf)
    with pytest.raises(ValueError):
        q.qlora_head_loss_fwd(x.float(), W, labels)


@pytest.mark.parametrize("M,V,K", [(1, 1, 8), (1, 17, 16), (2, 4095, 72), (8, 4097, 1016), (9, 5000, 1024),
                                   (16, 300, 1032), (3, 8193, 2048), (16, 4100, 2056), (7, 4111, 4088),
                                   (8, 9000, 4096), (15, 4113, 4096), (16, 64, 4104), (17, 4100, 1024)])
@pytest.mark.parametrize("kind", [BF16, F32], ids=["bf16", "f32"])
def test_head_loss_gradient_of_few_rows(M, V, K, kind):
    """Around the borders of the pass that reads W once: 16 rows, 16 entries a
    workgroup and 256 workgroups, slices of 1024, 2048 and 4096 columns. A row for
    each border of the vocabulary's entries whose probability stands there."""
    say("head few bwd", M, V, K, kind)
    x, W, labels, dloss = head_inputs(M, V, K, 400 + M, ids=I32)
    W = (W * math.sqrt(K) / 2).to(BF16)
    at = [v for v in (V - 1, 0, 15, 16, 4095, 4096, V - 2) if 0 <= v < V]
    for r, v in enumerate(at[:M]):
        x[r] = (W[v].float() * (14.0 / float((W[v].float() ** 2).sum()))).to(BF16)
        labels[r] = (v * 7 + 3) % V
    for odd in (False, True):
        xv, xbuf = strided(x, 5 if odd else 8, lead=int(odd))
        Wv, wbuf = strided(W, 3 if odd else 8, lead=int(odd))
        stats = torch.empty(2, M, device=DEV)
        q.qlora_head_loss_fwd(xv, Wv, labels.to(DEV), scale=0.75, stats_out=stats)
        dXv, buf = strided(torch.zeros(M, K, dtype=kind), 1 + 2 * odd, lead=int(odd))
        dX, none = q.qlora_head_loss_bwd(xv, Wv, labels.to(DEV), dloss.to(DEV), stats, scale=0.75, dX=dXv,
                                         want_dw=False)
        torch.cuda.synchronize()
        (want, err), _ = close.head_loss_bwd(host(x), host(W), labels.numpy(), dloss.numpy(), 0.75,
                                             3 if kind == F32 else 1)
        check(dX, want, err, "dX")
        assert none is None and int(torch.isnan(buf).sum()) == buf.numel() - M * K
        again, _ = q.qlora_head_loss_bwd(xv, Wv, labels.to(DEV), dloss.to(DEV), stats, scale=0.75, dx_dtype=kind,
                                         want_dw=False)
        assert torch.equal(again, dX)


@pytest.mark.parametrize("M,V,K", [(8, 40000, 64), (16, 33000, 72), (40, 40001, 24)])
def test_head_loss_both_gradients_of_few_rows(M, V, K):
    """The gradient of W in pieces beside the rows' in one pass, from a W that the
    tiles would copy."""
    say("head few both", M, V, K)
    x, W, labels, dloss = head_inputs(M, V, K, 450 + M)
    Wv, wbuf = strided(W, 3, lead=1)
    stats = torch.empty(2, M, device=DEV)
    q.qlora_head_loss_fwd(x.to(DEV), Wv, labels.to(DEV), stats_out=stats)
    for kind in (BF16, F32):
        dX, dW = q.qlora_head_loss_bwd(x.to(DEV), Wv, labels.to(DEV), dloss.to(DEV), stats, dx_dtype=kind,
                                       grad_dtype=kind)
        (wX, eX), (wW, eW) = close.head_loss_bwd(host(x), host(W), labels.numpy(), dloss.numpy(), 1.0,
                                                 3 if kind == F32 else 1)
        check(dX, wX, eX, "dX")
        check(dW, wW, eW, "dW")
        alone, _ = q.qlora_head_loss_bwd(x.to(DEV), Wv, labels.to(DEV), dloss.to(DEV), stats, dx_dtype=kind,
                                         want_dw=False)
        assert torch.equal(alone, dX)


@pytest.mark.parametrize("rows", [1, 31, 32, 33, 63, 64, 65, 96, 97, 127, 128, 129, 161, 255])
def test_head_loss_of_a_last_tile(rows):
    """Every count of groups of 32 live rows that a last tile can have."""
    M, V, K = 256 + rows, 260, 64
    say("head last tile", M, V, K)
    x, W, labels, dloss = head_inputs(M, V, K, 480 + rows, dead=0.0)
    dloss[:] = 1.0 / M
    stats = torch.empty(2, M, device=DEV)
    args = x.to(DEV), W.to(DEV), labels.to(DEV)
    loss = q.qlora_head_loss_fwd(*args, stats_out=stats)
    want, err, wstats, e_stats = close.head_loss_fwd(host(x), host(W), labels.numpy())
    check(loss, want, err, "loss")
    check(stats, wstats, e_stats, "stats")
    for kind in (BF16, F32):
        dX, dW = q.qlora_head_loss_bwd(*args, dloss.to(DEV), stats, dx_dtype=kind, grad_dtype=kind)
        (wX, eX), (wW, eW) = close.head_loss_bwd(host(x), host(W), labels.numpy(), dloss.numpy(), 1.0,
                                                 3 if kind == F32 else 1)
        check(dX, wX, eX, "dX")
        check(dW, wW, eW, "dW")
