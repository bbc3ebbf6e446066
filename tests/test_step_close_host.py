"""CPU tests of the operators that close a training step (the norm behind a
residual addition, the loss of the vocabulary head, the clipping of gradients):
the 64-bit gradients against central differences of the 64-bit forwards, the
host's checks of every argument, outputs over inputs, and the table of a
program's tensors. No kernel runs here."""
import ctypes
import os

import numpy as np
import pytest
import torch

import qlora_fine_tuning_blockwise_amd as q
from oracle import close
from qlora_fine_tuning_blockwise_amd import _lib

A = 1 << 30        # stand-in addresses, 64 MB apart; no accepted call is given them
FAR = 1 << 26
INVALID, SHAPE, ALIGN, DTYPE, WORKSPACE = 1, 2, 3, 4, 6


def _p(i, off=0):
    return ctypes.c_void_p(A + i * FAR + off)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from qlora_fine_tuning_blockwise_amd import build
        build.build()
    return _lib.load()


@pytest.fixture(scope="module")
def cpu(lib):
    if torch.cuda.is_available():
        pytest.skip("stand-in addresses: only where no kernel could run with them")
    return lib


def _with(f, base):
    def call(**kw):
        a = list(base)
        for j, w in kw.items():
            a[int(j[1:])] = w
        return f(*a)
    return call


# ---------------------------------------------------- gradients by differences
def _along(f, x, d, h=1e-5):
    """Central difference of f along d: its error is O(h^2) of the third
    derivative plus 2^-53 |f| / h, both below 1e-8 of the values here."""
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


def test_head_loss_gradients_are_the_forwards():
    g = np.random.default_rng(1)
    M, V, K, scale = 7, 19, 11, 0.7
    x, W = g.standard_normal((M, K)), g.standard_normal((V, K))
    labels = np.array([3, 0, 18, -1, 19, 3, 1 << 40])
    w = g.standard_normal(M)
    w[5] = 0.0
    (dX, _), (dW, _) = close.head_loss_bwd(x, W, labels, w, scale)

    def f(x_, W_):
        return (close.head_loss_fwd(x_, W_, labels, scale)[0] * w).sum()
    dx, dw = g.standard_normal((M, K)), g.standard_normal((V, K))
    for got, want in (((dX * dx).sum(), _along(lambda v: f(v, W), x, dx)),
                      ((dW * dw).sum(), _along(lambda v: f(x, v), W, dw))):
        assert abs(got - want) <= 1e-7 * max(1.0, abs(want))
    assert not dX[3].any() and not dX[4].any() and not dX[5].any() and not dX[6].any()
    loss = close.head_loss_fwd(x, W, labels, scale)[0]
    assert np.all(loss[[0, 1, 2, 5]] > 0) and not loss[[3, 4, 6]].any()


@pytest.mark.parametrize("center", [True, False])
def test_add_norm_gradients_are_the_forwards(center):
    g = np.random.default_rng(2)
    M, N, eps = 4, 15, 1e-5
    h, dY, dH = (g.standard_normal((M, N)) for _ in range(3))
    gamma = g.standard_normal(N)
    (dX, _), (dg, _), _ = close.add_norm_bwd(dY, dH, h, gamma, eps, center)

    def f(h_, g_):
        return (close.add_norm_fwd(h_, g_, None, eps, center)[0] * dY).sum() + (h_ * dH).sum()
    d, dn = g.standard_normal((M, N)), g.standard_normal(N)
    for got, want in (((dX * d).sum(), _along(lambda v: f(v, gamma), h, d)),
                      ((dg * dn).sum(), _along(lambda v: f(h, v), gamma, dn))):
        assert abs(got - want) <= 1e-7 * max(1.0, abs(want))


def test_a_lost_term_exceeds_the_bound():
    """What the GPU's losses and gradients are held to is narrow enough that an
    entry of the vocabulary which has its even share of the probability or more
    does not pass when it is left out or counted twice, nor a row of dW's sums."""
    g = np.random.default_rng(3)
    M, V, K = 40, 700, 64
    W = g.standard_normal((V, K)) * 2 / np.sqrt(K)
    x = g.standard_normal((M, K))
    labels = g.integers(0, V, M)
    loss, err, _, _ = close.head_loss_fwd(x, W, labels)
    z = x @ W.T
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    (dX, eX), (dW, eW) = close.head_loss_bwd(x, W, labels, np.ones(M), terms=3)
    rows, entries = np.nonzero(p > 1 / V)
    assert rows.size > M * V // 10
    assert (np.abs(np.log1p(-p[rows, entries])) > err[rows]).all()     # the loss without it
    lost = np.abs(p[rows, entries][:, None] * W[entries])
    assert (lost > eX[rows]).any(1).all()
    lost = np.abs(p[rows, entries][:, None] * x[rows])                 # dW without the row
    assert (lost > eW[entries]).any(1).all()


# ------------------------------------------------------------------- refusals
def test_add_norm_validation(lib):
    #       x      ldx t  res    ldr t  M  N   norm gamma  beta   wt eps   h      ldh y      ldy t  sc    stats
    base = [_p(0), 64, 1, _p(1), 64, 0, 4, 64, 0, _p(2), _p(3), 1, 1e-5, _p(4), 64, _p(5), 64, 1, None, None,
            None]
    call = _with(lib.qlora_add_norm_fwd, base)
    assert call(a6=-1) == INVALID and call(a8=2) == INVALID
    for bad in (-1e-6, float("nan"), float("inf")):
        assert call(a12=bad) == INVALID
    assert call(a0=None) == INVALID and call(a15=None) == INVALID
    assert call(a3=None) == INVALID and call(a13=None) == INVALID   # one of the two alone
    assert call(a17=4) == INVALID and call(a18=_p(6)) == INVALID    # codes and scales go together
    assert call(a7=0) == SHAPE and call(a7=16385, a1=20000, a4=20000, a14=20000, a16=20000) == SHAPE
    for i in (1, 4, 14, 16):
        assert call(**{f"a{i}": 63}) == SHAPE
    assert call(a6=1 << 25) == SHAPE and call(a1=1 << 62) == SHAPE
    assert call(a2=4) == DTYPE and call(a5=4) == DTYPE and call(a11=2) == DTYPE and call(a17=5) == DTYPE
    assert call(a0=_p(0, 1)) == ALIGN and call(a3=_p(1, 2)) == ALIGN and call(a13=_p(4, 2)) == ALIGN
    assert call(a15=_p(5, 1)) == ALIGN and call(a19=_p(6, 2)) == ALIGN
    assert call(a17=4, a18=_p(6, 2)) == ALIGN
    assert call(a6=0) == 0 and call(a6=0, a0=None, a3=None, a13=None, a15=None) == 0


def test_add_norm_bwd_validation(lib):
    #       dY     ld  t  dH     ld  h      ld  t  M  N   norm gamma wt eps  stats dX     ld  t  dg     db
    base = [_p(0), 64, 1, _p(1), 64, _p(2), 64, 1, 4, 64, 0, _p(3), 1, 1e-5, None, _p(4), 64, 0, _p(5), _p(6),
            0, _p(7), 1 << 24, None]
    call = _with(lib.qlora_add_norm_bwd, base)
    assert call(a8=-1) == INVALID and call(a10=7) == INVALID and call(a13=-1.0) == INVALID
    assert call(a0=None) == INVALID and call(a5=None) == INVALID
    for i in (1, 4, 6, 16):
        assert call(**{f"a{i}": 8}) == SHAPE
    assert call(a2=2) == DTYPE and call(a7=4) == DTYPE and call(a12=4) == DTYPE and call(a17=4) == DTYPE \
        and call(a20=2) == DTYPE
    assert call(a3=_p(1, 2)) == ALIGN and call(a18=_p(5, 2)) == ALIGN and call(a21=_p(7, 4)) == ALIGN
    need = q.qlora_norm_bwd_workspace_bytes(4, 64)
    assert call(a22=need - 1) == WORKSPACE and call(a21=None) == WORKSPACE
    assert call(a8=0, a18=None, a19=None) == 0
    # without dH, or without dX, the norm's own checks
    assert call(a3=None, a10=7) == INVALID and call(a15=None, a18=None, a19=None) == 0


def test_head_loss_validation(lib):
    #       x      ldx W      ldw M    V    K   labels it scale loss   stats ws     bytes
    base = [_p(0), 64, _p(1), 64, 100, 300, 64, _p(2), 3, 1.0, _p(3), None, _p(4), 1 << 24, None]
    call = _with(lib.qlora_head_loss_fwd, base)
    assert call(a4=-1) == INVALID
    for bad in (float("nan"), float("inf")):
        assert call(a9=bad) == INVALID
    for i in (0, 2, 7, 10):
        assert call(**{f"a{i}": None}) == INVALID
    assert call(a5=0) == SHAPE and call(a5=(1 << 31) - 1) == SHAPE and call(a6=0) == SHAPE
    assert call(a6=65537, a1=1 << 17, a3=1 << 17) == SHAPE
    assert call(a5=1 << 30, a6=1 << 11, a1=1 << 11, a3=1 << 11) == SHAPE   # V * K past 2^40
    assert call(a1=63) == SHAPE and call(a3=63) == SHAPE and call(a4=(1 << 20) + 1) == SHAPE
    assert call(a3=1 << 62) == SHAPE
    assert call(a8=0) == DTYPE
    assert call(a0=_p(0, 1)) == ALIGN and call(a2=_p(1, 1)) == ALIGN and call(a7=_p(2, 4)) == ALIGN \
        and call(a10=_p(3, 2)) == ALIGN and call(a11=_p(5, 2)) == ALIGN and call(a12=_p(4, 8)) == ALIGN
    need = q.qlora_head_loss_fwd_workspace_bytes(100, 300, 64)
    copied = q.qlora_head_loss_fwd_workspace_bytes(100, 300, 64, True)
    assert 0 < need < copied
    assert call(a13=need - 1) == WORKSPACE and call(a12=None) == WORKSPACE
    assert call(a2=_p(1, 2), a13=copied - 1) == WORKSPACE and call(a3=65, a13=copied - 1) == WORKSPACE
    assert call(a3=(1 << 20) + 8, a13=copied - 1) == WORKSPACE
    assert call(a4=0) == 0 and call(a4=0, a0=None, a2=None, a7=None, a10=None, a12=None) == 0
    for bad in ((-1, 300, 64), (8, 0, 64), (8, 300, 0), (8, 300, 65537), ((1 << 20) + 1, 300, 64)):
        assert q.qlora_head_loss_fwd_workspace_bytes(*bad) == 0
        assert q.qlora_head_loss_bwd_workspace_bytes(*bad) == 0
    assert q.qlora_head_loss_fwd_workspace_bytes(0, 300, 64) == 0


def test_head_loss_bwd_validation(lib):
    #       x      ldx W      ldw M    V    K   labels it scale stats  dloss  dX     ld  t  dW     t  acc
    base = [_p(0), 64, _p(1), 64, 100, 300, 64, _p(2), 3, 1.0, _p(3), _p(4), _p(5), 64, 1, _p(6), 1, 0,
            _p(7), 1 << 25, None]
    call = _with(lib.qlora_head_loss_bwd, base)
    assert call(a4=-1) == INVALID and call(a9=float("nan")) == INVALID
    for i in (0, 2, 7, 10, 11):
        assert call(**{f"a{i}": None}) == INVALID
    assert call(a13=63) == SHAPE and call(a1=63) == SHAPE and call(a5=0) == SHAPE
    assert call(a14=4) == DTYPE and call(a16=2) == DTYPE and call(a8=1) == DTYPE
    assert call(a10=_p(3, 2)) == ALIGN and call(a12=_p(5, 1)) == ALIGN and call(a15=_p(6, 8)) == ALIGN \
        and call(a18=_p(7, 8)) == ALIGN
    bf, f32 = torch.bfloat16, torch.float32
    sizes = [q.qlora_head_loss_bwd_workspace_bytes(100, 300, 64, False, *t)
             for t in ((bf, None), (f32, None), (None, bf), (None, f32), (bf, bf))]
    assert all(s > 0 for s in sizes) and sizes[0] < sizes[1] and sizes[2] < sizes[3] and sizes[4] > sizes[0]
    assert call(a19=sizes[4] - 1) == WORKSPACE and call(a18=None) == WORKSPACE
    assert call(a15=None, a19=sizes[0] - 1) == WORKSPACE
    assert call(a12=None, a15=None, a14=9, a16=9) == 0         # nothing asked for
    assert call(a4=0, a15=None) == 0 and call(a4=0, a17=1) == 0


def test_head_loss_workspace_stays_small():
    """A training batch's logits are never held: the workspace of the backward is
    a piece of them, and that of the forward 8 bytes for 256."""
    logits = 2048 * 128000 * 2
    assert q.qlora_head_loss_fwd_workspace_bytes(2048, 128000, 4096) < logits // 12
    acc = 512 * 256 * 256 * 4
    assert q.qlora_head_loss_bwd_workspace_bytes(2048, 128000, 4096) < logits // 3 + acc
    # long batches: at most 2048 entries of the vocabulary at once
    assert q.qlora_head_loss_bwd_workspace_bytes(1 << 20, 128000, 4096) < (1 << 20) * (2048 + 3 * 4096) * 2 + (1 << 30)


def _tensors(items):
    a = (_lib.Tensor * max(1, len(items)))()
    for t, (data, n, dtype, *rest) in zip(a, items):
        t.data, t.n, t.dtype, t.reserved = data, n, dtype, rest[0] if rest else 0
    return a


def test_grad_norm_validation(lib):
    good = _tensors([(A, 100, 1), (A + FAR, 7, 0), (None, 0, 1)])

    def norm(t=good, count=3, table=None, most=1.0, result=_p(5), ws=_p(6), size=1 << 20):
        return lib.qlora_grad_norm(t, count, table, most, result, ws, size, None)
    assert norm(count=-1) == INVALID and norm(t=None) == INVALID and norm(result=None) == INVALID
    assert norm(most=-1.0) == INVALID and norm(most=float("nan")) == INVALID
    assert norm(t=_tensors([(A, -1, 1)]), count=1) == INVALID
    assert norm(t=_tensors([(A, 4, 1, 1)]), count=1) == INVALID
    assert norm(t=_tensors([(None, 4, 1)]), count=1) == INVALID
    assert norm(count=(1 << 20) + 1) == SHAPE
    assert norm(t=_tensors([(A, 1 << 40, 1), (A, 1, 1)]), count=2) == SHAPE
    assert norm(t=_tensors([(A, 4, 2)]), count=1) == DTYPE
    assert norm(t=_tensors([(A + 1, 4, 1)]), count=1) == ALIGN
    assert norm(t=_tensors([(A + 2, 4, 0)]), count=1) == ALIGN
    assert norm(result=_p(5, 2)) == ALIGN and norm(ws=_p(6, 8)) == ALIGN and norm(table=_p(7, 8)) == ALIGN
    need = lib.qlora_grad_norm_workspace_bytes(good, 3)
    assert need > 0 and norm(size=need - 1) == WORKSPACE and norm(ws=None) == WORKSPACE
    assert norm(result=ctypes.c_void_p(A + 196)) == INVALID        # over the last elements
    assert norm(ws=ctypes.c_void_p(A + FAR + 16)) == INVALID and norm(result=_p(6)) == INVALID
    assert norm(table=_p(5)) == INVALID and norm(table=_p(6)) == INVALID
    assert lib.qlora_grad_norm_workspace_bytes(_tensors([(None, 0, 0)]), 1) == 0
    assert lib.qlora_grad_norm_workspace_bytes(None, 0) == 0
    assert lib.qlora_grad_norm_workspace_bytes(_tensors([(A, -1, 0)]), 1) == 0


def test_grad_scale_validation(lib):
    g = _tensors([(A, 100, 1), (A + FAR, 7, 0)])

    def scale(grads=g, out=None, count=2, table=None, out_table=None, factor=_p(5)):
        return lib.qlora_grad_scale(grads, out, count, table, out_table, factor, None)
    assert scale(grads=None) == INVALID and scale(factor=None) == INVALID and scale(count=-1) == INVALID
    assert scale(factor=_p(5, 1)) == ALIGN and scale(table=_p(7, 4)) == ALIGN
    assert scale(out=_tensors([(A, 100, 1), (A + FAR, 8, 0)])) == SHAPE
    assert scale(out=_tensors([(A, 100, 1), (A + FAR, 7, 1)])) == DTYPE
    assert scale(out=_tensors([(A, 100, 1), (None, 7, 0)])) == INVALID
    # shared memory: the same tensor twice, in place
    assert scale(grads=_tensors([(A, 100, 1), (A, 100, 1)])) == INVALID
    assert scale(grads=_tensors([(A, 100, 1), (A + 198, 10, 1)])) == INVALID
    # an output over another input, over another output, over the factor and tables
    assert scale(out=_tensors([(A + 2 * FAR, 100, 1), (A, 7, 0)])) == INVALID
    assert scale(out=_tensors([(A + 2 * FAR, 100, 1), (A + 2 * FAR + 196, 7, 0)])) == INVALID
    assert scale(out=_tensors([(A + 2, 100, 1), (A + FAR, 7, 0)])) == INVALID   # one element on
    assert scale(factor=ctypes.c_void_p(A + 8)) == INVALID
    assert scale(table=ctypes.c_void_p(A + 16), out_table=_p(7)) == INVALID
    assert scale(count=0) == 0 and scale(grads=_tensors([(None, 0, 1)]), count=1) == 0


def test_grad_scale_finds_shared_memory_in_any_order(cpu):
    """Random lists of runs: the call is refused exactly where an output meets
    another output or another input (an accepted call ends at its launch, which
    has no device here)."""
    g = np.random.default_rng(5)
    for trial in range(300):
        k = int(g.integers(1, 7))
        n = g.integers(1, 30, k)
        at = [int(v) * 4 for v in g.integers(0, 150, k)]
        to = [a if g.random() < 0.3 else int(g.integers(0, 300)) * 4 for a in at]
        runs = lambda p: [(a, a + 4 * int(m)) for a, m in zip(p, n)]  # noqa: E731
        meet = lambda a, b: a[0] < b[1] and b[0] < a[1]  # noqa: E731
        w, r = runs(to), runs(at)
        shared = any(meet(w[i], w[j]) for i in range(k) for j in range(i)) or \
            any(meet(w[i], r[j]) for i in range(k) for j in range(k) if at[j] != to[j])
        st = cpu.qlora_grad_scale(_tensors([(A + a, int(m), 0) for a, m in zip(at, n)]),
                                  _tensors([(A + a, int(m), 0) for a, m in zip(to, n)]), k, None, None, _p(5),
                                  None)
        assert (st == INVALID) == shared, (trial, at, to, n)


def test_tensor_table_holds_every_element_once(lib):
    for items in ([(A, 1, 1)], [(A + 2, 40000, 1), (None, 0, 0), (A + FAR, 8193, 0), (A + 2 * FAR, 3, 0)],
                  [(A, 200 << 20, 0), (1 << 40, 77, 1)]):   # 800 MB: larger pieces
        t = _tensors(items)
        need = lib.qlora_tensor_table_bytes(t, len(items))
        buf = np.zeros(need // 8, np.uint64)
        assert buf.ctypes.data % 16 == 0
        assert lib.qlora_tensor_table(t, len(items), buf.ctypes.data_as(ctypes.c_void_p), need) == 0
        assert need // 16 * 8 <= lib.qlora_grad_norm_workspace_bytes(t, len(items))
        assert need // 16 <= 16384 + len(items)
        rows = iter(buf.reshape(-1, 2))
        for data, n, dtype in items:
            at, end = data or 0, (data or 0) + n * (2 if dtype else 4)
            while at < end:
                p, word = (int(v) for v in next(rows))
                assert p == at and word >> 32 == dtype and word & 0xFFFFFFFF > 0
                at += (word & 0xFFFFFFFF) * (2 if dtype else 4)
            assert at == end
        assert next(rows, None) is None
    t = _tensors([(A, 100, 1)])
    room = np.zeros(64, np.uint64)
    p = room.ctypes.data
    assert lib.qlora_tensor_table(t, 1, None, 16) == INVALID and lib.qlora_tensor_table(t, 1, p + 8, 64) == ALIGN
    assert lib.qlora_tensor_table(t, 1, p, 15) == WORKSPACE and lib.qlora_tensor_table(t, -1, p, 64) == INVALID
    assert lib.qlora_tensor_table(None, 0, None, 0) == 0 and lib.qlora_tensor_table_bytes(None, 0) == 0


def test_adamw_scaled_validation(lib):
    #       p      g     t  factor m      v      pb    n  lr    b1   b2     eps   wd   step
    base = [_p(0), _p(1), 0, _p(2), _p(3), _p(4), None, 8, 1e-3, 0.9, 0.999, 1e-8, 0.0, 1, None]
    call = _with(lib.qlora_adamw_step_scaled, base)
    assert call(a7=-1) == INVALID and call(a13=0) == INVALID and call(a9=1.0) == INVALID
    assert call(a8=float("inf")) == INVALID and call(a2=2) == DTYPE
    for i in (0, 1, 3, 4, 5):
        assert call(**{f"a{i}": None}) == INVALID
    assert call(a3=_p(2, 2)) == ALIGN and call(a0=_p(0, 4)) == ALIGN
    assert call(a7=0) == 0


# ------------------------------------------------------ outputs over inputs
def _refused(f, base, changes):
    for what in changes:
        a = list(base)
        for i, v in what.items():
            a[i] = v
        assert f(*a) == INVALID, what


def test_add_norm_outputs_over_inputs(cpu):
    #       x      ldx t  res    ldr t  M  N   norm gamma  beta   wt eps   h      ldh y      ldy t  sc    stats
    base = [_p(0), 64, 1, _p(1), 64, 1, 4, 64, 0, _p(2), _p(3), 1, 1e-5, _p(4), 64, _p(5), 64, 1, None, _p(6),
            None]
    _refused(cpu.qlora_add_norm_fwd, base, [
        {15: _p(0)}, {15: _p(1)}, {15: _p(4)}, {13: _p(0, 2)}, {13: _p(1), 14: 96},
        {13: _p(0), 5: 0, 3: _p(1)},                     # over x in another type
        {13: _p(2)}, {15: _p(3, 64)}, {19: _p(0)}, {19: _p(5)}, {13: _p(6)},
        {17: 4, 18: _p(1)}, {17: 4, 18: _p(5, 60)}, {17: 4, 18: _p(7), 15: _p(0)}])
    #       dY     ld  t  dH     ld  h      ld  t  M  N   norm gamma wt eps  stats dX     ld  t  dg     db
    base = [_p(0), 64, 1, _p(1), 64, _p(2), 64, 1, 4, 64, 0, _p(3), 1, 1e-5, _p(8), _p(4), 64, 1, _p(5), _p(6),
            0, _p(7), 1 << 20, None]
    _refused(cpu.qlora_add_norm_bwd, base, [
        {15: _p(0, 2)}, {15: _p(1), 16: 96}, {15: _p(2), 17: 0}, {15: _p(0), 2: 0}, {18: _p(1)}, {19: _p(2)},
        {18: _p(6)}, {21: _p(1)}, {15: _p(8)}, {15: _p(3)}])


def test_head_loss_outputs_over_inputs(cpu):
    base = [_p(0), 64, _p(1), 64, 100, 300, 64, _p(2), 3, 1.0, _p(3), _p(5), _p(4), 1 << 24, None]
    _refused(cpu.qlora_head_loss_fwd, base, [
        {10: _p(0)}, {10: _p(1, 299 * 128)}, {10: _p(2)}, {11: _p(3)}, {12: _p(1)}, {11: _p(4)}])
    base = [_p(0), 64, _p(1), 64, 100, 300, 64, _p(2), 3, 1.0, _p(3), _p(4), _p(5), 64, 1, _p(6), 1, 0,
            _p(7), 1 << 25, None]
    _refused(cpu.qlora_head_loss_bwd, base, [
        {12: _p(0)}, {12: _p(1)}, {12: _p(6)}, {15: _p(1)}, {15: _p(0)}, {18: _p(1)}, {12: _p(3)}, {15: _p(4)}])


def test_python_argument_checks():
    """Shapes, types, strides and devices are refused before a pointer is
    taken (the tensors here are on the CPU, which is refused last)."""
    b = torch.bfloat16
    x, xb, W = torch.zeros(4, 8), torch.zeros(4, 8, dtype=b), torch.zeros(9, 8, dtype=b)
    ids, f4, st = torch.zeros(4, dtype=torch.int64), torch.zeros(4), torch.zeros(2, 4)
    e4m3 = torch.float8_e4m3fn
    cases = [
        lambda: q.qlora_add_norm_fwd(x, x),                                   # CPU
        lambda: q.qlora_add_norm_fwd(x, torch.zeros(4, 7)),
        lambda: q.qlora_add_norm_fwd(x, None, h=x),
        lambda: q.qlora_add_norm_fwd(x, x, y_dtype=torch.float16),
        lambda: q.qlora_add_norm_fwd(x, x, y_dtype=e4m3),                     # no scales
        lambda: q.qlora_add_norm_fwd(x, x, scales_out=f4),                    # no codes
        lambda: q.qlora_add_norm_fwd(x, x, y_dtype=e4m3, scales_out=f4[:3]),
        lambda: q.qlora_add_norm_fwd(x.t(), x),
        lambda: q.qlora_add_norm_bwd(x, x, torch.zeros(4, 7)),
        lambda: q.qlora_add_norm_bwd(x, x, xb, dx_dtype=torch.float32),       # dH of another type
        lambda: q.qlora_add_norm_bwd(x, x, grad_dtype=torch.float16),
        lambda: q.qlora_head_loss_fwd(xb, W, ids),                            # CPU
        lambda: q.qlora_head_loss_fwd(x, W, ids),
        lambda: q.qlora_head_loss_fwd(xb, W.float(), ids),
        lambda: q.qlora_head_loss_fwd(xb, W[:, :7], ids),
        lambda: q.qlora_head_loss_fwd(xb, W, ids[:3]),
        lambda: q.qlora_head_loss_fwd(xb, W, ids.short()),
        lambda: q.qlora_head_loss_fwd(xb, W, ids, stats_out=torch.zeros(4, 2)),
        lambda: q.qlora_head_loss_fwd(xb, W, ids, loss=torch.zeros(3)),
        lambda: q.qlora_head_loss_bwd(xb, W, ids, f4.double(), st),
        lambda: q.qlora_head_loss_bwd(xb, W, ids, f4, st[:1]),
        lambda: q.qlora_head_loss_bwd(xb, W, ids, f4, st, accumulate=True),
        lambda: q.qlora_head_loss_bwd(xb, W, ids, f4, st, dW=torch.zeros(8, 8)),
        lambda: q.qlora_head_loss_bwd(xb, W, ids, f4, st, dx_dtype=torch.float16),
        lambda: q.qlora_tensor_list([x.half()]),
        lambda: q.qlora_tensor_list([x.t()]),
        lambda: q.qlora_grad_norm([x]),                                       # CPU
        lambda: q.qlora_grad_norm([]),
        lambda: q.qlora_grad_norm([x], result=torch.zeros(3)),
        lambda: q.qlora_grad_scale([x], torch.zeros(1)),                      # the factor is not on the device
        lambda: q.qlora_adamw_step(f4, f4, f4.clone(), f4.clone(), 1, 1e-3, grad_factor=torch.zeros(1)),
    ]
    for i, c in enumerate(cases):
        with pytest.raises(ValueError):
            c()
            pytest.fail(f"case {i} was accepted")
