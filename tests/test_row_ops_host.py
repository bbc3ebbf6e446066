"""CPU tests of the row operators (embedding, norm, distillation): the 64-bit
gradients against central differences of the 64-bit forwards, and the host's
checks of every argument. No kernel runs here."""
import ctypes

import numpy as np
import pytest
import torch

import qlora_fine_tuning_blockwise_amd as q
from oracle import rows
from qlora_fine_tuning_blockwise_amd import _lib

FAKE = 1 << 20  # an aligned address that no accepted call is given


def _p(v):
    return ctypes.c_void_p(v)


@pytest.fixture(scope="module")
def lib():
    import os

    if not os.path.exists(_lib.LIB_PATH):
        from qlora_fine_tuning_blockwise_amd import build
        build.build()
    return _lib.load()


# ---------------------------------------------------- gradients by differences
def _along(f, x, d, h=1e-5):
    """Central difference of f along d: its error is O(h^2) of the third
    derivative plus 2^-53 |f| / h, both below 1e-8 of the values here."""
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("center", [True, False])
def test_norm_gradients_are_the_forwards(center):
    g = np.random.default_rng(1)
    M, N, eps = 5, 13, 1e-5
    x, dY = g.standard_normal((M, N)) + 0.5, g.standard_normal((M, N))
    gamma, beta = g.standard_normal(N), g.standard_normal(N)

    def f(x_, g_, b_):
        return (rows.norm_fwd(x_, g_, b_, eps, center)[0] * dY).sum()
    (dX, _), (dg, _), (db, _) = rows.norm_bwd(dY, x, gamma, eps, center)
    d, dn = g.standard_normal((M, N)), g.standard_normal(N)
    for got, want in (((dX * d).sum(), _along(lambda v: f(v, gamma, beta), x, d)),
                      ((dg * dn).sum(), _along(lambda v: f(x, v, beta), gamma, dn)),
                      ((db * dn).sum(), _along(lambda v: f(x, gamma, v), beta, dn))):
        assert abs(got - want) <= 1e-7 * max(1.0, abs(want))


def test_embed_gradient_is_the_forwards():
    g = np.random.default_rng(2)
    V, D, scale = 11, 6, 1.5
    ids = np.array([3, 0, 3, -1, 10, 11, 3, 1 << 40])
    W, d, dY = g.standard_normal((V, D)), g.standard_normal((V, D)), g.standard_normal((ids.size, D))
    dW, _ = rows.embed_bwd(dY, ids, V, scale)
    want = _along(lambda v: (rows.embed_fwd(v, ids, scale)[0] * dY).sum(), W, d)
    assert abs((dW * d).sum() - want) <= 1e-7 * max(1.0, abs(want))


def test_distill_gradient_is_the_forwards():
    g = np.random.default_rng(3)
    M, V, k, T = 6, 17, 5, 1.7
    z, d, t = g.standard_normal((M, V)) * 2, g.standard_normal((M, V)), g.standard_normal((M, k))
    ids = g.integers(0, V, (M, k))
    ids[1] = -1                      # no entry at all
    ids[2] = [4, 4, 4, 2, V]         # repeated, and one outside
    t[3, 1] = -np.inf
    w = g.standard_normal(M)
    w[4] = 0.0
    dz, _ = rows.distill_bwd(z, ids, t, w, T)
    want = _along(lambda v: (rows.distill_fwd(v, ids, t, T)[0] * w).sum(), z, d)
    assert abs((dz * d).sum() - want) <= 1e-7 * max(1.0, abs(want))
    assert not dz[1].any() and not dz[4].any()
    loss = rows.distill_fwd(z, ids, t, T)[0]
    assert loss[1] == 0 and np.all(loss >= 0)
    # the teacher's own distribution on all of the vocabulary: no loss
    same = rows.distill_fwd(z, np.tile(np.arange(V), (M, 1)), z, T)[0]
    assert np.all(np.abs(same) < 1e-14)


# ------------------------------------------------------------------- refusals
def _calls(f, base):
    def call(i, v, **kw):
        a = list(base)
        a[i] = v
        for j, w in kw.items():
            a[int(j[1:])] = w
        return f(*a)
    return call


def test_embed_validation(lib):
    #       W         ldw t  V   D   ids     it M  scale out      ldo t
    base = [_p(FAKE), 64, 1, 100, 64, _p(FAKE), 3, 8, 1.0, _p(FAKE), 64, 1, None]
    call = _calls(lib.qlora_embed_fwd, base)
    assert call(7, -1) == 1
    assert call(8, float("nan")) == 1 and call(8, float("inf")) == 1
    for i in (0, 5, 9):
        assert call(i, None) == 1
    assert call(3, 0) == 2 and call(3, (1 << 31) - 1) == 2
    assert call(4, 0) == 2 and call(4, (1 << 24) + 1, a1=1 << 25, a10=1 << 25) == 2
    assert call(3, 1 << 30, a4=1 << 11, a1=1 << 11, a10=1 << 11) == 2   # V * D past 2^40
    assert call(1, 63) == 2 and call(10, 63) == 2
    assert call(1, 1 << 62) == 2
    assert call(7, (1 << 24) + 1) == 2
    assert call(2, 2) == 4 and call(6, 1) == 4 and call(11, 3) == 4
    assert call(0, _p(FAKE + 1)) == 3 and call(5, _p(FAKE + 4)) == 3 and call(9, _p(FAKE + 1)) == 3
    assert call(0, _p(FAKE + 2), a2=0) == 3   # fp32 at a multiple of two bytes
    assert call(7, 0) == 0
    assert call(7, 0, a0=None, a5=None, a9=None) == 0


def test_embed_bwd_validation(lib):
    #       dY        ldy t  ids      it M  V    D   scale dW      gt acc ws        bytes
    base = [_p(FAKE), 64, 1, _p(FAKE), 2, 8, 100, 64, 1.0, _p(FAKE), 0, 0, _p(FAKE), 1 << 30, None]
    call = _calls(lib.qlora_embed_bwd, base)
    assert call(5, -1) == 1 and call(8, float("inf")) == 1
    for i in (0, 3, 9):
        assert call(i, None) == 1
    assert call(6, 0) == 2 and call(7, 0) == 2 and call(1, 60) == 2 and call(5, 1 << 25) == 2
    assert call(2, 3) == 4 and call(4, 0) == 4 and call(10, 2) == 4
    assert call(9, _p(FAKE + 8)) == 3 and call(12, _p(FAKE + 8)) == 3 and call(3, _p(FAKE + 2)) == 3
    need = q.qlora_embed_bwd_workspace_bytes(8, 64)
    assert need > 0
    assert call(13, need - 1) == 6 and call(12, None) == 6
    assert call(5, 0, a11=1) == 0   # nothing to add
    assert call(5, 0, a9=None) == 1
    assert q.qlora_embed_bwd_workspace_bytes(-1, 64) == 0
    assert q.qlora_embed_bwd_workspace_bytes(8, 0) == 0
    assert q.qlora_embed_bwd_workspace_bytes(0, 64) == 0
    # more tokens than the second grid dimension has tiles for
    assert call(5, (1 << 20) + 1) == 2 and q.qlora_embed_bwd_workspace_bytes((1 << 20) + 1, 64) == 0
    assert q.qlora_embed_bwd_workspace_bytes(1 << 20, 64) > 0


def test_norm_validation(lib):
    #       x         ldx t  M  N   norm gamma   beta      wt eps   y        ldy t  stats
    base = [_p(FAKE), 64, 1, 4, 64, 0, _p(FAKE), _p(FAKE), 1, 1e-5, _p(FAKE), 64, 1, None, None]
    call = _calls(lib.qlora_norm_fwd, base)
    assert call(3, -1) == 1 and call(5, 2) == 1 and call(5, -1) == 1
    for bad in (-1e-6, float("nan"), float("inf")):
        assert call(9, bad) == 1
    assert call(0, None) == 1 and call(10, None) == 1
    assert call(4, 0) == 2 and call(4, 16385, a1=20000, a11=20000) == 2
    assert call(1, 63) == 2 and call(11, 63) == 2 and call(3, 1 << 25) == 2
    assert call(2, 2) == 4 and call(8, 9) == 4 and call(12, 3) == 4
    assert call(0, _p(FAKE + 1)) == 3 and call(6, _p(FAKE + 1)) == 3 and call(13, _p(FAKE + 2)) == 3
    assert call(3, 0) == 0


def test_norm_bwd_validation(lib):
    #       dY        ld  t  x         ld  t  M  N   norm gamma   wt eps  stats dX       ld  t  dgamma
    base = [_p(FAKE), 64, 1, _p(FAKE), 64, 1, 4, 64, 0, _p(FAKE), 1, 1e-5, None, _p(FAKE), 64, 1,
            _p(FAKE), _p(FAKE), 0, _p(FAKE), 1 << 30, None]
    call = _calls(lib.qlora_norm_bwd, base)
    assert call(6, -1) == 1 and call(8, 7) == 1 and call(11, -1.0) == 1
    assert call(0, None) == 1 and call(3, None) == 1
    assert call(7, 16385, a1=20000, a4=20000, a14=20000) == 2
    assert call(1, 8) == 2 and call(4, 8) == 2 and call(14, 8) == 2
    assert call(2, 2) == 4 and call(5, 2) == 4 and call(10, 2) == 4 and call(15, 2) == 4 \
        and call(18, 2) == 4
    assert call(12, _p(FAKE + 2)) == 3 and call(16, _p(FAKE + 2)) == 3 and call(19, _p(FAKE + 4)) == 3
    need = q.qlora_norm_bwd_workspace_bytes(4, 64)
    assert call(20, need - 1) == 6 and call(19, None) == 6
    assert call(13, None, a16=None, a17=None) == 0         # nothing asked for
    assert call(6, 0, a16=None, a17=None) == 0
    assert q.qlora_norm_bwd_workspace_bytes(0, 64) == 0
    assert q.qlora_norm_bwd_workspace_bytes(4, 16385) == 0


def test_distill_validation(lib):
    #       z         ldz t  M  V    ids       it t        tt k  T    loss     stats ws    bytes
    base = [_p(FAKE), 100, 1, 4, 100, _p(FAKE), 2, _p(FAKE), 0, 8, 2.0, _p(FAKE), None, None, 0, None]
    call = _calls(lib.qlora_distill_fwd, base)
    assert call(3, -1) == 1
    for bad in (0.0, -1.0, float("nan"), float("inf"), 2.0 ** -21, 2.0 ** 21):
        assert call(10, bad) == 1
    for i in (0, 5, 7, 11):
        assert call(i, None) == 1
    assert call(4, 0) == 2 and call(4, (1 << 31) - 1, a1=1 << 31) == 2
    assert call(9, 0) == 2 and call(9, 1025) == 2 and call(1, 99) == 2 and call(3, 1 << 25) == 2
    assert call(2, 2) == 4 and call(6, 0) == 4 and call(8, 2) == 4
    assert call(0, _p(FAKE + 1)) == 3 and call(5, _p(FAKE + 2)) == 3 and call(12, _p(FAKE + 1)) == 3
    assert call(3, 0) == 0
    assert q.qlora_distill_fwd_workspace_bytes(-1, 100) == 0
    assert q.qlora_distill_fwd_workspace_bytes(1 << 20, 100) == 0   # one workgroup a row
    need = q.qlora_distill_fwd_workspace_bytes(4, 100000)
    assert need > 0
    assert call(4, 100000, a1=100000) == 6
    assert call(4, 100000, a1=100000, a13=_p(FAKE), a14=need - 1) == 6

    base = [_p(FAKE), 100, 1, 4, 100, _p(FAKE), 2, _p(FAKE), 0, 8, 2.0, _p(FAKE), _p(FAKE),
            _p(FAKE), 100, 1, None]
    call = _calls(lib.qlora_distill_bwd, base)
    for i in (0, 5, 7, 11, 12, 13):
        assert call(i, None) == 1
    assert call(14, 99) == 2 and call(15, 2) == 4 and call(13, _p(FAKE + 1)) == 3
    assert call(10, 0.0) == 1 and call(3, 0) == 0


def test_python_argument_checks():
    """Shapes, types, strides and devices are refused before a pointer is
    taken (the tensors here are on the CPU, which is refused last)."""
    f, b = torch.float32, torch.bfloat16
    x, gam = torch.zeros(4, 8), torch.zeros(8)
    cases = [
        lambda: q.qlora_norm_fwd(x),                                   # CPU
        lambda: q.qlora_norm_fwd(torch.zeros(8)),                      # dims
        lambda: q.qlora_norm_fwd(x.half()),                            # dtype
        lambda: q.qlora_norm_fwd(x.t()),                               # rows not contiguous
        lambda: q.qlora_norm_fwd(gam.expand(4, 8)),                    # a broadcast input
        lambda: q.qlora_norm_fwd(x, torch.zeros(7)),                   # width
        lambda: q.qlora_norm_fwd(x, gam, gam.to(b)),                   # two affine types
        lambda: q.qlora_norm_fwd(x, stats_out=torch.zeros(4, 2)),
        lambda: q.qlora_norm_bwd(torch.zeros(4, 7), x),
        lambda: q.qlora_norm_bwd(x, x, grad_dtype=torch.float16),
        lambda: q.qlora_embed_fwd(x, torch.zeros(3, dtype=torch.int16)),
        lambda: q.qlora_embed_fwd(x, torch.zeros(2, 2, dtype=torch.int64)),
        lambda: q.qlora_embed_fwd(x, torch.zeros(3, dtype=torch.int64)),
        lambda: q.qlora_embed_bwd(x, torch.zeros(5, dtype=torch.int64), 4),
        lambda: q.qlora_embed_bwd(x, torch.zeros(4, dtype=torch.int64), 4, accumulate=True),
        lambda: q.qlora_embed_bwd(x, torch.zeros(4, dtype=torch.int64), 4, dW=torch.zeros(5, 8)),
        lambda: q.qlora_distill_fwd(x, torch.zeros(4, 2), torch.zeros(4, 2)),
        lambda: q.qlora_distill_fwd(x, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 3)),
        lambda: q.qlora_distill_fwd(x, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)),
        lambda: q.qlora_distill_bwd(x, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2),
                                    torch.zeros(4, dtype=torch.float64), torch.zeros(2, 4)),
    ]
    for i, c in enumerate(cases):
        with pytest.raises(ValueError):
            c()
            pytest.fail(f"case {i} was accepted")
    assert f is torch.float32


def test_reductions_in_turn_use_places_of_their_own():
    """A workgroup's reductions of one and two values follow each other with a
    barrier each. Replayed on the host: what a wave may write before the others
    have passed the reduction's barrier is nothing that they may still read."""
    import os
    import re

    root = os.path.dirname(os.path.dirname(os.path.abspath(q.__file__)))
    src = open(os.path.join(root, "qlora_fine_tuning_blockwise_amd", "csrc", "rows.h")).read()
    most = int(re.search(r"constexpr int kMostReduced = (\d+);", src).group(1))
    expr = re.search(r"float\* half = red \+ par \* ([^;]+);", src).group(1)
    for waves in (2, 4, 8, 16):
        for sizes in ((1, 1, 2), (1, 2), (1, 1, 2, 1, 1, 2), (2, 1, 2, 1), (2, 2, 2)):
            read, par = set(), 0
            for k in sizes * 3:
                base = par * eval(expr, {"kMostReduced": most, "waves": waves, "K": k})
                place = set(range(base, base + k * waves))
                assert not place & read, (waves, sizes)
                assert max(place) < 2 * most * waves
                read, par = place, par ^ 1
