"""GPU tests of the outputs that the norm behind a residual addition may write over
its own inputs: dX over dY, over dH and over h, h over x and over the residual, at
the widths around every count of threads a row, with the bits of the same call on
outputs of their own."""
import itertools

import numpy as np
import pytest
import torch

import qlora_fine_tuning_blockwise_amd as q
from test_row_ops_gpu import BF16, DEV, F32, randn, say, strided

pytestmark = pytest.mark.gpu

# (rows, width): more rows than workgroups at the last of them, so that a workgroup
# goes on to further rows.
SHAPES = [(5, 1), (3, 3), (2, 7), (37, 64), (5, 511), (9, 512), (3, 1000), (7, 2047), (3, 2048), (5, 4096), (3, 5003),
          (2, 8192), (2, 8193), (3, 16384), (6000, 36), (700, 1030), (530, 5003)]


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("center", [True, False], ids=["layer", "rms"])
def test_gradient_over_an_input(M, N, center):
    g = np.random.default_rng(N + M)
    norm = q.NORM_LAYER if center else q.NORM_RMS
    gamma = randn(g, N, F32, 0.3, 1.0).to(DEV)
    for th, ty, tx in itertools.product((BF16, F32), repeat=3):
        say("add norm bwd over", M, N, th, ty, tx)
        h, dY, dH = randn(g, (M, N), th), randn(g, (M, N), ty), randn(g, (M, N), tx)
        for given, added in itertools.product((True, False), repeat=2):
            stats = None
            if given:
                stats = torch.empty(2, M, device=DEV)
                q.qlora_norm_fwd(h.to(DEV), eps=1e-5, norm=norm, stats_out=stats)

            def call(h_, dY_, dH_, dX=None):
                return q.qlora_add_norm_bwd(dY_, h_, dH_ if added else None, gamma, eps=1e-5, norm=norm, stats=stats,
                                            dx_dtype=tx, dX=dX)

            def fresh():
                return [strided(t, 3)[0] for t in (h, dY, dH)]
            want = call(*fresh())
            for k, t in enumerate((th, ty, tx)):
                if t != tx or (k == 2 and not added):
                    continue
                args = fresh()
                kept = [a.clone() for a in args]
                got = call(*args, dX=args[k])
                assert got[0] is args[k]
                for a, b in zip(got, want):
                    assert torch.equal(a, b), ("h", "dY", "dH")[k]
                for j in range(3):
                    assert j == k or torch.equal(args[j], kept[j])


@pytest.mark.parametrize("M,N", SHAPES)
def test_sum_over_an_input(M, N):
    g = np.random.default_rng(N + M)
    gamma = randn(g, N, F32, 0.3, 1.0).to(DEV)
    for tx, tr, out in itertools.product((BF16, F32), (BF16, F32), (BF16, F32, torch.float8_e4m3fn)):
        say("add norm fwd over", M, N, tx, tr, out)
        x, r = randn(g, (M, N), tx), randn(g, (M, N), tr)
        scales = [torch.empty(M, device=DEV) if out.itemsize == 1 else None for _ in range(2)]

        def call(x_, r_, s, h=None):
            return q.qlora_add_norm_fwd(x_, r_, gamma, eps=1e-5, norm=q.NORM_RMS, h=h, y_dtype=out, scales_out=s)
        y, h = call(x.to(DEV), r.to(DEV), scales[0])
        for k in range(2):
            args = [strided(x, 3)[0], strided(r, 5)[0]]
            if args[k].dtype != tr:
                continue
            y2, h2 = call(*args, scales[1], h=args[k])
            assert h2 is args[k] and torch.equal(h2, h)
            assert torch.equal(y2.view(torch.uint8), y.view(torch.uint8))
            assert scales[0] is None or torch.equal(*scales)


def test_infinite_norm_and_infinite_bound():
    """An infinite norm is above every finite bound (the factor is 0) and not above an
    infinite one (1); a NaN gives NaN either way."""
    for value, bound, want in ((torch.inf, 1.0, 0.0), (torch.inf, torch.inf, 1.0), (3.0, torch.inf, 1.0)):
        for kind in (BF16, F32):
            t = torch.full((300,), 1.0, dtype=kind, device=DEV)
            t[7] = value
            assert float(q.qlora_grad_norm([t], bound)[1]) == want
            t[9] = torch.nan
            assert bool(torch.isnan(q.qlora_grad_norm([t], bound)).all())


@pytest.mark.parametrize("place", range(4))
def test_factor_within_what_the_step_writes(place):
    """Refused, and nothing is written; within the gradient, which is only read, it
    is taken."""
    n = 1000
    written = [torch.full((n,), 0.5, device=DEV) for _ in range(3)] + [torch.full((n,), 0.5, dtype=BF16, device=DEV)]
    grad = torch.full((n,), 0.25, device=DEV)
    for at in (0, n // 2 - 1):
        factor = written[place].view(F32)[at:at + 1]
        with pytest.raises(RuntimeError):
            q.qlora_adamw_step(written[0], grad, written[1], written[2], 1, 1e-3, param_bf16=written[3],
                               grad_factor=factor)
        assert all(bool((t == 0.5).all()) for t in written)
    q.qlora_adamw_step(written[0], grad, written[1], written[2], 1, 1e-3, param_bf16=written[3], grad_factor=grad[7:8])
    assert not bool((written[0] == 0.5).any())
