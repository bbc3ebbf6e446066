"""Outputs of the row operators over their inputs: refused on the host before
anything is enqueued, whatever the strides; columns of one wider buffer share
no memory, and a norm may be written over its own input."""
import ctypes
import os
import subprocess

import pytest
import torch

import qlora_fine_tuning_blockwise_amd as q
from qlora_fine_tuning_blockwise_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 30        # stand-in addresses, 64 MB apart; every call here is refused
FAR = 1 << 26


def _p(i, off=0):
    return ctypes.c_void_p(A + i * FAR + off)


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("stand-in addresses: only where no kernel could run with them")
    if not os.path.exists(_lib.LIB_PATH):
        from qlora_fine_tuning_blockwise_amd import build
        build.build()
    return _lib.load()


def _refused(f, base, changes):
    for what in changes:
        a = list(base)
        for i, v in what.items():
            a[i] = v
        assert f(*a) == 1, what


def test_spans_against_the_bytes_that_they_hold(tmp_path):
    exe = str(tmp_path / "spans_check")
    cmd = ["g++", "-O1", "-std=c++17", "-Wall", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", os.path.join(ROOT, "tests", "csrc", "spans_check.cpp"), "-o", exe]
    for c in (cmd, [exe]):
        p = subprocess.run(c, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
        assert p.returncode == 0, p.stdout[-2000:]
    assert p.stdout.startswith("spans:")


def test_embed_outputs_over_inputs(lib):
    #       W      ldw t  V    D   ids    it M  scale out    ldo t
    base = [_p(0), 64, 1, 100, 64, _p(1), 3, 8, 1.0, _p(2), 64, 1, None]
    _refused(lib.qlora_embed_fwd, base, [
        {9: _p(0)},                                  # over the table's first rows
        {9: _p(0, 99 * 64 * 2)},                     # over its last one
        {9: _p(0, 64), 1: 96, 10: 96},               # half a row further
        {9: _p(1)}, {5: _p(2, 7 * 64 * 2)}])
    #       dY     ldy t  ids    it M  V    D   scale dW     gt acc ws     bytes
    base = [_p(0), 64, 1, _p(1), 2, 8, 100, 64, 1.0, _p(2), 0, 0, _p(3), 1 << 24, None]
    _refused(lib.qlora_embed_bwd, base, [
        {9: _p(0)}, {9: _p(1)}, {0: _p(2, 99 * 64 * 4)}, {12: _p(0)}, {12: _p(1)}, {12: _p(2)},
        {0: _p(2), 10: 1, 11: 1}])


def test_norm_outputs_over_inputs(lib):
    #       x      ldx t  M  N   norm gamma  beta   wt eps   y      ldy t  stats
    base = [_p(0), 64, 1, 4, 64, 0, _p(1), _p(2), 1, 1e-5, _p(3), 64, 1, _p(4), None]
    _refused(lib.qlora_norm_fwd, base, [
        {10: _p(0), 12: 0, 11: 32 + 32},             # x itself in another type
        {10: _p(0), 11: 72},                         # and at another stride
        {10: _p(0, 2)}, {10: _p(0, 128)},            # an element, a row further
        {10: _p(1)}, {10: _p(2)}, {13: _p(0)}, {13: _p(1)}, {13: _p(3, 256)}])
    #       dY     ld  t  x      ld  t  M  N   norm gamma  wt eps  stats  dX     ld  t  dgamma
    base = [_p(0), 64, 1, _p(1), 64, 1, 4, 64, 0, _p(2), 1, 1e-5, _p(3), _p(4), 64, 1,
            _p(5), _p(6), 0, _p(7), 1 << 20, None]
    _refused(lib.qlora_norm_bwd, base, [
        {13: _p(0, 2)}, {13: _p(0), 15: 0}, {13: _p(1), 14: 80}, {13: _p(2)}, {13: _p(3)},
        {16: _p(0)}, {16: _p(1)}, {16: _p(2)}, {17: _p(3)}, {16: _p(4)}, {17: _p(5, 16)},
        {19: _p(0)}, {19: _p(1)}, {19: _p(4)}, {19: _p(6)},
        {13: _p(0), 16: _p(0)}])


def test_distill_outputs_over_inputs(lib):
    V = 100000
    #       z      ldz t  M  V  ids    it t      tt k  T    loss   stats  ws     bytes
    base = [_p(0), V, 1, 4, V, _p(1), 2, _p(2), 0, 8, 2.0, _p(3), _p(4), _p(5), 1 << 24, None]
    _refused(lib.qlora_distill_fwd, base, [
        {11: _p(0)}, {11: _p(1)}, {11: _p(2)}, {12: _p(0, 3 * V * 2)}, {12: _p(3, 8)}, {13: _p(0)},
        {13: _p(3)}, {13: _p(4)}, {13: _p(2)}])
    #                                                       stats  dloss  dz     ldg t
    base = [_p(0), V, 1, 4, V, _p(1), 2, _p(2), 0, 8, 2.0, _p(3), _p(4), _p(5), V, 1, None]
    _refused(lib.qlora_distill_bwd, base, [
        {13: _p(0)},                                 # the gradient over the logits
        {13: _p(0), 15: 0},
        {13: _p(0, 2 * V), 1: 2 * V, 14: 2 * V - 2, 3: 2},   # only the second rows meet
        {13: _p(1)}, {13: _p(2)}, {13: _p(3)}, {13: _p(4)}])


# --------------------------------------------------------------------- on a GPU
@pytest.mark.gpu
def test_a_gradient_over_the_logits_is_refused_by_name():
    dev = torch.device("cuda:0")
    z = torch.randn(3, 500, device=dev)
    ids, t = torch.zeros(3, 4, dtype=torch.int64, device=dev), torch.zeros(3, 4, device=dev)
    stats = torch.empty(2, 3, device=dev)
    q.qlora_distill_fwd(z, ids, t, stats_out=stats)
    kept = z.clone()
    with pytest.raises(RuntimeError, match="an output over an input"):
        q.qlora_distill_bwd(z, ids, t, torch.ones(3, device=dev), stats, dlogits=z)
    with pytest.raises(RuntimeError, match="an output over an input"):
        q.qlora_norm_fwd(z[:, :400], y=z[:, 1:401])
    torch.cuda.synchronize()
    assert torch.equal(z, kept)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(1, 5), (70, 64), (3, 511), (700, 1030), (300, 4096), (5, 16381)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_norm_over_its_own_input_and_beside_it(M, N, dtype):
    """The same bits in a tensor of its own, over x, and in columns next to x
    in one buffer; the backward's over dY and over x, through the C entry."""
    dev = torch.device("cuda:0")
    print("norm in place", M, N, dtype, flush=True)
    g = torch.Generator().manual_seed(M + N)
    x = torch.randn(M, N, generator=g).to(dtype).to(dev)
    dY = torch.randn(M, N, generator=g).to(dtype).to(dev)
    gamma = torch.randn(N, generator=g).to(dtype).to(dev)
    for kind in (q.NORM_LAYER, q.NORM_RMS):
        want = q.qlora_norm_fwd(x, gamma, norm=kind)
        own = x.clone()
        assert q.qlora_norm_fwd(own, gamma, norm=kind, y=own) is own
        both = torch.cat([x, x], 1)
        q.qlora_norm_fwd(both[:, :N], gamma, norm=kind, y=both[:, N:])
        torch.cuda.synchronize()
        assert torch.equal(own, want) and torch.equal(both[:, N:], want) and torch.equal(both[:, :N], x)
        dX, dg, db = q.qlora_norm_bwd(dY, x, gamma, norm=kind)
        code = 1 if dtype == torch.bfloat16 else 0
        ws = torch.empty(q.qlora_norm_bwd_workspace_bytes(M, N), dtype=torch.uint8, device=dev)
        for over_x in (False, True):
            x2, y2, g2, b2 = x.clone(), dY.clone(), torch.empty_like(dg), torch.empty_like(db)
            st = _lib.load().qlora_norm_bwd(
                y2.data_ptr(), N, code, x2.data_ptr(), N, code, M, N, kind, gamma.data_ptr(), code,
                1e-5, None, (x2 if over_x else y2).data_ptr(), N, code, g2.data_ptr(), b2.data_ptr(),
                0, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
            assert st == 0
            torch.cuda.synchronize()
            assert torch.equal(x2 if over_x else y2, dX) and torch.equal(g2, dg) and torch.equal(b2, db)
