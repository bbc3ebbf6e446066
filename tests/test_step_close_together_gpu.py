"""GPU tests of the operators that close a training step as a program runs them
together: the residual stream's last norm, the head's loss and its gradients,
the adapter layer behind them, the clipping of all gradients, the optimizer;
captured and replayed, on two streams, and past 32-bit offsets."""
import math

import numpy as np
import pytest
import torch

import qlora_fine_tuning_blockwise_amd as q
from oracle import close
from test_row_ops_gpu import BF16, DEV, F32, check, host, randn, say

pytestmark = pytest.mark.gpu


class Close:
    """x = the adapted layer's output, h = x + residual, y = norm(h), the head's
    loss on y; gradients back to the layer's adapters, the norm and the head."""

    def __init__(self, M=150, V=1030, D=256, seed=0):
        g = np.random.default_rng(seed)
        dev = lambda t: t.to(DEV)  # noqa: E731
        self.M, self.V, self.D = M, V, D
        self.u = dev(randn(g, (M, D), BF16))
        self.residual = dev(randn(g, (M, D), BF16, 1.5))
        self.w = q.qlora_quantize_nf4_dq(dev(randn(g, (D, D), BF16, 0.06)))
        self.A, self.B = dev(randn(g, (D, 16), BF16, 0.06)), dev(randn(g, (16, D), BF16, 0.05))
        self.gamma = dev(randn(g, D, BF16, 0.2, 1.0))
        self.head = dev(randn(g, (V, D), BF16, 2.0 / math.sqrt(D)))
        self.labels = dev(torch.from_numpy(np.where(g.random(M) < 0.3, -100, g.integers(0, V, M))))
        self.dloss = torch.full((M,), 1.0 / M, device=DEV)
        self.stats, self.lstats = torch.empty(2, M, device=DEV), torch.empty(2, M, device=DEV)
        # The gradients that are clipped, in places that stay.
        self.grads = [torch.empty(D, 16, device=DEV), torch.empty(16, D, device=DEV), torch.empty(D, device=DEV),
                      torch.empty(V, D, dtype=BF16, device=DEV)]
        self.clipped = [torch.empty_like(t) for t in self.grads]
        self.lists = q.qlora_tensor_list(self.grads), q.qlora_tensor_list(self.clipped)
        self.max_norm = 0.05

    def run(self):
        o = {}
        o["x"] = q.qlora_linear_fwd(self.w, self.u, self.A, self.B, 32.0, y_dtype=BF16)
        o["y"], o["h"] = q.qlora_add_norm_fwd(o["x"], self.residual, self.gamma, norm=q.NORM_RMS,
                                              stats_out=self.stats)
        o["loss"] = q.qlora_head_loss_fwd(o["y"], self.head, self.labels, stats_out=self.lstats)
        o["dy"], _ = q.qlora_head_loss_bwd(o["y"], self.head, self.labels, self.dloss, self.lstats,
                                           dW=self.grads[3])
        o["dx"], dgamma, _ = q.qlora_add_norm_bwd(o["dy"], o["h"], None, self.gamma, norm=q.NORM_RMS,
                                                  stats=self.stats, want_dbeta=False)
        self.grads[2].copy_(dgamma)
        _, dA, dB = q.qlora_linear_bwd(self.w, self.u, o["dx"], self.A, self.B, 32.0, want_dx=False)
        self.grads[0].copy_(dA)
        self.grads[1].copy_(dB)
        o["norm"] = q.qlora_grad_norm(self.lists[0], self.max_norm)
        q.qlora_grad_scale(self.lists[0], o["norm"][1:], out=self.lists[1])
        for i, (a, b) in enumerate(zip(self.grads, self.clipped)):
            o[f"g{i}"], o[f"c{i}"] = a, b
        return o


def test_the_operators_together():
    """Each against its 64-bit form on the values that the step gave it, and the
    optimizer with the factor against the optimizer on clipped gradients."""
    s = Close()
    o = s.run()
    torch.cuda.synchronize()
    want, err, wst, est, _, _ = close.add_norm_fwd(host(o["h"]), host(s.gamma), None, 1e-5, False)
    assert torch.equal(o["h"], (o["x"].float() + s.residual.float()).to(BF16))
    check(o["y"], want, err, "y")
    check(s.stats, wst, est, "norm stats")
    want, err, wst, est = close.head_loss_fwd(host(o["y"]), host(s.head), host(s.labels))
    check(o["loss"], want, err, "loss")
    check(s.lstats, wst, est, "loss stats")
    (wX, eX), (wW, eW) = close.head_loss_bwd(host(o["y"]), host(s.head), host(s.labels), host(s.dloss))
    check(o["dy"], wX, eX, "dy")
    check(s.grads[3], wW, eW, "head gradient")
    (wX, eX), (wg, eg), _ = close.add_norm_bwd(host(o["dy"]), None, host(o["h"]), host(s.gamma), 1e-5, False)
    check(o["dx"], wX, eX, "dx")
    check(s.grads[2], wg, eg, "dgamma")
    norm, factor = close.grad_norm([host(t) for t in s.grads], float(np.float32(s.max_norm)))
    r = o["norm"].cpu().double()
    assert factor < 1 and abs(float(r[0]) - norm) <= 2.0 ** -23 * norm and abs(float(r[1]) - factor) <= 2.0 ** -23
    for a, b in zip(s.grads, s.clipped):
        assert torch.equal(b, (a.float() * o["norm"][1]).to(a.dtype))
    p = s.A.float()
    state = [[p.clone(), torch.zeros_like(p), torch.zeros_like(p)] for _ in range(2)]
    q.qlora_adamw_step(state[0][0], s.grads[0], state[0][1], state[0][2], 1, 1e-3, grad_factor=o["norm"][1:])
    q.qlora_adamw_step(state[1][0], s.clipped[0], state[1][1], state[1][2], 1, 1e-3)
    assert all(torch.equal(a, b) for a, b in zip(*state)) and not torch.equal(state[0][0], p)


@pytest.mark.parametrize("M", [33, 150, 300])
def test_a_captured_step_replays_with_the_same_bits(M):
    s = Close(M=M, V=1030, D=320, seed=3)
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
        got = {k: v.clone() for k, v in o.items()}
        for t in s.grads + s.clipped:
            t.fill_(5.0)
        eager = s.run()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(got[k], want[k]) and torch.equal(eager[k], want[k]), (replay, k)


def test_a_replayed_graph_follows_its_labels():
    """How many rows carry loss is read on the device: a graph that was captured
    with one batch's labels is right for another's."""
    s = Close(M=200, V=700, D=128, seed=5)
    s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = s.run()
    g = np.random.default_rng(1)
    for share in (0.0, 0.5, 1.0, 0.97):
        s.labels.copy_(torch.from_numpy(np.where(g.random(200) < share, -100, g.integers(0, 700, 200))))
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in o.items()}
        eager = s.run()
        torch.cuda.synchronize()
        for k in got:
            assert torch.equal(got[k], eager[k]), (share, k)


def test_tensors_without_a_list_are_captured_with_their_launch():
    """Plain tensors travel in the launches' arguments: a replay needs nothing of
    the call that captured them but the tensors."""
    g = np.random.default_rng(4)
    made = [randn(g, 3 * k + 1, (F32, BF16)[k % 2]).to(DEV) for k in range(200)]
    out = [torch.empty_like(t) for t in made]

    def run():
        r = q.qlora_grad_norm(made, 1.0)
        q.qlora_grad_scale(made, r[1:], out=out)
        return r
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = run()
    for replay in range(3):
        for t in made:
            t.mul_(1.5)
        for t in out:
            t.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        got, result = [t.clone() for t in out], r.clone()
        eager = run()
        torch.cuda.synchronize()
        assert torch.equal(result, eager) and all(torch.equal(a, b) for a, b in zip(got, out)), replay
        assert float(result[1]) < 1


def test_two_streams_at_once():
    """Two independent steps on two streams, launched in turn without waits, and
    the stream argument in the place of the current stream."""
    a, b = Close(seed=1), Close(M=40, seed=2)
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
    y, h = q.qlora_add_norm_fwd(wa["x"], a.residual, a.gamma, norm=q.NORM_RMS, stream=sa)
    loss = q.qlora_head_loss_fwd(y, a.head, a.labels, stream=sa)
    dy, dW = q.qlora_head_loss_bwd(wb["y"], b.head, b.labels, b.dloss, b.lstats, stream=sb)
    dx, _, _ = q.qlora_add_norm_bwd(dy, wb["h"], dy, b.gamma, norm=q.NORM_RMS, stream=sb)
    r = q.qlora_grad_norm([dx, dW], stream=sb)
    q.qlora_grad_scale([dx], r[1:], stream=sb)
    torch.cuda.synchronize()
    assert torch.equal(h, wa["h"]) and torch.equal(y, wa["y"]) and torch.equal(loss, wa["loss"])
    assert torch.equal(dy, wb["dy"]) and torch.equal(dW, wb["g3"])
    n = math.sqrt(float((dx.double() ** 2).sum() + (dW.double() ** 2).sum()))
    assert abs(float(r[0]) - n) <= 2.0 ** -22 * n


@pytest.mark.parametrize("M", [20011, 140003])
def test_many_rows_of_a_long_batch(M):
    """More rows than threads in the one workgroup that gathers them, and than a
    grid's second dimension has places for, most without a label; their losses
    and gradients as the same rows' alone."""
    g = np.random.default_rng(8)
    V, K = 515, 64
    x, W = randn(g, (M, K), BF16).to(DEV), randn(g, (V, K), BF16, 0.25).to(DEV)
    labels = torch.from_numpy(np.where(g.random(M) < 0.8, -100, g.integers(0, V, M))).to(DEV)
    dloss = randn(g, M).to(DEV)
    stats = torch.empty(2, M, device=DEV)
    loss = q.qlora_head_loss_fwd(x, W, labels, stats_out=stats)
    dX, dW = q.qlora_head_loss_bwd(x, W, labels, dloss, stats, dx_dtype=F32, grad_dtype=F32)
    at = (labels >= 0).nonzero()[:, 0]
    some = torch.cat([at[:50], at[-50:], at[len(at) // 2:len(at) // 2 + 50]])
    want, err, _, _ = close.head_loss_fwd(host(x[some]), host(W), host(labels[some]))
    check(loss[some], want, err, "loss")
    (wX, eX), _ = close.head_loss_bwd(host(x[some]), host(W), host(labels[some]), host(dloss[some]), 1.0, 3)
    check(dX[some], wX, eX, "dX")
    _, (wW, eW) = close.head_loss_bwd(host(x[at]), host(W), host(labels[at]), host(dloss[at]), 1.0, 3)
    check(dW, wW, eW, "dW")
    dead = (labels < 0).nonzero()[:, 0]
    assert not loss[dead].any() and not stats[:, dead].any() and not dX[dead].any()


@pytest.mark.parametrize("M", [3, 70])
def test_head_past_32_bit_offsets(M):
    """A head of 2.2e9 elements that is zero but for three rows: their logits and
    a row of even ones give the loss, and dW the rows."""
    V, K = 540001, 4096
    say("head past 32 bits", M)
    g = np.random.default_rng(M)
    W = torch.zeros(V, K, dtype=BF16, device=DEV)
    at = [7, 524300, V - 1]
    rows = randn(g, (3, K), BF16, 4 / 64)
    W[torch.tensor(at, device=DEV)] = rows.to(DEV)
    x = randn(g, (M, K), BF16)
    labels = torch.tensor([at[i % 3] if i % 5 else 99 for i in range(M)])
    dloss = torch.full((M,), 1.0 / M)
    stats = torch.empty(2, M, device=DEV)
    args = x.to(DEV), W, labels.to(DEV)
    loss = q.qlora_head_loss_fwd(*args, stats_out=stats)
    z = host(x).astype(np.float64) @ host(rows).astype(np.float64).T
    e_z = 2 * 2.0 ** -24 * (K / 8 + 16) * (np.abs(host(x)).astype(np.float64) @ np.abs(host(rows)).T)
    L = np.log(np.exp(z).sum(1) + V - 3)
    zl = np.array([z[i, i % 3] if i % 5 else 0.0 for i in range(M)])
    tol = 2 * e_z.max(1) + 2.0 ** -24 * (V / 16 + 64 + 8 * np.abs(z).max(1) + 40)
    assert np.all(np.abs(host(loss) - (L - zl)) <= tol)
    dX, dW = q.qlora_head_loss_bwd(*args, dloss.to(DEV), stats)
    p = np.exp(z - L[:, None])
    hot = np.zeros((M, 4))
    hot[np.arange(M), [i % 3 if i % 5 else 3 for i in range(M)]] = 1.0
    W4 = np.concatenate([host(rows).astype(np.float64), np.zeros((1, K))])
    p4 = np.concatenate([p, np.exp(-L)[:, None]], 1)
    wX = ((np.concatenate([p, np.zeros((M, 1))], 1) - hot) / M) @ W4
    eX = (p4 * (tol[:, None] + 2.0 ** -8)) @ np.abs(W4) / M + 2.0 ** -20 * (p4 + hot) @ np.abs(W4) / M
    check(dX, wX, eX, "dX")
    d = (p4 - hot) / M
    e_d = (p4 * (tol[:, None] + 2.0 ** -22) + np.abs(p4 - hot) * 2.0 ** -8) / M
    got = dW[torch.tensor(at + [99], device=DEV)]
    xs = host(x).astype(np.float64)
    check(got, d.T @ xs, e_d.T @ np.abs(xs) + 2.0 ** -20 * np.abs(d).T @ np.abs(xs), "dW")
    # an even row in the middle: the same gradient as its neighbours
    assert torch.equal(dW[300000], dW[300001]) and bool((dW[300000] != 0).any())
