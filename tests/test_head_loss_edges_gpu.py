"""GPU tests of the vocabulary head's loss at the ends of what it accepts: no
rows, and sizes past what one launch holds."""
import math

import pytest
import torch

import qlora_fine_tuning_blockwise_amd as q
from test_row_ops_gpu import BF16, DEV, F32, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V,K", [(1, 1), (3, 3), (5, 103), (255, 257)])
@pytest.mark.parametrize("kind", [BF16, F32], ids=["bf16", "f32"])
def test_head_loss_without_rows_of_odd_sizes(V, K, kind):
    """All of dW is zero, also where its elements are odd in number, and nothing
    behind it is touched."""
    x, W = torch.empty(0, K, dtype=BF16, device=DEV), torch.ones(V, K, dtype=BF16, device=DEV)
    labels, none = torch.empty(0, dtype=torch.int64, device=DEV), torch.empty(0, device=DEV)
    stats = torch.empty(2, 0, device=DEV)
    buf = torch.full((V * K + 9,), 7.0, dtype=kind, device=DEV)
    dW = buf[:V * K].view(V, K)
    q.qlora_head_loss_bwd(x, W, labels, none, stats, want_dx=False, dW=dW)
    assert not dW.any() and bool((buf[V * K:] == 7.0).all())


def room(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of device memory")


@pytest.mark.parametrize("M", [2, 40])
def test_head_loss_of_a_vocabulary_past_one_launch(M):
    """V above 2^30: four threads an entry are more than 2^32. All logits are 0 but
    for the labels', at the ends of the parts that are launched: with n entries of
    logit 0 the sum is exp(z) + n, exactly enough in fp32 for a bound of its
    rounding, 2^-16 of a logarithm near 21 (V / 128 partial sums, 256 to a thread, each
    at most a step of 2^-24)."""
    room(24)
    V, K = (1 << 30) + 1000, 1
    say("head vocabulary", M, V)
    W = torch.zeros(V, K, dtype=BF16, device=DEV)
    at = torch.tensor([0, (1 << 29) - 1, 1 << 29, (1 << 30) - 1, 1 << 30, V - 1], device=DEV)
    W[at, 0] = 1.0
    labels = at[torch.arange(M, device=DEV) % len(at)].clone()
    if M > 6:
        labels[6] = -1
    x = torch.full((M, K), 24.0, dtype=BF16, device=DEV)
    x[1] = 20.0
    stats = torch.empty(2, M, device=DEV)
    loss = q.qlora_head_loss_fwd(x, W, labels, stats_out=stats).double().cpu()
    for m in range(M):
        z = 20.0 if m == 1 else 24.0
        L = math.log(len(at) + (V - len(at)) * math.exp(-z))
        want = (0.0, 0.0, 0.0) if m == 6 else (L, z, L)
        got = (float(loss[m]), float(stats[0, m]), float(stats[1, m]))
        assert got[1] == want[1] and abs(got[0] - want[0]) < 2 ** -16 * 21 and got[2] == got[0]


def test_head_loss_of_copied_pieces_past_one_launch():
    """2^20 rows by 2^20 entries of a copied W: 2^24 tiles a piece of it, of which a
    count of threads that is cut to 32 bits leaves 8192."""
    room(48)
    M, V, K = 1 << 20, (1 << 20) + 300, 1
    say("head tiles", M, V)
    g = torch.Generator(device=DEV).manual_seed(5)
    W = torch.randn(V, K, generator=g, device=DEV).to(BF16)
    x = torch.full((M, K), math.nan, dtype=BF16, device=DEV)
    labels = torch.full((M,), -1, device=DEV)
    live = torch.arange(0, M, 953, device=DEV)  # 1101 rows
    x[live, 0] = (torch.rand(len(live), generator=g, device=DEV) * 3).to(BF16)
    labels[live] = torch.randint(0, V, (len(live),), generator=g, device=DEV)
    labels[:1], labels[live[-1]] = V - 1, 262144
    loss = q.qlora_head_loss_fwd(x, W, labels)
    z = torch.cat([torch.logsumexp(x[r].double() @ W.double().t(), 1) for r in live.split(100)])
    want = z - x[live, 0].double() * W[labels[live], 0].double()
    # (V / 16 + 64) roundings of 2^-24 in a sum whose logarithm is near 14
    assert bool(((loss[live].double() - want).abs() < (V / 16 + 64) * 2.0 ** -24).all())
    loss[live] = 0.0
    assert not loss.any()


def test_head_loss_of_rows_past_one_launch():
    """M K above 2^35: more than 2^32 threads gather x, of which a count that is cut
    to 32 bits leaves 1023 rows."""
    room(160)
    M, V, K = 1 << 20, 256, 32800
    say("head rows", M, K)
    g = torch.Generator(device=DEV).manual_seed(6)
    W = (torch.randn(V, K, generator=g, device=DEV) / 64).to(BF16)
    x = torch.empty(M, K, dtype=BF16, device=DEV)  # of the rows without a label nothing is read
    labels = torch.full((M,), -1, device=DEV)
    live = torch.arange(7, M, 601, device=DEV)  # 1745 rows
    x[live] = torch.randn(len(live), K, generator=g, device=DEV).to(BF16)
    labels[live] = torch.arange(len(live), device=DEV) * 3 % V
    loss = q.qlora_head_loss_fwd(x, W, labels)
    z = x[live].double() @ W.double().t()
    want = torch.logsumexp(z, 1) - z[torch.arange(len(live), device=DEV), labels[live]]
    # 2 u (K / 8 + 16) of the sum of the products' sizes, at the label and in the sum
    size = float((x[live].double().abs() @ W.double().abs().t()).max())
    assert bool(((loss[live].double() - want).abs() < 4 * 2.0 ** -24 * (K / 8 + 32) * size).all())
    loss[live] = 0.0
    assert not loss.any()


def test_head_loss_without_rows_past_one_launch():
    """dW of more than 2^32 words."""
    room(40)
    V, K = (1 << 17) + 3, 1 << 15
    say("head zeros", V, K)
    x, W = torch.empty(0, K, dtype=BF16, device=DEV), torch.empty(V, K, dtype=BF16, device=DEV)
    labels, none = torch.empty(0, dtype=torch.int64, device=DEV), torch.empty(0, device=DEV)
    dW = torch.ones(V, K, device=DEV)
    q.qlora_head_loss_bwd(x, W, labels, none, torch.empty(2, 0, device=DEV), want_dx=False, dW=dW)
    assert int(dW.count_nonzero()) == 0


@pytest.mark.parametrize("M,K", [(1, 64), (16, 64), (40, 100), (64, 64), (100, 100)])
def test_head_loss_does_no_work_without_labels(M, K):
    """No row has a label: W is neither multiplied nor copied, so that the
    workspace's end, where the sums of a few rows or a copy of W would lie, stays as
    it was. With one label it does not."""
    V = 5000
    x, W = torch.ones(M, K, dtype=BF16, device=DEV), torch.ones(V, K, dtype=BF16, device=DEV)
    labels, dloss = torch.full((M,), -100, device=DEV), torch.ones(M, device=DEV)
    need = q.qlora_head_loss_fwd_workspace_bytes(M, V, K, K % 32 != 0)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    end = ws if M <= 64 else ws[-V * K * 2:]
    stats = torch.empty(2, M, device=DEV)
    for labelled in (0, 1):
        if labelled:
            labels[M // 2] = 4999
        ws.fill_(7)
        loss = q.qlora_head_loss_fwd(x, W, labels, stats_out=stats, workspace=ws)
        assert bool((end == 7).all()) == (not labelled)
        assert int(loss.count_nonzero()) == labelled
        _, dW = q.qlora_head_loss_bwd(x, W, labels, dloss, stats)
        assert bool(dW.any()) == bool(labelled)
