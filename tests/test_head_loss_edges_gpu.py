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
