"""The workspace of the head loss's backward against what include/qlora_amd.h
states of it. No kernel runs here."""
import itertools

import pytest
import torch

import qlora_fine_tuning_blockwise_amd as q

MB = 1 << 20
PIECE = {None: 0, torch.bfloat16: 128 * MB, torch.float32: 384 * MB}


def whole(n, to):
    return -(-n // to) * to


@pytest.mark.parametrize("V,K", [(1, 1), (300, 64), (32003, 1027), (32000, 4096), (128000, 4096), (128000, 8192),
                                 (1 << 20, 33), (3000, 65536)])
@pytest.mark.parametrize("M", [1, 16, 17, 64, 65, 300, 2048, 8191, 32768])
def test_backward_workspace_is_as_stated(M, V, K):
    for copy, dx, dw in itertools.product((False, True), PIECE, PIECE):
        got = q.qlora_head_loss_bwd_workspace_bytes(M, V, K, copy, dx, dw)
        rows, width = whole(M, 256), whole(K, 32)
        most = PIECE[dw] + 2 * rows * width * 2 + 32 * rows
        if dx is not None and M <= 16 and K <= 4096 and K % 8 == 0:
            most += 256 * 4 * M * whole(K, 16)
        elif dx is not None:
            most += PIECE[dx] + max(128 * MB, (rows // 256) * (whole(K, 256) // 256) * 256 * 1024)
        if copy:
            most += 32768 * width * 2
        assert 0 < got <= most + 12 * 256, (copy, dx, dw)  # each part in whole 256 bytes


def test_what_a_training_batch_takes():
    """128 MB and no more would hold for one bf16 output without its sums only."""
    size = lambda dx, dw: q.qlora_head_loss_bwd_workspace_bytes(2048, 128000, 4096, False, dx, dw) // MB  # noqa: E731
    assert size(torch.bfloat16, None) == 269
    assert size(torch.bfloat16, torch.bfloat16) == 410
    assert size(torch.float32, torch.float32) == 910
