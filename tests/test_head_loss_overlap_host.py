"""Outputs of the head loss over its inputs, on the host. No kernel runs here."""
import ctypes

import pytest
import torch

from qlora_fine_tuning_blockwise_amd import _lib

A, FAR, INVALID = 1 << 30, 1 << 26, 1  # stand-in addresses, which no accepted call is given


def _p(i, off=0):
    return ctypes.c_void_p(A + i * FAR + off)


@pytest.mark.parametrize("grad_dtype", [0, 1])
def test_no_rows_and_dW_over_W(grad_dtype):
    """A batch without rows writes zeros to all of dW: not over W."""
    if torch.cuda.is_available():
        pytest.skip("stand-in addresses: only where no kernel could run with them")
    call = _lib.load().qlora_head_loss_bwd

    def bwd(dW, accumulate=0):
        return call(None, 64, _p(1), 64, 0, 300, 64, None, 3, 1.0, None, None, None, 64, 1, dW, grad_dtype, accumulate,
                    None, 0, None)
    size = 300 * 64 * (2 if grad_dtype else 4)
    for off in (0, 16, 300 * 64 * 2 - 16, 16 - size):
        assert bwd(_p(1, off)) == INVALID
        assert bwd(_p(1, off), accumulate=1) == 0  # nothing is written
    for off in (300 * 64 * 2, -size):
        assert bwd(_p(1, off)) != INVALID
