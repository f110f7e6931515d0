"""The head scan's gradients where two heads share a workgroup (bfloat16, shared q and k, enough of them): both widths
of the column tile, both heights, a group of two heads and one of many, ragged rows, two segments."""
import pytest
import torch

import test_gpu_head as base

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", [
    # b, L, h, hk, dk, dv
    (8, 520, 32, 1, 72, 40),   # eight wavefronts a head, 64 rows
    (8, 515, 32, 16, 40, 24),  # four, 32 rows; pairs are whole groups
    (16, 200, 32, 8, 64, 64),  # four, 64 rows, one segment
    (16, 130, 32, 4, 136, 32),  # eight, 32 rows, a second tile of eight columns
], ids=str)
@pytest.mark.parametrize("mode", ["plain", "full"])
def test_backward_pairs(case, mode):
    base.test_backward(case, torch.bfloat16, mode)
