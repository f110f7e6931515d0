"""The linear layer at sizes that take each of its tiles: 16 columns and few rows, 96 x 96, 128 x 128 with k in parts,
256 x 256, the last three also with rows that are no whole number of 16-byte chunks.  The checks are those of the small
sizes."""
import pytest
import torch

import test_gpu_layer as base

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case,dtype,act", [
    ((5, 100, 5000), torch.bfloat16, "gelu"),
    ((5, 101, 5000), torch.float32, "silu"),
    ((4099, 768, 1536), torch.float32, "silu"),      # 96 x 96 forward, 128 x 128 in two parts for dW
    ((300, 4096, 2048), torch.float32, "none"),      # 128 x 128 in five parts
    ((300, 4096, 2048), torch.bfloat16, "silu"),
    ((777, 1111, 2222), torch.float32, "none"),      # every operand copied, odd outputs
    ((700, 1536, 1001), torch.bfloat16, "silu"),
    ((4099, 1027, 3001), torch.bfloat16, "gelu"),    # 256 x 256 of copied operands, odd outputs
], ids=str)
def test_linear_tiles(case, dtype, act):
    base.test_linear(case, dtype, act)
