"""The differentiable head scan used without gradients: a module's learned decay goes in as it is."""
import pytest
import torch

import selective_state_space_ssm_amd as ssm
from selective_state_space_ssm_amd import autograd as ag

from test_gpu_head import DEV, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_a_learned_decay_per_head(mode):
    x, _, _ = make(2, 70, 4, 2, 32, 48, torch.float32, seed=51, decay="head")
    want = ssm.ssm_head_scan_fwd(**x)
    decay = torch.nn.Parameter(x["g_head"])
    with mode():
        got = ag.head_scan(**dict(x, g_head=decay))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(ValueError, match="takes no gradient"):
        ag.head_scan(**dict(x, g_head=decay))
