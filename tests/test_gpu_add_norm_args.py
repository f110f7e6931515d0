"""The norm with the residual's addition: a residual stream of another type than the one asked for is refused, not taken."""
import pytest
import torch

import selective_state_space_ssm_amd as ssm
from selective_state_space_ssm_amd import autograd as ag

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def test_a_residual_of_another_type_than_asked_for():
    x = torch.randn(3, 64, device=DEV).bfloat16()
    for residual, asked in ((x.clone(), torch.float32), (x.float(), torch.bfloat16)):
        for f in (ssm.ssm_add_norm, ssm.ssm_add_norm_e4m3, ag.add_norm):
            with pytest.raises(TypeError):
                f(x, residual, residual_dtype=asked)
        y, h = ssm.ssm_add_norm(x, residual, residual_dtype=residual.dtype)
        assert h.dtype == residual.dtype
    assert ssm.ssm_add_norm(x, residual_dtype=torch.float32)[1].dtype == torch.float32
    assert ssm.ssm_add_norm(x)[1].dtype == torch.bfloat16
