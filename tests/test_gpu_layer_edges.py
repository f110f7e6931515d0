"""The linear layer's activations far out, and the wrappers' backward with gradients as autograd hands them over."""
import numpy as np
import pytest
import torch

import selective_state_space_ssm_amd as ssm
from selective_state_space_ssm_amd import autograd as ag

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.mark.parametrize("rows", [2, 40], ids=["few", "tiles"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activations_far_out(act, rows):
    """pre = +-1e3 .. 1e30 and +inf: the value itself, or zero; slopes one, or zero."""
    w = torch.tensor([1e3, 1e10, 1e19, 1e20, 1e30, -1e3, -1e10, -1e19, -1e20, -1e30], device=DEV)
    x = torch.ones(rows, 1, device=DEV)
    out, pre = ssm.ssm_linear(x, w[:, None].contiguous(), act=act, return_pre=True)
    assert torch.equal(pre, w.expand(rows, -1))
    up = w > 0
    assert torch.equal(out[:, up], pre[:, up]) and float(out[:, ~up].abs().max()) == 0
    _, _, db = ssm.ssm_linear_bwd(x, w[:, None].contiguous(), torch.ones_like(pre), pre, act, want_dx=False, want_dW=False)
    assert torch.equal(db, rows * up.float())
    inf = ssm.ssm_linear(x * float("inf"), torch.ones(1, 1, device=DEV), act=act)
    assert bool((inf == float("inf")).all())


def test_gradients_of_a_concatenation():
    """They are views at any place of one tensor: what each wrapper gets is taken all the same."""
    r = torch.Generator().manual_seed(4)
    rnd = lambda *s: torch.randn(s, generator=r).to(DEV).requires_grad_()
    x, w, W, q, k, v = rnd(3, 5), rnd(5), rnd(5, 5), rnd(1, 3, 1, 5), rnd(1, 3, 1, 5), rnd(1, 3, 1, 5)
    h0 = rnd(1, 1, 5, 5)
    parts = lambda: (ag.linear(x, W), ag.gate_norm(x, w), *ag.head_scan(q, k, v, h0=h0))
    leaves = (x, w, W, q, k, v, h0)
    weight = torch.randn(1 + 15 + 15 + 15 + 25, generator=r).to(DEV)
    whole = torch.cat([x.new_zeros(1)] + [p.flatten() for p in parts()])
    got = torch.autograd.grad((whole * weight).sum(), leaves)
    at, alone = 1, []
    for p in parts():
        alone.append(weight[at:at + p.numel()].clone().view_as(p))
        at += p.numel()
    want = torch.autograd.grad(parts(), leaves, alone)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(bool(torch.isfinite(a).all()) and float(a.abs().max()) > 0 for a in got)
