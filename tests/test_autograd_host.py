"""What the differentiable wrappers ask the library for (CPU, the library's calls replaced)."""
import pytest
import torch

from selective_state_space_ssm_amd import autograd as ag


@pytest.fixture
def asked(monkeypatch):
    calls = []

    def fake(x, W, bias=None, residual=None, act="none", return_pre=False):
        calls.append(return_pre)
        pre = x @ W.t()
        return (pre.clone(), pre) if return_pre else pre

    monkeypatch.setattr(ag, "ssm_linear", fake)
    return calls


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_linear_keeps_the_value_before_act_only_for_a_backward(asked, mode):
    """Without gradients nothing is kept, although the weights require them."""
    x, W = torch.randn(3, 4), torch.nn.Parameter(torch.randn(5, 4))
    residual = torch.randn(3, 5, requires_grad=True)
    with mode():
        ag.linear(x, W, act="silu")
    ag.linear(x, W, act="none")
    ag.linear(x, W.detach(), residual=residual, act="silu")
    assert asked == [False, False, False]
    ag.linear(x, W, act="silu")
    ag.linear(x.clone().requires_grad_(), W.detach(), act="gelu")
    ag.linear(x, W.detach(), torch.zeros(5, requires_grad=True), act="gelu")
    assert asked[3:] == [True, True, True]
