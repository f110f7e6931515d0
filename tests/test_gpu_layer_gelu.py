"""gelu and its slope keep their digits in the tail: relative errors on a grid of pre in [-12, 12], float32.

The value is p times a normal distribution function made of a fit (1.2e-7), an exponential and a reciprocal of the
hardware (2^-23 each, the reciprocal's through at most twice its relative size), a second exponential, and about ten
products and sums of terms no larger than the result: 1.2e-7 + (2 + 2 * 2 + 10) * 2^-24 < 1.1e-6.
"""
import math

import numpy as np
import pytest
import torch

import selective_state_space_ssm_amd as ssm

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BOUND = 1.1e-6


def grid():
    p = torch.cat([torch.linspace(-12, 12, 24001), torch.tensor([-0.0, 1e-30, -1e-30, 1e-4, -1e-4])])
    return p.to(DEV)


def cdf(p):
    return np.array([0.5 * math.erfc(-v / math.sqrt(2)) for v in p])


@pytest.mark.parametrize("rows", [1, 40], ids=["few", "tiles"])
def test_value(rows):
    p = grid()
    out, pre = ssm.ssm_linear(torch.ones(rows, 1, device=DEV), p[:, None].contiguous(), act="gelu", return_pre=True)
    assert torch.equal(pre, p.expand(rows, -1))
    x = p.double().cpu().numpy()
    want = x * cdf(x)
    for r in (0, rows - 1):
        err = np.abs(out[r].double().cpu().numpy() - want)
        bad = err > BOUND * np.abs(want)
        assert not bad.any(), (x[bad][:5], float((err / np.maximum(np.abs(want), 1e-300)).max()))


def test_slope():
    """p phi(p) + cdf(p): relative to the two terms, which cancel near p = -0.75."""
    p = grid()
    one = torch.ones(1, p.numel(), device=DEV)
    _, _, slope = ssm.ssm_linear_bwd(torch.ones(1, 1, device=DEV), p[:, None].contiguous(), one, p[None].contiguous(), "gelu",
                                     want_dx=False, want_dW=False)
    x = p.double().cpu().numpy()
    phi = np.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    want = x * phi + cdf(x)
    err = np.abs(slope.double().cpu().numpy() - want)
    size = np.abs(x) * phi + cdf(x)
    assert (err <= BOUND * size).all(), float((err / size).max())
