"""How much of the gradients' error is rounding to their own type, and how much more the delta scan's backward may add.

A gradient rounded to its type is off by half a step of it and by what its arithmetic is off by: what goes past half a step
is at most the latter.  bfloat16 storage: states, R, r and e are float32 and enter products as two parts, off by 2^-17 of
themselves at most, a product of two of them by 2^-16, independent of each other, so that a sum of products is off by 2^-16
of the root of the sum of its products' squares (``oracle.delta.delta_scan_spread``); the norm over all tokens of what goes past half a step is held to
that.  float32 storage: sums in float32 as in test_gpu_delta.py.
"""
import numpy as np
import pytest
import torch

import selective_state_space_ssm_amd as ssm
from oracle import delta

from test_gpu_delta import IDS, TYPES, f64, make

pytestmark = pytest.mark.gpu

NAMES = ("dq", "dk", "dv", "dg", "dbeta")
CASES = [(1, 130, 2, 2, 128, 128), (1, 200, 2, 2, 256, 256), (2, 300, 4, 4, 64, 64), (1, 1500, 2, 2, 16, 33),
         (1, 700, 3, 3, 100, 72)]


def half_step(x, dtype):
    """Half the distance between the numbers of the type around x."""
    bits = {torch.bfloat16: 8, torch.float32: 24}[dtype]
    return np.ldexp(0.5, np.frexp(x)[1] - bits)


def past_rounding(got, want):
    off = np.abs(got.double().cpu().numpy() - want)
    return np.maximum(off - half_step(want, got.dtype) * (1 + 2.0 ** -20), 0)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("decay", [1.0, 0.05], ids=["decay", "slow"])
def test_gradients_are_rounded_once(case, decay, dtype):
    x, do, dlast = make(*case, dtype, seed=5)
    x["g"] = x["g"] * decay
    y, d, dl = f64(x), do.double().cpu().numpy(), dlast.double().cpu().numpy()
    want = delta.delta_scan_bwd(**y, do=d, dlast=dl)
    spread = delta.delta_scan_spread(**y, do=d, dlast=dl, chunk=64 if dtype == torch.bfloat16 else 32)
    got = ssm.ssm_delta_scan_bwd(**x, do=do, dlast=dlast)
    by = 2.0 ** -16 if dtype == torch.bfloat16 else 6 * np.sqrt(case[4] + case[5] + 160) * 2.0 ** -24
    for n in NAMES:
        past, most = np.linalg.norm(past_rounding(got[n], want[n])), by * np.linalg.norm(spread[n])
        print(f"[delta precision] {n} {past / most:.3f}", flush=True)
        assert past <= most, (n, past / most)
