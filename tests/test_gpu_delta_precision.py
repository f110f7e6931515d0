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

from test_gpu_delta import IDS, TYPES, close, f64, kappa, make

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


def bounds(x, dtype, do, dlast):
    """test_gpu_delta's, with nothing for what the gradients find kept: float32."""
    y = f64(x)
    dk, dv = y["q"].shape[3], y["v"].shape[3]
    return y, delta.delta_scan_errors(**y, do=do.double().cpu().numpy(), dlast=None if dlast is None else dlast.double().cpu().numpy(),
                                      step=6 * np.sqrt(dk + dv + 160) * 2.0 ** -24,
                                      pair=2.0 ** -16 * kappa(y, dtype) if dtype == torch.bfloat16 else 0.0,
                                      chunk=64 if dtype == torch.bfloat16 else 32)


def check(x, do, dlast, dtype, names=NAMES + ("dh0",)):
    y, e = bounds(x, dtype, do, dlast)
    o, last = ssm.ssm_delta_scan_fwd(**x)
    got = ssm.ssm_delta_scan_bwd(**x, do=do, dlast=dlast)
    wo, wl = delta.delta_scan(**y)
    want = delta.delta_scan_bwd(**y, do=do.double().cpu().numpy(), dlast=None if dlast is None else dlast.double().cpu().numpy())
    close("o", o, wo, e["o"])
    close("last", last, wl, e["last"])
    for n in names:
        close(n, got[n], want[n], e[n])
    return got, want


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("by", [1e10, 1e-10], ids=["large", "small"])
def test_later_tokens_of_another_size(by, dtype):
    """The second half of each chunk's values far larger or smaller than the first's: what comes first does not know of it."""
    x, do, dlast = make(2, 192, 2, 2, 48, 64, dtype, seed=31, h0=False)
    late = (torch.arange(192, device=do.device) // 16 % 2).bool()
    x["v"][:, late] = (x["v"][:, late].float() * by).to(dtype)
    x["g"][:, ::32] = float("-inf")
    check(x, do, dlast, dtype, ())


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("by", [1e12, 1e-12], ids=["large", "small"])
def test_packed_sequences_of_different_sizes(by, dtype):
    """Two sequences that share a chunk, values and gradients of the first times and over a factor: each is as exact as by
    itself."""
    x, do, dlast = make(1, 128, 2, 2, 64, 64, dtype, seed=32)
    at = 41
    x["g"][:, at] = float("-inf")
    x["v"][:, :at] = (x["v"][:, :at].float() * by).to(dtype)
    x["h0"] *= by
    do[:, at:] = (do[:, at:].float() * by).to(dtype)
    dlast *= by
    check(x, do, dlast, dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("rate", [0.5, 1.0, 2.0])
def test_a_loss_on_the_last_tokens_alone(rate, dtype):
    """With a decay at every token the gradients of those before are as much smaller, and as exact."""
    x, do, _ = make(1, 64, 2, 2, 64, 64, dtype, seed=33, h0=False)
    x["g"][:] = -rate
    do[:, :-2] = 0
    check(x, do, None, dtype, ("dq", "dk", "dv", "dbeta", "dh0"))
