"""Values of the delta scan that are not finite, in packed and in ragged rows: where the state starts anew (g = -inf) at a
chunk's first token nothing of what it held comes through, and a row without tokens hands on what it was given, however the
row is cut into segments."""
import pytest
import torch

import selective_state_space_ssm_amd as ssm

import test_gpu_delta as base
from test_gpu_delta import DEV, IDS, TYPES, make

pytestmark = pytest.mark.gpu

BAD = [float("inf"), float("nan"), -3.4e38]

# b, L, h, hk, dk, dv; tokens with g = -inf, all of them whole chunks (64 tokens, 32 for float32) on
SEGMENTS = [((1, 4000, 1, 1, 32, 32), (640, 1984)), ((2, 1600, 3, 1, 80, 48), (64, 704, 768)),
            ((1, 2500, 2, 2, 256, 136), (1280,)), ((1, 16384, 4, 4, 64, 64), (1024, 9088))]
WHOLE = [((2, 300, 2, 1, 48, 64), (64, 128, 192))]
CASE_IDS = lambda c: "x".join(map(str, c))


def both(x, do, dlast):
    o, last = ssm.ssm_delta_scan_fwd(**x)
    return dict(ssm.ssm_delta_scan_bwd(do=do, dlast=dlast, **x), o=o, last=last)


def same(got, want, lo, hi, names, what):
    for n in names:
        assert torch.equal(got[n][:, lo:hi], want[n][:, lo:hi]), (n, lo, hi, what)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("case,cuts", SEGMENTS + WHOLE, ids=CASE_IDS)
def test_what_a_state_held_is_gone_after_a_start(case, cuts, dtype):
    """A start state, a value and a key of the first sequence: the other sequences' outputs and the last state keep their
    bits."""
    x, _, _ = make(*case, dtype, seed=case[1])
    for c in cuts:
        x["g"][:, c] = float("-inf")
    o, last = ssm.ssm_delta_scan_fwd(**x)
    assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(last).all())

    def check(y, what):
        o2, last2 = ssm.ssm_delta_scan_fwd(**y)
        assert torch.equal(o2[:, cuts[0]:], o[:, cuts[0]:]) and torch.equal(last2, last), what
        return o2

    for bad in BAD:
        y = dict(x, h0=x["h0"].clone())
        y["h0"][:, :, 3, 5] = bad
        check(y, ("h0", bad))
    for n in ("v", "k"):
        for bad in BAD[:2]:
            y = dict(x, **{n: x[n].clone()})
            y[n][:, 7, :, 5] = bad
            o2 = check(y, (n, bad))
            assert not bool(torch.isfinite(o2[:, cuts[0] - 1, :, 5]).any())  # and reach what they are part of


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("case,cuts", SEGMENTS + WHOLE, ids=CASE_IDS)
def test_what_a_gradient_held_is_gone_before_a_start(case, cuts, dtype):
    """The last state's gradient and an output's: what lies before the last start keeps its bits."""
    x, do, dlast = make(*case, dtype, seed=case[1])
    for c in cuts:
        x["g"][:, c] = float("-inf")
    want = both(x, do, dlast)
    for bad in BAD[:2]:
        d, e = dlast.clone(), do.clone()
        d[:, :, 3, 5] = bad
        e[:, -3, :, 5] = bad
        for got in (both(x, do, d), both(x, e, dlast)):
            same(got, want, 0, cuts[-1], ("dq", "dk", "dv", "dg", "dbeta"), bad)
            assert torch.equal(got["dh0"], want["dh0"]), bad


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("case", [c for c, _ in SEGMENTS], ids=CASE_IDS)
def test_rows_without_tokens_hand_on_what_they_are_given(case, dtype):
    """One value that is not finite stays the only one."""
    b, L, h, hk, dk, dv = case
    x, do, dlast = make(2, L, h, hk, dk, dv, dtype, seed=L)
    x["lengths"] = torch.tensor([0, L], dtype=torch.int32, device=do.device)
    for bad in (float("inf"), -3.4e38):
        x["h0"][0, :, 3, 5] = bad
        dlast[0, :, 3, 5] = bad
        r = both(x, do, dlast)
        assert torch.equal(r["last"][0], x["h0"][0]) and torch.equal(r["dh0"][0], dlast[0])
        assert bool(torch.isfinite(r["o"]).all()) and bool(torch.isfinite(r["dh0"][1]).all())


def starts_of_their_own(x, seed):
    r = torch.Generator().manual_seed(seed)
    x["g"][(torch.rand(x["g"].shape, generator=r) < 0.03).to(DEV)] = float("-inf")


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("case", [(2, 200, 4, 2, 48, 64), (1, 1500, 2, 1, 16, 33), (1, 130, 2, 2, 128, 128), (1, 100, 1, 1, 256, 40),
                                  (16, 200, 32, 8, 64, 64), (3, 130, 6, 3, 136, 72)], ids=CASE_IDS)
def test_heads_that_start_at_tokens_of_their_own(case, dtype, monkeypatch):
    """Starts drawn for every head and token by itself, ragged rows, against the oracle: forward and gradients with the
    bounds of the plain cases."""
    made = base.make

    def with_starts(*a, **kw):
        x, do, dlast = made(*a, **kw)
        if x["g"] is not None:
            starts_of_their_own(x, 45)
        return x, do, dlast

    monkeypatch.setattr(base, "make", with_starts)
    base.test_forward(case, dtype, "full")
    base.test_backward(case, dtype, "full")
