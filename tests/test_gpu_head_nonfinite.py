"""Non-finite values in packed sequences: where the state starts anew (g = -inf), nothing that it held or that was added
to it before comes through, whatever it is.  A value may spoil its own chunk (64 tokens, 32 for float32); everything
else that does not depend on it keeps its bits."""
import numpy as np
import pytest
import torch

import selective_state_space_ssm_amd as ssm
from oracle import head

import test_gpu_head as base
from test_gpu_head import DEV, IDS, TYPES, close, make, oracle_args

pytestmark = pytest.mark.gpu

BAD = [float("inf"), float("nan"), -3.4e38]


def chunk(dtype):
    return 64 if dtype == torch.bfloat16 else 32


# tokens, heads, qk heads; tokens with g = -inf
PACKED = [(300, 2, 2, (70, 71, 200)), (1500, 2, 1, (130, 640, 641, 1408)), (260, 4, 2, (64, 128))]


def packed(case, dtype, seed):
    L, h, hk, cuts = case
    x, do, dlast = make(2, L, h, hk, 48, 64, dtype, seed=seed)
    for c in cuts:
        x["g"][:, c] = float("-inf")
    return x, do, dlast


def same(got, want, lo, hi, names, what):
    for n in names:
        assert torch.equal(got[n][:, lo:hi], want[n][:, lo:hi]), (n, lo, hi, what)


def run(x, do, dlast):
    o, last = ssm.ssm_head_scan_fwd(**x)
    return dict(ssm.ssm_head_scan_bwd(do=do, dlast=dlast, **x), o=o, last=last)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("case", PACKED, ids=lambda c: str(c[0]))
def test_what_a_state_held_is_gone_after_a_start(case, dtype):
    """A start state and a token of the first sequence, forwards: outputs from the next start in a later chunk on, the
    last state and what is taken from the states in the gradients (dq, and dg from there on)."""
    L, h, hk, cuts = case
    x, do, dlast = packed(case, dtype, seed=41)
    want = run(x, do, dlast)
    for bad in BAD:
        y = dict(x, h0=x["h0"].clone())
        y["h0"][:, :, 3, 5] = bad
        got = run(y, do, dlast)
        same(got, want, cuts[0], L, ("o", "dq", "dk", "dv", "dg"), bad)
        assert torch.equal(got["last"], want["last"])
        assert torch.equal(got["dh0"], want["dh0"])
    for at in (0, cuts[0] - 1, cuts[-1] - 1):
        after = -(-(at + 1) // chunk(dtype)) * chunk(dtype)  # the chunk after the value's
        start = min([c for c in cuts if c > at])
        for n in ("k", "v"):
            for bad in BAD[:2]:
                y = dict(x, **{n: x[n].clone()})
                y[n][:, at, :, 7] = bad
                got = run(y, do, dlast)
                same(got, want, max(start, after), L, ("o", "dq", "dk", "dv", "dg"), (n, at, bad))
                assert torch.equal(got["last"], want["last"]), (n, at, bad)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("case", PACKED, ids=lambda c: str(c[0]))
def test_what_a_gradient_held_is_gone_before_a_start(case, dtype):
    """The last state's gradient, and a token's, backwards: dk, dv and dg before the start, dh0."""
    L, h, hk, cuts = case
    x, do, dlast = packed(case, dtype, seed=42)
    want = run(x, do, dlast)
    for bad in BAD:
        d = dlast.clone()
        d[:, :, 3, 5] = bad
        got = run(x, do, d)
        same(got, want, 0, cuts[-1], ("dq", "dk", "dv", "dg"), bad)
        assert torch.equal(got["dh0"], want["dh0"])
    for at in (L - 1, cuts[0], cuts[-1]):
        before = at // chunk(dtype) * chunk(dtype)  # the value's chunk
        start = max([c for c in cuts if c <= at])
        for bad in BAD[:2]:
            for n in ("do", "q"):
                y, d = x, do
                if n == "do":
                    d = do.clone()
                    d[:, at, :, 7] = bad
                else:
                    y = dict(x, q=x["q"].clone())
                    y["q"][:, at, :, 7] = bad
                got = run(y, d, dlast)
                same(got, want, 0, min(start, before), ("dq", "dk", "dv"), (n, at, bad))
                assert torch.equal(got["dh0"], want["dh0"]), (n, at, bad)
                # dg is summed over its sequence: one that ends in the value's chunk is spoiled with it
                clean = start if start <= before else max([c for c in cuts if c < start], default=0)
                same(got, want, 0, clean, ("dg",), (n, at, bad))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_a_key_reaches_its_sequence_s_later_outputs_alone(dtype):
    """Starts inside one chunk: the outputs before a key that is not finite and those of the next sequence."""
    x, _, _ = make(1, 90, 2, 2, 48, 64, dtype, seed=46)
    x["g"][:, [5, 20]] = float("-inf")
    want, last = ssm.ssm_head_scan_fwd(**x)
    for bad in BAD[:2]:
        y = dict(x, k=x["k"].clone())
        y["k"][:, 9, :, 7] = bad
        o, last2 = ssm.ssm_head_scan_fwd(**y)
        assert torch.equal(o[:, :9], want[:, :9]) and torch.equal(o[:, 20:], want[:, 20:]) and torch.equal(last2, last)
        assert not bool(torch.isfinite(o[:, 9:20]).any())


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_a_start_at_the_first_token(dtype):
    """Nothing of the start state is left, and no gradient reaches it: dh0 is zero."""
    x, do, dlast = make(2, 40, 2, 2, 32, 32, dtype, seed=43)
    x["g"][:, 0] = float("-inf")
    want = run(x, do, dlast)
    for bad in BAD:
        got = run(dict(x, h0=torch.full_like(x["h0"], bad)), do, dlast)
        for n in want:
            assert torch.equal(got[n], want[n]), n
        d = do.clone()
        d[:, -1] = bad
        assert float(run(x, d, dlast)["dh0"].abs().max()) == 0
    assert float(want["dh0"].abs().max()) == 0


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_step(dtype):
    x, _, _ = make(3, 1, 2, 1, 40, 36, dtype, seed=44)
    one = {n: x[n][:, 0].contiguous() for n in ("q", "k", "v", "g")}
    one["g"][1] = float("-inf")
    o, s = ssm.ssm_head_step(state=x["h0"].clone(), **one)
    for bad in BAD:
        state = x["h0"].clone()
        state[1] = bad
        o2, s2 = ssm.ssm_head_step(state=state, **one)
        assert torch.equal(o2, o) and torch.equal(s2, s)
    fixed = torch.tensor([float("-inf"), -1.0], device=DEV)
    one["g"] = None
    o, s = ssm.ssm_head_step(state=x["h0"].clone(), g_head=fixed, **one)
    state = x["h0"].clone()
    state[:, 0] = float("nan")
    o2, s2 = ssm.ssm_head_step(state=state, g_head=fixed, **one)
    assert torch.equal(o2, o) and torch.equal(s2, s)


def starts_of_their_own(x, seed):
    r = torch.Generator().manual_seed(seed)
    x["g"][(torch.rand(x["g"].shape, generator=r) < 0.02).to(DEV)] = float("-inf")


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("case", [(2, 200, 4, 2, 48, 64), (1, 1500, 2, 1, 16, 33), (1, 130, 2, 2, 128, 128),
                                  (1, 100, 1, 1, 256, 40), (16, 200, 32, 8, 64, 64), (16, 130, 32, 4, 136, 32)], ids=str)
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
