"""The head scan's gradient of the decays where a running sum over the length could go wrong: packed sequences.  The
tolerances are those of test_gpu_head."""
import numpy as np
import pytest
import torch

import selective_state_space_ssm_amd as ssm
from oracle import head

from test_gpu_head import DEV, IDS, TYPES, adds, close, make, oracle_args

pytestmark = pytest.mark.gpu


def dg_bound(x, do, dlast, want, dtype):
    """What dg may be off (test_backward's bound): the dots summed over the tokens from t to the segment's end."""
    num = lambda t: None if t is None else np.abs(t.double().cpu().numpy())
    a = oracle_args(x, True)
    rep = x["v"].shape[2] // x["q"].shape[2]
    a = {**a, "q": np.repeat(a["q"], rep, 2), "k": np.repeat(a["k"], rep, 2)}
    B = head.head_scan_bwd(do=num(do), dlast=num(dlast), **a)
    dots = (a["q"] * B["dq"]).sum(-1) + (a["k"] * B["dk"]).sum(-1)
    reach = 4096 if dtype == torch.bfloat16 else 1024
    span = np.stack([dots[:, t:(t // reach + 1) * reach].sum(1) for t in range(dots.shape[1])], 1)
    each = adds(x) * 2.0 ** -24 + (2.0 ** -15 if dtype == torch.bfloat16 else 0)
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    return half * np.abs(want) + each * (2 * span + B["dg"]) + 1e-30


CUTS = [0, 17, 18, 64, 131, 300, 700, 1300]  # several segments, chunk borders on and off the cuts


def packed(dtype, seed, **kw):
    x, do, dlast = make(1, CUTS[-1], 2, 1, 48, 64, dtype, seed=seed, **kw)
    for c in CUTS[1:-1]:
        x["g"][:, c] = float("-inf")
    return x, do, dlast


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_packed_sequences_against_each_alone(dtype):
    """Later sequences with gradients up to 1e4 times the others': each one's dg is that of a run over it alone."""
    x, do, dlast = packed(dtype, seed=31)
    for i, f in enumerate((1, 1e4, 1, 1e3, 1, 30, 1e4)):
        do[:, CUTS[i]:CUTS[i + 1]] *= f
    r = ssm.ssm_head_scan_bwd(do=do, dlast=dlast, **x)
    for lo, hi in zip(CUTS[:-1], CUTS[1:]):
        y = dict(x, **{n: x[n][:, lo:hi].contiguous() for n in ("q", "k", "v", "g")}, h0=x["h0"] if lo == 0 else None)
        if lo:
            y["g"][:, 0] = 0
        d, dl = do[:, lo:hi], dlast if hi == CUTS[-1] else None
        num = lambda t: None if t is None else t.double().cpu().numpy()
        want = head.head_scan_bwd(do=num(d), dlast=num(dl), **oracle_args(y))["dg"]
        close(f"dg {lo}", r["dg"][:, lo:hi], want, dg_bound(y, d, dl, want, dtype))
        if lo:
            assert float(r["dg"][:, lo].abs().max()) == 0


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_what_follows_a_sequence_leaves_its_gradients_alone(dtype):
    """Packed sequences have nothing to do with each other: the later ones' gradients, 1e4 times as large, change no bit
    of the earlier ones', and the earlier ones' values none of the later ones' outputs."""
    x, do, dlast = packed(dtype, seed=32)
    want = ssm.ssm_head_scan_bwd(do=do, dlast=dlast, **x)
    o, last = ssm.ssm_head_scan_fwd(**x)
    for c in CUTS[1:-1]:
        d = do.clone()
        d[:, c:] *= 1e4
        got = ssm.ssm_head_scan_bwd(do=d, dlast=1e4 * dlast, **x)
        for n in ("dq", "dk", "dv", "dg"):
            assert torch.equal(got[n][:, :c], want[n][:, :c]), (n, c)
        v = x["v"].clone()
        v[:, :c] *= 1e4
        o2, last2 = ssm.ssm_head_scan_fwd(**dict(x, v=v))
        assert torch.equal(o2[:, c:], o[:, c:]) and torch.equal(last2, last), c


def own_pair(x, do):
    """The part of |q| |dq| and of |k| |dk| that comes from a token's own k, v and q, do: it is no part of dg."""
    q, k, v, d = (t.double().abs().cpu().numpy() for t in (x["q"], x["k"], x["v"], do))
    rep = v.shape[2] // q.shape[2]
    return x["scale"] * np.repeat((q * k).sum(-1), rep, 2) * (d * v).sum(-1)


FAST = [-4.0, -8.0, -14.0, -16.0, -20.0, -30.0]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("hk", [6, 2], ids=["own", "shared"])
@pytest.mark.parametrize("L", [50, 700, 1500])
def test_heads_that_forget_fast(L, hk, dtype):
    """dg of a head whose decay leaves little of the token before is as small as that little: what a token's own pair
    gives to q . dq and to k . dk, e^8 to e^30 times as much, must leave no rounding in it.  Rows of two lengths."""
    x, do, dlast = make(2, L, 6, hk, 48, 40, dtype, seed=33 + L)
    x["g"][:] = torch.tensor(FAST, device=DEV).to(dtype)
    x["lengths"] = torch.tensor([L, L - 7], dtype=torch.int32, device=DEV)
    x["h0"] *= 1e-4
    got = ssm.ssm_head_scan_bwd(do=do, **x)["dg"]
    want = head.head_scan_bwd(do=do.double().cpu().numpy(), **oracle_args(x))["dg"]
    num = lambda t: np.abs(t.double().cpu().numpy())
    a = oracle_args(x, True)
    a = {**a, "q": np.repeat(a["q"], 6 // hk, 2), "k": np.repeat(a["k"], 6 // hk, 2)}
    B = head.head_scan_bwd(do=num(do), **a)
    live = (np.arange(L)[None, :] < np.array([L, L - 7])[:, None])[..., None]
    dots = ((a["q"] * B["dq"]).sum(-1) + (a["k"] * B["dk"]).sum(-1) - 2 * own_pair(x, do)) * live
    reach = 4096 if dtype == torch.bfloat16 else 1024
    span = np.stack([dots[:, t:(t // reach + 1) * reach].sum(1) for t in range(L)], 1)
    each = adds(x) * 2.0 ** -24 + (2.0 ** -15 if dtype == torch.bfloat16 else 0)
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    close("dg", got, want, half * np.abs(want) + each * (2 * np.maximum(span, 0) + B["dg"]) + 1e-30)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_strong_and_absent_decay(dtype):
    """Heads that forget within a token, never, at every token or at every other one."""
    x, do, dlast = make(1, 160, 4, 4, 32, 32, dtype, seed=4)
    x["g"][..., 0] = -30.0
    x["g"][..., 1] = 0.0
    x["g"][..., 2] = float("-inf")
    x["g"][:, ::2, 3] = -88.0
    got = ssm.ssm_head_scan_bwd(do=do, dlast=dlast, **x)["dg"]
    num = lambda t: t.double().cpu().numpy()
    want = head.head_scan_bwd(do=num(do), dlast=num(dlast), **oracle_args(x))["dg"]
    close("dg", got, want, dg_bound(x, do, dlast, want, dtype))
    assert float(got[..., 2].abs().max()) == 0


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_rows_without_tokens(dtype):
    L = 150
    x, do, dlast = make(7, L, 2, 2, 32, 48, dtype, seed=1)
    x["lengths"] = torch.tensor([0, 1, 64, 65, L, -5, L + 9], dtype=torch.int32, device=DEV)
    got = ssm.ssm_head_scan_bwd(do=do, dlast=dlast, **x)["dg"]
    num = lambda t: t.double().cpu().numpy()
    want = head.head_scan_bwd(do=num(do), dlast=num(dlast), **oracle_args(x))["dg"]
    close("dg", got, want, dg_bound(x, do, dlast, want, dtype))
