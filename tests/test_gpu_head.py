"""GPU parity of the head scan (ssm_head_scan_fwd, ssm_head_scan_bwd, ssm_head_step) against the float64 oracle.

Tolerances, element by element.  Let B be the result with every product taken in absolute value (the oracle run on
|q|, |k|, |v|, |do|): any float32 sum of the same products is off by at most n 2^-24 B, n the additions in a row
(products over d, a chunk of at most 64, two per chunk for the state, and a few roundings of decays and scales).
bfloat16 adds half a step of the output, 2^-8 |result|, and what scores and the state lose in two parts, 2^-16 B each.  dg is a sum of dots of q with dq and k with dk before those are rounded, scores in two parts (2^-16 B each),
from a segment's end (at most 1024 tokens for float32, 4096 for bfloat16) to the token, plus <R, S> there.
"""
import numpy as np
import pytest
import torch

import selective_state_space_ssm_amd as ssm
from oracle import head
from selective_state_space_ssm_amd import autograd as ag

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
TYPES = [torch.float32, torch.bfloat16]
IDS = ["f32", "bf16"]


def make(b, L, h, hk, dk, dv, dtype, seed, decay="token", h0=True, ragged=False, fused=False):
    r = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=r)
    if fused:
        row = rnd(b, L, 2 * hk * dk + h * dv + 8).to(dtype).to(DEV)
        q, k, v = (t.unflatten(-1, (n, -1)) for t, n in zip(row[..., 8:].split([hk * dk, hk * dk, h * dv], -1), (hk, hk, h)))
    else:
        q, k, v = (rnd(b, L, n, d).to(dtype).to(DEV) for n, d in ((hk, dk), (hk, dk), (h, dv)))
    x = dict(q=q, k=k, v=v, g=None, g_head=None, h0=None, lengths=None, scale=dk ** -0.5)
    rate = torch.logspace(-2, 0.7, h)
    if decay == "token":
        x["g"] = (-rate * torch.nn.functional.softplus(rnd(b, L, h))).to(dtype).to(DEV)
    elif decay == "head":
        x["g_head"] = (-rate).to(DEV)
    if h0:
        x["h0"] = rnd(b, h, dk, dv).to(DEV)
    if ragged:
        n = torch.randint(0, L + 1, (b,), generator=r).to(torch.int32)
        n[0] = L
        x["lengths"] = n.to(DEV)
    return x, rnd(b, L, h, dv).to(dtype).to(DEV), rnd(b, h, dk, dv).to(DEV)


def oracle_args(x, absolute=False):
    a = {n: (None if x[n] is None else x[n].double().cpu().numpy()) for n in ("q", "k", "v", "h0")}
    if absolute:
        a = {n: None if t is None else np.abs(t) for n, t in a.items()}
    g = x["g"] if x["g"] is not None else x["g_head"]
    return dict(a, g=None if g is None else g.double().cpu().numpy(), lengths=x["lengths"], scale=x["scale"])


def adds(x):
    b, L, _, dk = x["q"].shape
    return dk + x["v"].shape[3] + 64 + 2 * (L // 32 + 1) + 32


def close(name, got, want, bound):
    got = got.double().cpu().numpy()
    bad = np.abs(got - want) > bound
    assert not bad.any(), (name, int(bad.sum()), float(np.max(np.abs(got - want) / np.maximum(bound, 1e-300))))


def bounds(x, want, B, low):
    n = adds(x) * 2.0 ** -24
    tiny = 1e-30
    if low == torch.bfloat16:
        return 2.0 ** -8 * np.abs(want) + (2 * 2.0 ** -16 + n) * 1.01 * B + tiny
    return n * B + tiny


CASES = [
    # b, L, h, hk, dk, dv
    (1, 1, 1, 1, 1, 1),
    (1, 17, 4, 4, 32, 32),
    (2, 64, 2, 1, 64, 64),       # whole chunks
    (2, 65, 3, 3, 48, 80),       # one past a chunk, widths between tiles
    (1, 130, 2, 2, 128, 128),
    (2, 100, 4, 2, 37, 19),      # nothing aligned
    (1, 200, 2, 1, 256, 256),    # the widest
    (1, 1500, 2, 1, 16, 33),     # segments; an odd width
    (3, 40, 6, 3, 64, 130),      # a third column tile of two columns
    (1, 2100, 1, 1, 100, 200),
]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("case", CASES, ids=["x".join(map(str, c)) for c in CASES])
@pytest.mark.parametrize("mode", ["plain", "full"])
def test_forward(case, dtype, mode):
    b, L, h, hk, dk, dv = case
    full = mode == "full"
    x, _, _ = make(b, L, h, hk, dk, dv, dtype, seed=L + dk, decay="token" if full else "head", h0=full, ragged=full, fused=full)
    print(f"[head fwd] {case} {dtype} {mode}", flush=True)
    o, last = ssm.ssm_head_scan_fwd(**x)
    torch.cuda.synchronize(DEV)
    wo, wl = head.head_scan(**oracle_args(x))
    bo, bl = head.head_scan(**oracle_args(x, True))
    close("o", o, wo, bounds(x, wo, bo, dtype))
    close("last", last, wl, bounds(x, wl, bl, torch.float32))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("case", CASES, ids=["x".join(map(str, c)) for c in CASES])
@pytest.mark.parametrize("mode", ["plain", "full"])
def test_backward(case, dtype, mode):
    b, L, h, hk, dk, dv = case
    full = mode == "full"
    x, do, dlast = make(b, L, h, hk, dk, dv, dtype, seed=L + dv, h0=full, ragged=full, fused=full)
    print(f"[head bwd] {case} {dtype} {mode}", flush=True)
    dlast = dlast if full else None
    got = ssm.ssm_head_scan_bwd(do=do, dlast=dlast, **x)
    torch.cuda.synchronize(DEV)
    num = lambda t: None if t is None else t.double().cpu().numpy()
    a, ab = oracle_args(x), oracle_args(x, True)
    want = head.head_scan_bwd(do=num(do), dlast=num(dlast), **a)
    B = head.head_scan_bwd(do=np.abs(num(do)), dlast=None if dlast is None else np.abs(num(dlast)), **ab)
    rep = h // hk
    for n in ("dq", "dk", "dv"):
        close(n, got[n], want[n], bounds(x, want[n], B[n], dtype))
    close("dh0", got["dh0"], want["dh0"], bounds(x, want["dh0"], B["dh0"], torch.float32))
    # dg: what the dots may be off, summed over the tokens from t to the segment's end; B's own dg bounds <R, S>
    ab1 = {**ab, "q": np.repeat(ab["q"], rep, 2), "k": np.repeat(ab["k"], rep, 2)}
    Bh = head.head_scan_bwd(do=np.abs(num(do)), dlast=None if dlast is None else np.abs(num(dlast)), **ab1)
    dots = (ab1["q"] * Bh["dq"]).sum(-1) + (ab1["k"] * Bh["dk"]).sum(-1)
    reach = 4096 if dtype == torch.bfloat16 else 1024
    span = np.stack([dots[:, t:(t // reach + 1) * reach].sum(1) for t in range(L)], 1)
    each = adds(x) * 2.0 ** -24 + (2.0 ** -15 if dtype == torch.bfloat16 else 0)
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    # <R, S> of a segment's end is at most B's dg there plus what it lost on the way, which `span` holds
    close("dg", got["dg"], want["dg"], half * np.abs(want["dg"]) + each * (2 * span + Bh["dg"]) + 1e-30)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("case", [(1, 1, 1, 1, 1), (3, 4, 2, 64, 64), (2, 6, 3, 100, 37), (2, 2, 1, 256, 256), (1, 3, 3, 48, 80)],
                         ids=str)
def test_step(case, dtype):
    b, h, hk, dk, dv = case
    print(f"[head step] {case} {dtype}", flush=True)
    for decay in ("token", "head", "none"):
        x, _, _ = make(b, 1, h, hk, dk, dv, dtype, seed=dk, decay=decay)
        one = {n: None if x[n] is None else x[n][:, 0].contiguous() for n in ("q", "k", "v", "g")}
        state = x["h0"].clone()
        out = torch.empty_like(state)
        o, new = ssm.ssm_head_step(one["q"], one["k"], one["v"], state, g=one["g"], g_head=x["g_head"], scale=x["scale"],
                                   state_out=out)
        assert new is out and torch.equal(state, x["h0"])
        o2, new2 = ssm.ssm_head_step(one["q"], one["k"], one["v"], state, g=one["g"], g_head=x["g_head"], scale=x["scale"])
        assert new2 is state and torch.equal(state, out) and torch.equal(o, o2)  # in place: the same
        torch.cuda.synchronize(DEV)
        wo, wl = head.head_scan(**oracle_args(x))
        bo, bl = head.head_scan(**oracle_args(x, True))
        n = adds(x) * 2.0 ** -24
        close("o", o[:, None], wo, n * bo + (2.0 ** -8 * np.abs(wo) if dtype == torch.bfloat16 else 0) + 1e-30)
        close("state", new, wl, n * bl + 1e-30)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_prompt_then_tokens_is_one_sequence(dtype):
    """A prompt's last state, stepped on token by token, against the scan over all of it."""
    x, _, _ = make(2, 70, 4, 2, 64, 48, dtype, seed=9)
    wo, wl = head.head_scan(**oracle_args(x))
    bo, bl = head.head_scan(**oracle_args(x, True))
    cut = dict(x, **{n: x[n][:, :66] for n in ("q", "k", "v")}, g=x["g"][:, :66].contiguous())
    _, state = ssm.ssm_head_scan_fwd(**cut)
    for t in range(66, 70):
        o, state = ssm.ssm_head_step(*(x[n][:, t].contiguous() for n in ("q", "k", "v")), state, g=x["g"][:, t].contiguous(),
                                     scale=x["scale"])
        n = adds(x) * 2.0 ** -24
        close(f"o{t}", o, wo[:, t], n * bo[:, t] + (2.0 ** -8 * np.abs(wo[:, t]) if dtype == torch.bfloat16 else 0) + 1e-30)
    close("state", state, wl, adds(x) * 2.0 ** -24 * bl)
