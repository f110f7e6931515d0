"""GPU parity of the delta scan (ssm_delta_scan_fwd, ssm_delta_scan_bwd, ssm_delta_step) against the float64 oracle.

Tolerances.  ``oracle.delta.delta_scan_errors`` carries every step's own rounding through the recurrence.  What goes in:
a float32 sum of n products is off by at most 6 sqrt(n) 2^-24 of the product of its vectors' norms (probabilistic
rounding error analysis, N. J. Higham and T. Mary, SIAM J. Sci. Comput. 41, 2019, with 6 standard deviations), n the
additions in a row (d_key, d_value, a chunk's 64 tokens twice, some roundings of decays and scales).  bfloat16 storage
adds 2^-16 for products of values in two parts, times 1 + |M|, since what is corrected among a chunk's tokens is M times
as large; half a step of float16, 2^-11, for the states, r and e that the gradients are made of; and half a step of the
result, 2^-8 of it (float32: 2^-24, in the sums).
"""
import numpy as np
import pytest
import torch

import selective_state_space_ssm_amd as ssm
from oracle import delta
from selective_state_space_ssm_amd import autograd as ag

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
TYPES = [torch.float32, torch.bfloat16]
IDS = ["f32", "bf16"]
RATES = ("g", "beta")


def make(b, L, h, hk, dk, dv, dtype, seed, g=True, beta=True, h0=True, ragged=False, fused=False, alike=0.3):
    r = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=r)
    unit = lambda t: t / t.square().sum(-1, keepdim=True).sqrt()
    q, k, v = unit(rnd(b, L, hk, dk)), unit(rnd(b, L, hk, dk) + alike * rnd(1, 1, hk, dk)), rnd(b, L, h, dv)
    if fused:
        row = torch.cat([rnd(b, L, 8), q.flatten(2), k.flatten(2), v.flatten(2)], -1).to(dtype).to(DEV)
        q, k, v = (t.unflatten(-1, (n, -1)) for t, n in zip(row[..., 8:].split([hk * dk, hk * dk, h * dv], -1), (hk, hk, h)))
    else:
        q, k, v = (t.to(dtype).to(DEV) for t in (q, k, v))
    rate = torch.logspace(-2, 0.7, h)
    x = dict(q=q, k=k, v=v, scale=dk ** -0.5, g=None, beta=None, h0=None, lengths=None)
    if g:
        x["g"] = (-rate * torch.nn.functional.softplus(rnd(b, L, h))).to(dtype).to(DEV)
    if beta:
        x["beta"] = torch.sigmoid(2 * rnd(b, L, h)).to(dtype).to(DEV)
        x["beta"][:, L // 2] = 0
    if h0:
        x["h0"] = rnd(b, h, dk, dv).to(DEV)
    if ragged:
        n = torch.randint(0, L + 1, (b,), generator=r).to(torch.int32)
        n[0] = L
        x["lengths"] = n.to(DEV)
    return x, rnd(b, L, h, dv).to(dtype).to(DEV), rnd(b, h, dk, dv).to(DEV)


def f64(x):
    return {n: t.double().cpu().numpy() if isinstance(t, torch.Tensor) and t.is_floating_point() else t for n, t in x.items()}


def kappa(y, dtype):
    """1 + the largest norm of a chunk's M."""
    C = 64 if dtype == torch.bfloat16 else 32
    b, L, hk, _ = y["k"].shape
    h = y["v"].shape[2]
    most = 0.0
    for i in range(b):
        for j in range(h):
            for t in range(0, L, C):
                k = y["k"][i, t:t + C, j // (h // hk)]
                G = np.cumsum(y["g"][i, t:t + C, j]) if y["g"] is not None else np.zeros(len(k))
                G = np.maximum(G, -1e4)
                N = np.tril(k @ k.T * np.exp(np.minimum(G[:, None] - G[None], 0)), -1)
                bt = y["beta"][i, t:t + C, j] if y["beta"] is not None else np.ones(len(k))
                most = max(most, np.linalg.norm(N @ np.linalg.inv(np.eye(len(k)) + bt[:, None] * N), 2))
    return 1 + most


def errors(x, dtype, do=None, dlast=None):
    y = f64(x)
    dk, dv = y["q"].shape[3], y["v"].shape[3]
    return delta.delta_scan_errors(**y, do=None if do is None else do.double().cpu().numpy(),
                                   dlast=None if dlast is None else dlast.double().cpu().numpy(),
                                   step=6 * np.sqrt(dk + dv + 2 * 64 + 32) * 2.0 ** -24,
                                   pair=2.0 ** -16 * kappa(y, dtype) if dtype == torch.bfloat16 else 0.0,
                                   kept=2.0 ** -11 if dtype == torch.bfloat16 else 0.0,
                                   chunk=64 if dtype == torch.bfloat16 else 32)


def close(name, got, want, bound):
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    got = got.double().cpu().numpy()
    assert got.shape == want.shape and np.isfinite(got).all(), name
    if name in ("last", "dh0"):
        off, size = (np.sqrt((t * t).sum((-1, -2))) for t in (got - want, want))
    elif name in ("dg", "dbeta"):
        off, size = np.abs(got - want), np.abs(want)
    else:
        off, size = (np.sqrt((t * t).sum(-1)) for t in (got - want, want))
    most = bound * 1.01 + half * size + 1e-30
    assert (off <= most).all(), (name, int((off > most).sum()), float((off / most).max()))


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
CASE_IDS = ["x".join(map(str, c)) for c in CASES]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("case", CASES, ids=CASE_IDS)
@pytest.mark.parametrize("mode", ["plain", "full"])
def test_forward(case, dtype, mode):
    b, L, h, hk, dk, dv = case
    full = mode == "full"
    x, _, _ = make(b, L, h, hk, dk, dv, dtype, seed=L + dk, g=full, beta=full, h0=full, ragged=full, fused=full)
    print(f"[delta fwd] {case} {dtype} {mode}", flush=True)
    o, last = ssm.ssm_delta_scan_fwd(**x)
    torch.cuda.synchronize(DEV)
    wo, wl = delta.delta_scan(**f64(x))
    e = errors(x, dtype)
    close("o", o, wo, e["o"])
    close("last", last, wl, e["last"])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("case", CASES, ids=CASE_IDS)
@pytest.mark.parametrize("mode", ["plain", "full"])
def test_backward(case, dtype, mode):
    b, L, h, hk, dk, dv = case
    full = mode == "full"
    x, do, dlast = make(b, L, h, hk, dk, dv, dtype, seed=L + dv, g=full, beta=full, h0=full, ragged=full, fused=full)
    print(f"[delta bwd] {case} {dtype} {mode}", flush=True)
    dl = dlast if full else None
    got = ssm.ssm_delta_scan_bwd(**x, do=do, dlast=dl)
    torch.cuda.synchronize(DEV)
    y = f64(x)
    want = delta.delta_scan_bwd(**y, do=do.double().cpu().numpy(), dlast=None if dl is None else dl.double().cpu().numpy())
    e = errors(x, dtype, do, dl)
    for n in ("dq", "dk", "dv", "dg", "dbeta", "dh0"):
        if got[n] is None:
            assert n in ("dg", "dbeta") and not full
            continue
        if n == "dg" and not full:
            continue
        close(n, got[n], want[n] if n != "dg" or x["h0"] is not None else np.where(np.arange(L)[None, :, None] == 0, 0, want[n]),
              e[n])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("case", [(1, 1, 1, 1, 1), (3, 4, 2, 32, 32), (2, 6, 3, 64, 130), (5, 2, 1, 128, 128), (2, 2, 2, 256, 256),
                                  (1, 3, 3, 37, 19), (7, 4, 4, 100, 64)], ids=str)
@pytest.mark.parametrize("inplace", [True, False], ids=["inplace", "out"])
def test_step(case, dtype, inplace):
    b, h, hk, dk, dv = case
    x, _, _ = make(b, 1, h, hk, dk, dv, dtype, seed=dk, g=not inplace or dk != 32, beta=dk != 64)
    one = {n: None if x[n] is None else x[n][:, 0].contiguous() for n in ("q", "k", "v", "g", "beta")}
    if one["beta"] is not None:
        one["beta"].fill_(0.7)
    print(f"[delta step] {case} {dtype}", flush=True)
    before = x["h0"].clone()
    out = None if inplace else torch.full_like(before, 7.0)
    o, state = ssm.ssm_delta_step(one["q"], one["k"], one["v"], one["beta"], x["h0"], g=one["g"], scale=x["scale"], state_out=out)
    torch.cuda.synchronize(DEV)
    assert state is (x["h0"] if inplace else out)
    assert inplace or torch.equal(x["h0"], before)
    y = {n: None if t is None else t.double().cpu().numpy()[:, None] for n, t in one.items()}
    y.update(h0=before.double().cpu().numpy(), lengths=None, scale=x["scale"])
    wo, ws = delta.delta_scan(**y)
    e = delta.delta_scan_errors(**y, step=6 * np.sqrt(dk + 32) * 2.0 ** -24)
    close("o", o, wo[:, 0], e["o"][:, 0])
    close("last", state, ws, e["last"])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_steps_go_on_from_the_scan(dtype):
    """A prompt, then token by token, is the scan of all of it."""
    x, _, _ = make(2, 70, 4, 2, 64, 48, dtype, seed=4)
    n = 66
    cut = {m: t[:, :n] if m in ("q", "k", "v") else (t[:, :n].contiguous() if m in RATES else t) for m, t in x.items()}
    _, state = ssm.ssm_delta_scan_fwd(**cut)
    y = f64(x)
    wo, wl = delta.delta_scan(**y)
    e = errors(x, dtype)
    for t in range(n, 70):
        one = {m: x[m][:, t].contiguous() for m in ("q", "k", "v", "g", "beta")}
        o, state = ssm.ssm_delta_step(one["q"], one["k"], one["v"], one["beta"], state, g=one["g"], scale=x["scale"])
        close("o", o, wo[:, t], e["o"][:, t])
    close("last", state, wl, e["last"])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_autograd(dtype):
    x, do, dlast = make(2, 90, 4, 2, 64, 64, dtype, seed=11)
    leaf = {n: t.clone().requires_grad_() for n, t in x.items() if n in ("q", "k", "v", "g", "beta", "h0")}
    o, last = ag.delta_scan(leaf["q"], leaf["k"], leaf["v"], leaf["beta"], g=leaf["g"], h0=leaf["h0"], scale=x["scale"])
    ((o.float() * do.float()).sum() + (last * dlast).sum()).backward()
    want = delta.delta_scan_bwd(**f64(x), do=do.double().cpu().numpy(), dlast=dlast.double().cpu().numpy())
    e = errors(x, dtype, do, dlast)
    for n in leaf:
        close("d" + n, leaf[n].grad, want["d" + n], e["d" + n])
