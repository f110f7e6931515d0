"""GPU parity of the gated grouped norm and the token-major linear layer (ssm_gate_norm, ssm_linear and their
gradients) against the float64 oracles, and of the block they form with the head scan.

Tolerances, element by element, from the kernels' roundings: n float32 additions in a row of terms t are off by at
most n 2^-24 sum |t|; the storage type rounds a result by at most half a step (2^-24 or 2^-8 of it).
"""
import numpy as np
import pytest
import torch

import selective_state_space_ssm_amd as ssm
from oracle import head, layer
from selective_state_space_ssm_amd import autograd as ag

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
TYPES = [torch.float32, torch.bfloat16]
IDS = ["f32", "bf16"]
U = 2.0 ** -24


def half(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else U


def num(t):
    return None if t is None else t.detach().double().cpu().numpy()


def close(name, got, want, bound):
    assert tuple(got.shape) == np.shape(want), (name, got.shape, np.shape(want))
    err = np.abs(num(got) - want)
    assert (err <= bound + 1e-30).all(), (name, int((err > bound).sum()), float(np.max(err / np.maximum(bound, 1e-30))))


# rows, channels, groups: single values, groups below, at and between vector sizes, one and two wavefront shapes, the
# workgroup shapes, rows that are not 16-byte aligned
NORMS = [(1, 1, 1), (3, 8, 2), (5, 96, 12), (7, 256, 2), (33, 4096, 32), (4, 100, 2), (3, 999, 3), (2, 1536, 1),
         (5, 2600, 2), (3, 6000, 1), (2, 8192, 1), (1, 8191, 1), (70, 640, 5)]


def norm_case(case, dtype, gate, seed):
    rows, c, groups = case
    r = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, c, generator=r) + 0.3).to(dtype).to(DEV)
    w = (1 + 0.2 * torch.randn(c, generator=r)).to(DEV)
    z = torch.randn(rows, c, generator=r).to(dtype).to(DEV) if gate != "none" else None
    dy = torch.randn(rows, c, generator=r).to(dtype).to(DEV)
    return x, w, z, dy


def norm_parts(x, w, z, groups, center, gate_first, eps):
    """|n^| with what its own error scales with, r (per value), and the gate, for the tolerances."""
    X, Z = num(x), num(z)
    gate = np.ones_like(X) if Z is None else Z / (1 + np.exp(-Z))
    u = (X * gate if gate_first else X).reshape(X.shape[0], groups, -1)
    big = np.abs(u) + np.abs(u).mean(-1, keepdims=True)  # what a value and the mean subtracted from it round by
    if center:
        u = u - u.mean(-1, keepdims=True)
    r = 1 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    off = r * big + np.abs(u * r) * (1 + r * r * (np.abs(u) * big).mean(-1, keepdims=True))
    shape = lambda t: np.broadcast_to(t, u.shape).reshape(X.shape)
    return shape(u * r), shape(off), shape(r), gate


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("case", NORMS, ids=str)
@pytest.mark.parametrize("gate", ["none", "last", "first"])
@pytest.mark.parametrize("center", [False, True], ids=["rms", "center"])
def test_gate_norm(case, dtype, gate, center):
    x, w, z, dy = norm_case(case, dtype, gate, seed=sum(case))
    print(f"[norm] {case} {dtype} {gate} {center}", flush=True)
    groups, first, eps = case[2], gate == "first", 1e-5
    kw = dict(groups=groups, eps=eps, center=center, gate_first=first)
    N = 140 * U  # at most 64 values a lane, 8 more levels, and the roundings of gate, rsqrt and products
    y = ssm.ssm_gate_norm(x, w, z, **kw)
    dx, dw, dz = ssm.ssm_gate_norm_bwd(x, dy, w, z, **kw)
    dx2, dw2, _ = ssm.ssm_gate_norm_bwd(x, dy, w, z, **kw)
    torch.cuda.synchronize(DEV)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    n, off, r, s = norm_parts(x, w, z, groups, center, first, eps)
    W, DY, X = num(w), num(dy), num(x)
    outer = np.ones_like(s) if first else s
    want = layer.gate_norm(x, w, z, **kw)
    close("y", y, want, half(dtype) * np.abs(want) + N * np.abs(W * outer) * off)
    wx, ww, wz = layer.gate_norm_bwd(x, dy, w, z, **kw)
    p = np.abs(DY * outer * W)
    mean = lambda t: np.broadcast_to(t.reshape(X.shape[0], groups, -1).mean(-1, keepdims=True),
                                     (X.shape[0], groups, X.shape[1] // groups)).reshape(X.shape)
    a = np.abs(n) + off
    du = N * r * 4 * (p + mean(p) + a * (mean(p * a) + mean(p)))
    close("dx", dx, wx, half(dtype) * np.abs(wx) + du * (np.abs(s) if first else 1) + N * np.abs(wx))
    rows = X.shape[0]
    close("dw", dw, ww, (N + rows * U) * (np.abs(DY * outer) * a).sum(0) + U * np.abs(ww))
    if z is not None:
        Z = num(z)
        sg = 1 / (1 + np.exp(-Z))
        slope = np.abs(sg * (1 + Z * (1 - sg))) + 0.1  # near its zero the slope's own terms round
        bz = N * (np.abs(wz) + slope * ((du * np.abs(X)) / N + np.abs(wx * X) if first else np.abs(DY * W) * a))
        close("dz", dz, wz, half(dtype) * np.abs(wz) + bz)


def test_gate_norm_without_weight_and_of_flat_rows():
    x = torch.full((4, 64), 3.0, device=DEV)
    x[2] = 0
    y = ssm.ssm_gate_norm(x, center=True, groups=2)
    dx, dw, dz = ssm.ssm_gate_norm_bwd(x, torch.ones_like(x), center=True, groups=2, want_dweight=False)
    assert dw is None and dz is None
    assert float(y.abs().max()) == 0 and float(dx.abs().max()) <= 64 * U * 1e-5 ** -0.5
    y = ssm.ssm_gate_norm(x)
    assert torch.allclose(y[0], torch.full_like(y[0], 3 / (9 + 1e-5) ** 0.5), rtol=1e-6) and float(y[2].abs().max()) == 0


# rows, d_in, d_out
LINEARS = [(1, 1, 1), (1, 64, 64), (8, 512, 200), (16, 4096, 96), (17, 40, 24), (100, 96, 520), (65, 130, 66), (7, 37, 30),
           (300, 1001, 257), (513, 256, 768), (2, 2056, 2048), (1030, 72, 4104), (1, 3, 1500)]


def linear_case(case, dtype, seed, bias=True, residual=True):
    rows, k, m = case
    r = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=r)
    x, W = rnd(rows, k).to(dtype).to(DEV), (rnd(m, k) * k ** -0.5).to(dtype).to(DEV)
    return (x, W, rnd(m).to(dtype).to(DEV) if bias else None, rnd(rows, m).to(dtype).to(DEV) if residual else None,
            rnd(rows, m).to(dtype).to(DEV))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("case", LINEARS, ids=str)
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_linear(case, dtype, act):
    extras = act != "silu"
    x, W, bias, res, dout = linear_case(case, dtype, seed=sum(case), bias=extras, residual=extras)
    print(f"[linear] {case} {dtype} {act}", flush=True)
    out, pre = ssm.ssm_linear(x, W, bias, res, act, return_pre=True)
    out2 = ssm.ssm_linear(x, W, bias, res, act)
    got = ssm.ssm_linear_bwd(x, W, dout, pre if act != "none" else None, act)
    again = ssm.ssm_linear_bwd(x, W, dout, pre if act != "none" else None, act)
    torch.cuda.synchronize(DEV)
    assert torch.equal(out, out2) and all(torch.equal(a, b) for a, b in zip(got, again))
    rows, k, m = case
    X, Wn, D = np.abs(num(x)), np.abs(num(W)), np.abs(num(dout))
    wo, wp = layer.linear(x, W, bias, res, act)
    E = (k + 16) * U * (X @ Wn.T + (0 if bias is None else np.abs(num(bias))))
    close("pre", pre, wp, half(dtype) * np.abs(wp) + E)
    # slopes are at most 1.13; the activation itself is off by a few steps of its argument
    close("out", out, wo, half(dtype) * np.abs(wo) + 1.13 * E + 16 * U * (1 + np.abs(wp)) ** 2 * (act != "none")
          + 2 * U * (np.abs(wo) + (0 if res is None else np.abs(num(res)))))
    wx, ww, wb, dp = layer.linear_bwd(x, W, dout, pre, act)
    low = half(dtype) if act != "none" else 0.0  # dpre's own rounding
    ed = 64 * U * D * (1 + np.abs(num(pre))) ** 2 * (act != "none")
    dpa = np.abs(dp)
    close("dx", got[0], wx, half(dtype) * np.abs(wx) + ((low + (m + 16) * U) * dpa + 1.01 * ed) @ Wn)
    close("dW", got[1], ww, half(dtype) * np.abs(ww) + ((low + (rows + 16) * U) * dpa + 1.01 * ed).T @ X)
    close("dbias", got[2], wb, half(dtype) * np.abs(wb) + ((rows + 16) * U * dpa + 1.01 * ed).sum(0))


def test_linear_parts_alone():
    """Each gradient asked for by itself has the bits it has in company; leading dimensions are kept."""
    x, W, bias, res, dout = linear_case((24, 64, 40), torch.bfloat16, seed=3)
    _, pre = ssm.ssm_linear(x, W, bias, res, "silu", return_pre=True)
    dx, dW, db = ssm.ssm_linear_bwd(x, W, dout, pre, "silu")
    assert torch.equal(ssm.ssm_linear_bwd(x, W, dout, pre, "silu", want_dW=False, want_dbias=False)[0], dx)
    assert torch.equal(ssm.ssm_linear_bwd(x, W, dout, pre, "silu", want_dx=False, want_dbias=False)[1], dW)
    assert torch.equal(ssm.ssm_linear_bwd(x, W, dout, pre, "silu", want_dx=False, want_dW=False)[2], db)
    out = ssm.ssm_linear(x.view(2, 3, 4, 64), W, bias, res.view(2, 3, 4, 40), "silu")
    assert out.shape == (2, 3, 4, 40) and torch.equal(out.view(24, 40), ssm.ssm_linear(x, W, bias, res, "silu"))


# ------------------------------------------------------------ the block
def block(leaf, state=None, lengths=None, heads=4, dv=32):
    """Head scan, norm of every head with its gate, output layer with the residual."""
    o, last = ag.head_scan(leaf["q"], leaf["k"], leaf["v"], g=leaf["g"], h0=state, lengths=lengths)
    b, L = o.shape[:2]
    y = ag.gate_norm(o.reshape(b, L, heads * dv), leaf["w"], leaf["z"], groups=heads)
    return ag.linear(y, leaf["W"], leaf["bias"], leaf["x"], act="silu"), last


def block_leaves(dtype, b=2, L=75, heads=4, hk=2, dk=48, dv=32, dm=72, seed=5):
    r = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=r)
    t = {"q": rnd(b, L, hk, dk), "k": rnd(b, L, hk, dk), "v": rnd(b, L, heads, dv),
         "g": -0.3 * torch.nn.functional.softplus(rnd(b, L, heads)), "z": rnd(b, L, heads * dv),
         "W": rnd(dm, heads * dv) * (heads * dv) ** -0.5, "bias": rnd(dm), "x": rnd(b, L, dm)}
    t = {n: v.to(dtype).to(DEV).requires_grad_() for n, v in t.items()}
    t["w"] = (1 + 0.1 * rnd(heads * dv)).to(DEV).requires_grad_()
    return t


def block_calls(t, dout, dlast):
    """The block and its gradients by the library's calls, in the chain's order."""
    b, L = t["x"].shape[:2]
    o, last = ssm.ssm_head_scan_fwd(t["q"], t["k"], t["v"], g=t["g"])
    rows = o.reshape(b, L, -1)
    y = ssm.ssm_gate_norm(rows, t["w"], t["z"], groups=4)
    out, pre = ssm.ssm_linear(y, t["W"], t["bias"], t["x"], "silu", return_pre=True)
    dy, dW, db = ssm.ssm_linear_bwd(y, t["W"], dout, pre, "silu")
    do, dw, dz = ssm.ssm_gate_norm_bwd(rows, dy, t["w"], t["z"], groups=4)
    h = ssm.ssm_head_scan_bwd(t["q"], t["k"], t["v"], do.reshape(o.shape), g=t["g"], dlast=dlast)
    return dict(out=out, last=last, q=h["dq"], k=h["dk"], v=h["dv"], g=h["dg"], z=dz, W=dW, bias=db, x=dout, w=dw)


def block_run(dtype):
    t = block_leaves(dtype)
    out, last = block(t)
    r = torch.Generator().manual_seed(6)
    dout, dlast = torch.randn(out.shape, generator=r).to(dtype).to(DEV), torch.randn(last.shape, generator=r).to(DEV)
    got = dict(zip(t, torch.autograd.grad([out, last], list(t.values()), [dout, dlast])), out=out, last=last)
    return {n: v.detach() for n, v in t.items()}, dout, dlast, got


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_block_is_the_chain_of_its_calls(dtype):
    """Through autograd the block gives the bits of its calls one after the other (each is held to its oracle above)."""
    t, dout, dlast, got = block_run(dtype)
    want = block_calls(t, dout, dlast)
    torch.cuda.synchronize(DEV)
    for n in want:
        assert torch.equal(got[n], want[n]), n


def test_block_gradients():
    """The float32 block against a chain of the float64 oracles.  A link's result is off by at most about 100 2^-24 of
    the terms it sums, and what it is given by as much more: seven links on the longest chain.  The terms are at most
    a few times the results here (75 tokens, widths up to 128): a factor of four is allowed for that."""
    t, dout, dlast, got = block_run(torch.float32)
    b, L = t["x"].shape[:2]
    scale = 48 ** -0.5
    o, wl = head.head_scan(t["q"], t["k"], t["v"], t["g"], scale=scale)
    o2 = o.reshape(b, L, -1)
    y = layer.gate_norm(o2, t["w"], t["z"], groups=4)
    wo, pre = layer.linear(y, t["W"], t["bias"], t["x"], "silu")
    dy, dW, db, _ = layer.linear_bwd(y, t["W"], dout, pre, "silu")
    dx, dw, dz = layer.gate_norm_bwd(o2, dy, t["w"], t["z"], groups=4)
    h = head.head_scan_bwd(t["q"], t["k"], t["v"], dx.reshape(o.shape), t["g"], scale=scale, dlast=dlast)
    want = dict(out=wo, last=wl, q=h["dq"], k=h["dk"], v=h["dv"], g=h["dg"], z=dz, W=dW, bias=db, x=num(dout), w=dw)
    for n, w in want.items():
        e = np.linalg.norm(num(got[n]) - w) / np.linalg.norm(w)
        assert e <= 4 * 7 * 100 * U, (n, e)


def test_block_step_follows_prompt():
    """Prompt, then tokens one by one, through the serving forms of the three: the same as the whole sequence."""
    t = {n: v.detach() for n, v in block_leaves(torch.float32).items()}
    whole, last = block(t)
    cut = dict(t, **{n: t[n][:, :70].contiguous() for n in ("q", "k", "v", "g", "z", "x")})
    first, state = block(cut)
    outs = [first]
    for i in range(70, 75):
        o, state = ssm.ssm_head_step(*(t[n][:, i].contiguous() for n in ("q", "k", "v")), state, g=t["g"][:, i].contiguous())
        y = ssm.ssm_gate_norm(o.reshape(2, -1), t["w"], t["z"][:, i].contiguous(), groups=4)
        outs.append(ssm.ssm_linear(y, t["W"], t["bias"], t["x"][:, i].contiguous(), "silu")[:, None])
    got = torch.cat(outs, 1)
    # both sides are float32 chains: 2-norm within twice the chain's bound above
    assert float((got - whole).norm() / whole.norm()) <= 2 * 7 * 100 * U
    assert float((state - last).norm() / last.norm()) <= 2 * 7 * 100 * U


@pytest.mark.parametrize("act", ["none", "silu"])
def test_linear_large_tiles(act):
    """Sizes that take the 256 x 256 tiles: ragged rows, columns and k tails in all three products, split sums in dW."""
    rows, k, m = 3336, 1928, 3592
    x, W, bias, res, dout = linear_case((rows, k, m), torch.bfloat16, seed=8)
    out, pre = ssm.ssm_linear(x, W, bias, res, act, return_pre=True)
    got = ssm.ssm_linear_bwd(x, W, dout, pre if act != "none" else None, act)
    torch.cuda.synchronize(DEV)
    # sampled rows and columns against the oracle: the tiles' corners and edges, and some inside
    rs = np.unique(np.r_[0, 15, 16, 255, 256, 257, 1000, 2047, 2048, rows - 9, rows - 8, rows - 1])
    cs = np.unique(np.r_[0, 63, 255, 256, 511, 1536, 1799, 1927])
    half_ = half(torch.bfloat16)
    X, Wn, D, P = num(x), num(W), num(dout), num(pre)
    wo, wp = layer.linear(X[rs], Wn, num(bias), num(res)[rs], act)
    E = (k + 16) * U * (np.abs(X[rs]) @ np.abs(Wn).T + np.abs(num(bias)))
    close("pre", pre[rs], wp, half_ * np.abs(wp) + E)
    close("out", out[rs], wo, half_ * np.abs(wo) + 1.13 * E + 16 * U * (1 + np.abs(wp)) ** 2
          + 2 * U * (np.abs(wo) + np.abs(num(res)[rs])))
    dp = D if act == "none" else D * layer.act(P, act)[1]
    low = half_ if act != "none" else 0.0
    ed = 64 * U * np.abs(D) * (1 + np.abs(P)) ** 2 * (act != "none")
    wx = dp[rs] @ Wn
    close("dx", got[0][rs], wx, half_ * np.abs(wx) + ((low + (m + 16) * U) * np.abs(dp[rs]) + 1.01 * ed[rs]) @ np.abs(Wn))
    ww = dp.T @ X[:, cs]
    close("dW", got[1][:, cs], ww, half_ * np.abs(ww) + ((low + (rows + 16) * U) * np.abs(dp) + 1.01 * ed).T @ np.abs(X[:, cs]))
    wb = dp.sum(0)
    close("dbias", got[2], wb, half_ * np.abs(wb) + ((rows + 16) * U * np.abs(dp) + 1.01 * ed).sum(0))
