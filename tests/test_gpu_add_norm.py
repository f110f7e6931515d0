"""GPU parity of the norm with the residual's addition (ssm_add_norm, ssm_add_norm_e4m3, ssm_add_norm_bwd) against the
float64 oracle.

Tolerances, element by element.  h is one float32 addition, rounded to its type: half a step of the exact sum.  Against
the oracle of that h, y is off by half a step of its type and by the float32 sum of n squares (half of 6 sqrt(n) 2^-24 of
it, probabilistic analysis with 6 standard deviations, N. J. Higham and T. Mary, SIAM J. Sci. Comput. 41, 2019) and eight
roundings.  e4m3: half a step is 2^-4 of the value, or 2^-10 of the scale below the smallest normal one.  The gradients'
sums over n channels, and dweight's over the rows, count the same way, of the products' absolute values.
"""
import numpy as np
import pytest
import torch

import selective_state_space_ssm_amd as ssm
from oracle import layer
from selective_state_space_ssm_amd import autograd as ag

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F32, BF16 = torch.float32, torch.bfloat16
TYPES = [(F32, F32), (BF16, BF16), (BF16, F32)]
IDS = ["f32", "bf16", "bf16-f32"]
U = 2.0 ** -24
SIZES = [(1, 1), (3, 7), (5, 64), (33, 100), (9, 128), (17, 500), (4, 512), (6, 1001), (11, 1024), (3, 1531), (5, 2048), (2, 4096),
         (3, 4099), (2, 8191), (2, 8192), (1500, 768), (2100, 96)]


def half(t):
    return 2.0 ** -8 if t.dtype == BF16 else U


def f64(t):
    return t.double().cpu().numpy()


def make(rows, n, xt, rt, seed, weight=True):
    r = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=r)
    x, res = rnd(rows, n).to(xt).to(DEV), (2 * rnd(rows, n) + rnd(rows, 1)).to(rt).to(DEV)
    w = (1 + 0.2 * rnd(n)).to(DEV) if weight else None
    return x, res, w, rnd(rows, n).to(xt).to(DEV), rnd(rows, n).to(rt).to(DEV)


def close(got, want, bound, name):
    off = np.abs(f64(got) - want)
    assert (off <= bound).all(), (name, float((off / np.maximum(bound, 1e-300)).max()))


def relative(n):
    return (3 * np.sqrt(n) + 8) * U


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(size, types):
    rows, n = size
    x, res, w, _, _ = make(rows, n, *types, seed=n, weight=n % 3 != 0)
    print(f"[add norm] {size} {types}", flush=True)
    y, h = ssm.ssm_add_norm(x, res, w, eps=1e-5)
    torch.cuda.synchronize(DEV)
    s = f64(x) + f64(res)
    close(h, s, half(h) * 1.001 * np.abs(s) + 1e-30, "h")
    want = layer.add_norm(f64(h), None if w is None else f64(w))
    close(y, want, (half(y) * 1.01 + relative(n)) * np.abs(want) + 1e-30, "y")


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("size,group", [(s, 0) for s in SIZES] + [((5, 32), 32), ((7, 96), 32), ((3, 64), 64), ((9, 448), 64),
                                                                   ((33, 128), 128), ((4, 2048), 128), ((2, 2176), 128),
                                                                   ((3, 8192), 32), ((2, 4096), 64)], ids=str)
def test_e4m3(size, group, types):
    rows, n = size
    x, res, w, _, _ = make(rows, n, *types, seed=n + 1, weight=n % 3 != 1)
    x[0, :group or n] = 0  # a group of nothing
    res[0, :group or n] = 0
    print(f"[add norm e4m3] {size} {group} {types}", flush=True)
    y, scale, h = ssm.ssm_add_norm_e4m3(x, res, w, group=group, eps=1e-5)
    torch.cuda.synchronize(DEV)
    s = f64(x) + f64(res)
    close(h, s, half(h) * 1.001 * np.abs(s) + 1e-30, "h")
    want = layer.add_norm(f64(h), None if w is None else f64(w)).reshape(rows, -1, group or n)
    top = np.abs(want).max(-1) / 448
    assert scale.shape == top.shape
    close(scale, top, (relative(n) + 2 * U) * top, "scale")
    sc = f64(scale)[..., None]
    got = f64(y.float()).reshape(want.shape) * sc
    bound = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * sc) * 1.001 + (relative(n) + 4 * U) * np.abs(want)
    assert (np.abs(got - want) <= bound).all()
    assert scale[0, 0] == 0 and not y.float()[0, :group or n].any()


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("given", [True, False], ids=["dh", "no dh"])
def test_backward(size, types, given):
    rows, n = size
    x, res, w, dy, dh = make(rows, n, *types, seed=n + 2, weight=n % 3 != 2)
    dh = dh if given else None
    _, h = ssm.ssm_add_norm(x, res, w)
    print(f"[add norm bwd] {size} {types}", flush=True)
    dx, dres, dw = ssm.ssm_add_norm_bwd(h, dy, w, dh)
    torch.cuda.synchronize(DEV)
    ww = None if w is None else f64(w)
    want, wdw = layer.add_norm_bwd(f64(h), f64(dy), ww, None if dh is None else f64(dh))
    hh, p = f64(h), f64(dy) * (1 if w is None else ww)
    r = 1 / np.sqrt((hh * hh).mean(-1, keepdims=True) + 1e-5)
    parts = np.abs(r * p) + np.abs(hh) * r * (np.abs(p * hh) * r * r).mean(-1, keepdims=True)
    bound = 4 * relative(n) * parts + 2 * U * (0 if dh is None else np.abs(f64(dh)))
    close(dx, want, bound + half(dx) * 1.01 * np.abs(want) + 1e-30, "dx")
    close(dres, want, bound + half(dres) * 1.01 * np.abs(want) + 1e-30, "dresidual")
    assert (dres is dx) == (types[0] == types[1])
    close(dw, wdw, ((6 * np.sqrt(rows) + 8) * U + relative(n)) * np.abs(f64(dy) * hh * r).sum(0) + 1e-30, "dweight")


def test_gradient_by_differences():
    """One direction in x, residual and weight together, central differences of the oracle's loss."""
    x, res, w, dy, dh = make(5, 36, F32, F32, seed=3)
    leaf = [t.clone().requires_grad_() for t in (x, res, w)]
    y, h = ag.add_norm(*leaf)
    ((y * dy).sum() + (h * dh).sum()).backward()
    r = np.random.RandomState(1)
    d = [r.randn(*t.shape) for t in (x, res, w)]

    def loss(e):
        a, b, c = (f64(t) + e * u for t, u in zip((x, res, w), d))
        return (layer.add_norm(a + b, c) * f64(dy)).sum() + ((a + b) * f64(dh)).sum()

    num = (loss(1e-5) - loss(-1e-5)) / 2e-5
    got = sum((f64(t.grad) * u).sum() for t, u in zip(leaf, d))
    assert abs(num - got) <= 1e-4 * max(1.0, abs(num)), (num, got)


@pytest.mark.parametrize("types", TYPES, ids=IDS)
def test_in_place_and_without(types):
    x, res, w, _, _ = make(9, 300, *types, seed=8)
    y, h = ssm.ssm_add_norm(x, res, w)
    own = res.clone()
    y2, h2 = ssm.ssm_add_norm(x, own, w, h=own)
    assert h2 is own and torch.equal(h2, h) and torch.equal(y2, y)
    y3, h3 = ssm.ssm_add_norm(x, None, w, residual_dtype=types[1])
    assert h3.dtype == types[1] and torch.equal(h3, x.to(types[1]))
    want = layer.add_norm(f64(x), f64(w))
    close(y3, want, (half(y3) * 1.01 + relative(300)) * np.abs(want) + 1e-30, "y")


def test_not_finite():
    """A row with a value that is no number or infinite is lost, the others are as they are without it."""
    x, res, w, _, _ = make(6, 256, BF16, F32, seed=5)
    y, s, h = ssm.ssm_add_norm_e4m3(x, res, w, group=64)
    res2 = res.clone()
    res2[2, 10], res2[4, 0] = float("nan"), float("inf")
    y2, s2, _ = ssm.ssm_add_norm_e4m3(x, res2, w, group=64)
    keep = [0, 1, 3, 5]
    assert torch.equal(y2.view(torch.uint8)[keep], y.view(torch.uint8)[keep]) and torch.equal(s2[keep], s[keep])
    assert s2[2].isnan().all() and y2.float()[2].isnan().all()
    assert s2[4, 0].isnan() and y2.float()[4, :64].isnan().all() and not s2[4, 1:].any()
    tiny = torch.full((2, 64), 1e-41, device=DEV)  # values whose reciprocal is not finite
    y3, s3, _ = ssm.ssm_add_norm_e4m3(tiny, None, torch.full((64,), 1e-3, device=DEV), eps=1.0)
    assert torch.isfinite(y3.float()).all() and torch.isfinite(s3).all()


@pytest.mark.parametrize("types", TYPES, ids=IDS)
def test_autograd(types):
    x, res, w, dy, dh = make(40, 96, *types, seed=21)
    leaf = [t.clone().requires_grad_() for t in (x, res, w)]
    y, h = ag.add_norm(*leaf)
    gx, gr, gw = torch.autograd.grad([y, h], leaf, [dy, dh])
    dx, dres, dw = ssm.ssm_add_norm_bwd(h.detach(), dy, w, dh)
    assert torch.equal(gx, dx) and torch.equal(gr, dres) and torch.equal(gw, dw)
    (only,) = torch.autograd.grad([ag.add_norm(*leaf)[1].float().sum()], [leaf[0]])
    assert torch.equal(only, torch.ones_like(only))
