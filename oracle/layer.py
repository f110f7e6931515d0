"""float64 oracles of the gated grouped norm and the linear layer on token rows, NumPy on the CPU, from their
definitions; share no code with the GPU path."""
import math

import numpy as np

from .head import _arr


def _erfc(x):
    return np.vectorize(math.erfc, otypes=[np.float64])(x)


def gate_norm(x, weight=None, z=None, groups=1, eps=1e-5, center=False, gate_first=False):
    x, w, z = _arr(x), _arr(weight), _arr(z)
    gate = 1.0 if z is None else z / (1 + np.exp(-z))
    u = (x * gate if gate_first else x).reshape(*x.shape[:-1], groups, -1)
    if center:
        u = u - u.mean(-1, keepdims=True)
    n = (u / np.sqrt((u * u).mean(-1, keepdims=True) + eps)).reshape(x.shape)
    y = n if w is None else n * w
    return y if gate_first else y * gate


def gate_norm_bwd(x, dy, weight=None, z=None, groups=1, eps=1e-5, center=False, gate_first=False):
    """(dx, dweight, dz or None)."""
    x, dy, z = _arr(x), _arr(dy), _arr(z)
    w = np.ones(x.shape[-1]) if weight is None else _arr(weight)
    sg = None if z is None else 1 / (1 + np.exp(-z))
    gate = 1.0 if z is None else z * sg
    slope = None if z is None else sg * (1 + z * (1 - sg))
    split = lambda t: t.reshape(*x.shape[:-1], groups, -1)
    u = split(x * gate if gate_first else x)
    if center:
        u = u - u.mean(-1, keepdims=True)
    r = 1 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    n = (u * r).reshape(x.shape)
    dn = dy * (1.0 if gate_first else gate)
    p = split(dn * w)
    du = p - split(n) * (p * split(n)).mean(-1, keepdims=True)
    if center:
        du = du - p.mean(-1, keepdims=True)
    du = (du * r).reshape(x.shape)
    dw = (dn * n).reshape(-1, x.shape[-1]).sum(0)
    if z is None:
        return du, dw, None
    return (du * gate, dw, du * x * slope) if gate_first else (du, dw, dy * w * n * slope)


def act(p, kind):
    """(value, slope) of an activation."""
    if kind == "silu":
        s = 1 / (1 + np.exp(-p))
        return p * s, s * (1 + p * (1 - s))
    if kind == "gelu":
        cdf = 0.5 * _erfc(-p / math.sqrt(2))
        return p * cdf, cdf + p * np.exp(-p * p / 2) / math.sqrt(2 * math.pi)
    return p, np.ones_like(p)


def linear(x, W, bias=None, residual=None, kind="none"):
    """(out, pre)."""
    pre = _arr(x) @ _arr(W).T
    if bias is not None:
        pre = pre + _arr(bias)
    out = act(pre, kind)[0]
    return (out if residual is None else out + _arr(residual)), pre


def linear_bwd(x, W, dout, pre=None, kind="none"):
    """(dx, dW, dbias, dpre) for a given pre (ignored with "none")."""
    x, W, dout = _arr(x), _arr(W), _arr(dout)
    dpre = dout if kind == "none" else dout * act(_arr(pre), kind)[1]
    d2 = dpre.reshape(-1, W.shape[0])
    return dpre @ W, d2.T @ x.reshape(-1, W.shape[1]), d2.sum(0), dpre


def add_norm(h, weight=None, eps=1e-5):
    """y of the norm that acts on h = x + residual as it is stored."""
    h = _arr(h)
    n = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    return n if weight is None else n * _arr(weight)


def add_norm_bwd(h, dy, weight=None, dh=None, eps=1e-5):
    """(dx = dresidual, dweight)."""
    h, dy = _arr(h), _arr(dy)
    p = dy if weight is None else dy * _arr(weight)
    r = 1 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    d = r * (p - h * r * (p * h * r).mean(-1, keepdims=True))
    return d if dh is None else d + _arr(dh), (dy * h * r).reshape(-1, h.shape[-1]).sum(0)
