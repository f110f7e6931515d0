"""The bound that the gradients of the delta scan are held to on the GPU (test_gpu_delta_precision.py), on the CPU: dg and
dbeta made as the kernels make them, chunk by chunk from the states at its ends, pass it, and with one of their terms left
out, halved, zero or made from states in float16 they do not."""
import numpy as np
import pytest
import torch

from oracle import delta

import test_oracle_delta as base

CASES = [(1, 130, 2, 2, 128, 128), (1, 100, 1, 1, 256, 256), (2, 150, 4, 4, 64, 64)]
C = 64


def chunk_form(x, do, dlast, mistake=None):
    """dg by dots with the gradients of q and k from the end of each chunk, dbeta by e . r."""
    Q, K, V, a, bt, live, _ = delta._prepare(**{n: x[n] for n in ("q", "k", "v", "g", "beta", "lengths")})
    DO = np.where(live[..., None, None], do, 0.0)
    S, r = delta._forward(Q, K, V, a, bt, x["h0"])
    b, L, h, dk = Q.shape
    R = np.zeros((L + 1, *S[0].shape))  # after token t, without its own q and do
    R[L] = dlast
    e = np.zeros_like(V)
    for t in reversed(range(L)):
        m = R[t + 1] + x["scale"] * Q[:, t, :, :, None] * DO[:, t, :, None, :]
        e[:, t] = np.matmul(K[:, t, :, None, :], m)[:, :, 0]
        R[t] = a[:, t, :, None, None] * (m - K[:, t, :, :, None] * (bt[:, t, :, None] * e[:, t])[:, :, None])
    half = lambda t: t.astype(np.float16).astype(np.float64) if mistake == "float16" else t
    dg = np.zeros((b, L, h))
    for t0 in range(0, L, C):
        t1 = min(t0 + C, L)
        for i in range(b):
            for j in range(h):
                q, k, g = Q[i, t0:t1, j], K[i, t0:t1, j], np.cumsum(np.log(a[i, t0:t1, j]))
                u, f, d = (bt[i, t0:t1, j, None] * half(r[i, t0:t1, j]), bt[i, t0:t1, j, None] * half(e[i, t0:t1, j]),
                           x["scale"] * DO[i, t0:t1, j])
                S0, R1 = half(S[t0, i, j]), half(R[t1, i, j])
                D = np.tril(np.exp(g[:, None] - g[None]), -1)
                dP, dN = D * (d @ u.T), -D * (f @ u.T)
                end = np.exp(g[-1] - g)[:, None] * (u @ R1.T)
                dq = np.exp(g)[:, None] * (d @ S0.T) + dP @ k
                plus = end + dP.T @ q + dN.T @ k
                minus = -np.exp(g)[:, None] * (f @ S0.T) + dN @ k
                terms = (q * dq).sum(1) - (k * plus).sum(1) + (k * minus).sum(1)
                edge, last = np.exp(g[-1]) * (R1 * S0).sum(), (k * end).sum()
                dg[i, t0:t1, j] = np.cumsum(terms[::-1])[::-1] + (0 if mistake == "edge" else edge) + (0 if mistake == "end" else last)
    db = (e * r).sum(-1)
    if mistake in ("half", "zero", "sign"):
        dg, db = ({"half": 0.5, "zero": 0.0, "sign": -1.0}[mistake] * t for t in (dg, db))
    return dg, db


def bfloat(x):
    return torch.from_numpy(x).to(torch.bfloat16)


def ratio(got, want, spread):
    off = np.abs(bfloat(got).double().numpy() - want)
    half = np.ldexp(0.5, np.frexp(want)[1] - 8)
    return np.linalg.norm(np.maximum(off - half * (1 + 2.0 ** -20), 0)) / (2.0 ** -16 * np.linalg.norm(spread))


def inputs(case):
    b, L, h, hk, dk, dv = case
    x, do, dlast = base.make(b=b, L=L, h=h, hk=hk, dk=dk, dv=dv, seed=L)
    x["lengths"] = None
    x["g"] = 0.03 * x["g"]  # so that a chunk's end still matters at its start
    x["q"] = x["q"] / np.sqrt(dk)
    return x, do, dlast


@pytest.mark.parametrize("case", CASES, ids=str)
def test_the_chunk_form_is_the_definition(case):
    x, do, dlast = inputs(case)
    want = delta.delta_scan_bwd(**x, do=do, dlast=dlast)
    dg, db = chunk_form(x, do, dlast)
    for got, w in ((dg, want["dg"]), (db, want["dbeta"])):
        assert np.linalg.norm(got - w) <= 1e-11 * np.linalg.norm(w)


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("mistake", ["edge", "end", "half", "zero", "sign", "float16"])
def test_planted_mistakes_are_seen(case, mistake):
    x, do, dlast = inputs(case)
    want = delta.delta_scan_bwd(**x, do=do, dlast=dlast)
    spread = delta.delta_scan_spread(**x, do=do, dlast=dlast, chunk=C)
    right, wrong = chunk_form(x, do, dlast), chunk_form(x, do, dlast, mistake)
    for n, a, b in zip(("dg", "dbeta"), right, wrong):
        assert ratio(a, want[n], spread[n]) <= 2.0 ** -4
        if n == "dg" or mistake in ("half", "zero", "sign"):
            assert ratio(b, want[n], spread[n]) > 1, n
