"""Pins of the head scan's float64 oracle (CPU): the sum over pairs it is defined by, finite differences, and the
chunked form's identities."""
import numpy as np
import pytest

from oracle import head


def _inputs(seed, b=2, L=9, hk=2, rep=2, dk=3, dv=4):
    r = np.random.default_rng(seed)
    h = hk * rep
    return dict(q=r.standard_normal((b, L, hk, dk)), k=r.standard_normal((b, L, hk, dk)),
                v=r.standard_normal((b, L, h, dv)), g=-r.exponential(0.5, (b, L, h)),
                h0=r.standard_normal((b, h, dk, dv)), scale=0.7)


def test_forward_is_the_sum_over_pairs():
    x = _inputs(1)
    o, last = head.head_scan(**x)
    b, L, hk, dk = x["q"].shape
    h = x["v"].shape[2]
    for bi in range(b):
        for hi in range(h):
            G = np.cumsum(x["g"][bi, :, hi])
            for i in range(L):
                want = np.exp(G[i]) * x["q"][bi, i, hi // 2] @ x["h0"][bi, hi]
                for j in range(i + 1):
                    want = want + np.exp(G[i] - G[j]) * (x["q"][bi, i, hi // 2] @ x["k"][bi, j, hi // 2]) * x["v"][bi, j, hi]
                np.testing.assert_allclose(o[bi, i, hi], 0.7 * want, rtol=1e-12, atol=1e-12)
            want = np.exp(G[-1]) * x["h0"][bi, hi] + sum(
                np.exp(G[-1] - G[j]) * np.outer(x["k"][bi, j, hi // 2], x["v"][bi, j, hi]) for j in range(L))
            np.testing.assert_allclose(last[bi, hi], want, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("lengths", [None, [9, 5], [0, 1]])
def test_gradients_are_the_differences(lengths):
    x = _inputs(2)
    r = np.random.default_rng(3)
    do, dlast = r.standard_normal(x["v"].shape), r.standard_normal(x["h0"].shape)

    def loss(**kw):
        o, last = head.head_scan(**{**x, **kw}, lengths=lengths)
        return (o * do).sum() + (last * dlast).sum()

    got = head.head_scan_bwd(x["q"], x["k"], x["v"], do, x["g"], x["h0"], lengths, x["scale"], dlast)
    for n in ("q", "k", "v", "g", "h0"):
        for _ in range(12):
            at = tuple(r.integers(0, s) for s in x[n].shape)
            e = 1e-5
            up, dn = x[n].copy(), x[n].copy()
            up[at] += e
            dn[at] -= e
            want = (loss(**{n: up}) - loss(**{n: dn})) / (2 * e)
            assert abs(got["d" + n][at] - want) <= 1e-7 * max(1, abs(want)), (n, at)


def test_state_carries_a_split_sequence():
    x = _inputs(4)
    o, last = head.head_scan(**x)
    cut = lambda lo, hi: {n: (x[n][:, lo:hi] if n in "qkvg" else x[n]) for n in x}
    o1, s = head.head_scan(**cut(0, 4))
    o2, s2 = head.head_scan(**{**cut(4, 9), "h0": s})
    np.testing.assert_allclose(np.concatenate([o1, o2], 1), o, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(s2, last, rtol=1e-12, atol=1e-12)
    o3, s3 = head.head_step(x["q"][:, 0], x["k"][:, 0], x["v"][:, 0], x["h0"], x["g"][:, 0], 0.7)
    np.testing.assert_allclose(o3, o[:, 0], rtol=1e-12, atol=1e-12)


def test_minus_infinity_starts_anew():
    x = _inputs(5)
    x["g"][:, 4] = -np.inf
    o, last = head.head_scan(**x)
    fresh = {n: (x[n][:, 4:] if n in "qkvg" else x[n]) for n in x}
    fresh["g"] = fresh["g"].copy()
    fresh["g"][:, 0] = 0
    o2, s2 = head.head_scan(**{**fresh, "h0": None})
    np.testing.assert_allclose(o[:, 4:], o2, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(last, s2, rtol=1e-12, atol=1e-12)
