"""The delta scan's float64 oracle: against the matrix form of its state, the head scan's oracle where the rule has
nothing to take out, differences for every gradient, and planted mistakes (CPU)."""
import numpy as np
import pytest

from oracle import delta, head


def make(b=2, L=7, h=4, hk=2, dk=5, dv=3, seed=0):
    r = np.random.RandomState(seed)
    k = r.randn(b, L, hk, dk)
    x = dict(q=r.randn(b, L, hk, dk), k=k / np.sqrt((k * k).sum(-1, keepdims=True)), v=r.randn(b, L, h, dv),
             g=-np.abs(r.randn(b, L, h)), beta=1 / (1 + np.exp(-r.randn(b, L, h))), h0=r.randn(b, h, dk, dv),
             lengths=[L, L - 3][:b], scale=0.4)
    return x, r.randn(b, L, h, dv), r.randn(b, h, dk, dv)


def test_state_by_matrices():
    x, _, _ = make(b=1, h=1, hk=1)
    S = x["h0"][0, 0]
    for t in range(7):
        k, a, bt = x["k"][0, t, 0], np.exp(x["g"][0, t, 0]), x["beta"][0, t, 0]
        S = a * (np.eye(5) - bt * np.outer(k, k)) @ S + bt * np.outer(k, x["v"][0, t, 0])
        o, last = delta.delta_scan(**{n: (v[:, :t + 1] if n in ("q", "k", "v", "g", "beta") else v)
                                      for n, v in dict(x, lengths=None).items()})
        np.testing.assert_allclose(last[0, 0], S, rtol=1e-12, atol=1e-13)
        np.testing.assert_allclose(o[0, t, 0], 0.4 * S.T @ x["q"][0, t, 0], rtol=1e-12, atol=1e-13)


def test_chunk_form():
    """r = x - M (beta x) with M = N (I + diag(beta) N)^-1, and its transpose for the gradients."""
    r = np.random.RandomState(3)
    C = 9
    N, beta = np.tril(r.randn(C, C), -1), r.rand(C)
    beta[4] = 0.0
    M = N @ np.linalg.inv(np.eye(C) + beta[:, None] * N)
    x = r.randn(C)
    want = np.linalg.solve(np.eye(C) + N * beta[None, :], x)
    np.testing.assert_allclose(x - M @ (beta * x), want, rtol=1e-11, atol=1e-12)
    back = np.linalg.solve(np.eye(C) + N.T * beta[None, :], x)
    np.testing.assert_allclose(x - M.T @ (beta * x), back, rtol=1e-11, atol=1e-12)


def test_orthogonal_keys_are_the_head_scan():
    """Keys that are orthogonal to each other and to the state take nothing out."""
    x, _, _ = make(b=1, L=4, h=1, hk=1, dk=5)
    x.update(k=np.eye(5)[None, :4, None], h0=None, g=None, beta=None, lengths=None)
    o, last = delta.delta_scan(**x)
    y = {n: x[n] for n in ("q", "k", "v", "h0", "lengths", "scale")}
    wo, wl = head.head_scan(**y)
    np.testing.assert_allclose(o, wo)
    np.testing.assert_allclose(last, wl)


def test_gradients_by_differences():
    x, do, dlast = make()
    want = delta.delta_scan_bwd(**x, do=do, dlast=dlast)
    r = np.random.RandomState(9)

    def loss(y):
        o, last = delta.delta_scan(**y)
        return (o * do).sum() + (last * dlast).sum()

    for n in ("q", "k", "v", "g", "beta", "h0"):
        d, eps = r.randn(*x[n].shape), 1e-6
        num = (loss(dict(x, **{n: x[n] + eps * d})) - loss(dict(x, **{n: x[n] - eps * d}))) / (2 * eps)
        got = (want["d" + n] * d).sum()
        assert abs(num - got) <= 1e-7 * max(1, abs(got)), (n, num, got)


def test_lengths_and_starts():
    x, do, dlast = make()
    o, last = delta.delta_scan(**x)
    cut = {n: (v[1:, :4] if n in ("q", "k", "v", "g", "beta") else v[1:]) for n, v in x.items() if n not in ("lengths", "scale")}
    o1, last1 = delta.delta_scan(**cut, scale=x["scale"])
    np.testing.assert_allclose(o[1, :4], o1[0])
    np.testing.assert_allclose(last[1], last1[0])
    assert not o[1, 4:].any()
    x["g"][:, 3] = -np.inf  # the state starts anew at token 3
    o, last = delta.delta_scan(**dict(x, lengths=None))
    tail = {n: v[:, 3:] for n, v in x.items() if n in ("q", "k", "v", "g", "beta")}
    o1, last1 = delta.delta_scan(**tail, scale=x["scale"])
    np.testing.assert_allclose(o[:, 3:], o1)
    np.testing.assert_allclose(last, last1)


@pytest.mark.parametrize("mistake", ["decay after", "beta twice", "no delta"])
def test_planted_mistakes_are_seen(mistake):
    x, _, _ = make()
    o, last = delta.delta_scan(**x)
    y = dict(x)
    if mistake == "decay after":
        y["g"] = np.roll(x["g"], 1, 1)
    elif mistake == "beta twice":
        y["beta"] = x["beta"] ** 2
    else:
        wo, wl = head.head_scan(x["q"], x["k"], x["v"] * x["beta"][..., None], x["g"], x["h0"], x["lengths"], x["scale"])
        assert np.abs(wo - o).max() > 0.05
        return
    bad, _ = delta.delta_scan(**y)
    bound = delta.delta_scan_errors(**x, step=6 * np.sqrt(64) * 2.0 ** -24, pair=2.0 ** -15)
    off = np.sqrt(((bad - o) ** 2).sum(-1))
    assert (off > bound["o"] + 2.0 ** -8 * np.sqrt((o * o).sum(-1))).any()
