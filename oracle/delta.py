"""float64 oracle of the delta scan (the head scan with the gated delta rule), token by token from its definition:

    S~_t = e^{g_t} S_{t-1},  r_t = v_t - S~_t^T k_t,  S_t = S~_t + beta_t k_t r_t^T,  o_t = scale S_t^T q_t

and its gradients, every state kept.  NumPy on the CPU; shares no code with the GPU path.  q, k: [b, L, hk, dk];
v, do: [b, L, h, dv]; g, beta: [b, L, h] (or None); h0, dlast: [b, h, dk, dv].

``delta_scan_errors`` gives, next to the results, what an implementation that rounds may be off by: every step's own
rounding carried through the recurrence, whose transition (I - beta k k^T) e^g lengthens nothing while beta |k|^2 <= 2.
"""
import numpy as np

from .head import _arr


def _prepare(q, k, v, g, beta, lengths):
    q, k, v, g, beta = (_arr(t) for t in (q, k, v, g, beta))
    b, L, hk, dk = q.shape
    h, dv = v.shape[2:]
    lens = np.full(b, L) if lengths is None else np.clip(np.asarray([int(n) for n in lengths]), 0, L)
    live = np.arange(L)[None, :] < lens[:, None]
    a = np.ones((b, L, h)) if g is None else np.exp(g)
    a = np.where(live[..., None], a, 1.0)
    bt = np.where(live[..., None], 1.0 if beta is None else beta, 0.0) * np.ones((b, L, h))
    put = lambda t: np.where(live[..., None, None], t, 0.0)
    rep = h // hk
    return np.repeat(put(q), rep, 2), np.repeat(put(k), rep, 2), put(v), a, bt, live, rep


def _forward(Q, K, V, a, bt, h0):
    b, L, h, dk = Q.shape
    dv = V.shape[3]
    S = np.zeros((L + 1, b, h, dk, dv))
    r = np.zeros((b, L, h, dv))
    if h0 is not None:
        S[0] = _arr(h0)
    for t in range(L):
        s = a[:, t, :, None, None] * S[t]
        r[:, t] = V[:, t] - np.matmul(K[:, t, :, None, :], s)[:, :, 0]
        S[t + 1] = s + K[:, t, :, :, None] * (bt[:, t, :, None] * r[:, t])[:, :, None, :]
    return S, r


def delta_scan(q, k, v, g=None, beta=None, h0=None, lengths=None, scale=1.0):
    """(o, last state)."""
    Q, K, V, a, bt, live, _ = _prepare(q, k, v, g, beta, lengths)
    S, _ = _forward(Q, K, V, a, bt, h0)
    o = scale * np.matmul(Q.transpose(1, 0, 2, 3)[..., None, :], S[1:])[..., 0, :].transpose(1, 0, 2, 3)
    return o * live[..., None, None], S[-1]


def _backward(Q, K, V, DO, a, bt, S, r, scale, dlast):
    b, L, h, dk = Q.shape
    R = np.zeros((b, h, dk, V.shape[3])) if dlast is None else _arr(dlast).copy()
    dq, dkk, dvv = np.zeros_like(Q), np.zeros_like(K), np.zeros_like(V)
    dg, db, norms = np.zeros((b, L, h)), np.zeros((b, L, h)), np.zeros((b, L, h))
    for t in reversed(range(L)):
        R = R + scale * Q[:, t, :, :, None] * DO[:, t, :, None, :]
        norms[:, t] = np.sqrt((R * R).sum((-1, -2)))
        s = a[:, t, :, None, None] * S[t]
        e = np.matmul(K[:, t, :, None, :], R)[:, :, 0]
        beta = bt[:, t, :, None]
        dvv[:, t] = beta * e
        db[:, t] = (e * r[:, t]).sum(-1)
        dq[:, t] = scale * np.matmul(S[t + 1], DO[:, t, :, :, None])[..., 0]
        dkk[:, t] = beta * np.matmul(R, r[:, t, :, :, None])[..., 0] - np.matmul(s, dvv[:, t, :, :, None])[..., 0]
        R = R - K[:, t, :, :, None] * dvv[:, t, :, None, :]
        dg[:, t] = (R * s).sum((-1, -2))
        R = a[:, t, :, None, None] * R
    return dq, dkk, dvv, dg, db, R, norms


def delta_scan_bwd(q, k, v, do, g=None, beta=None, h0=None, lengths=None, scale=1.0, dlast=None):
    """dict of dq, dk (summed over the heads that share them), dv, dg, dbeta [b, L, h], dh0."""
    Q, K, V, a, bt, live, rep = _prepare(q, k, v, g, beta, lengths)
    DO = np.where(live[..., None, None], _arr(do), 0.0)
    S, r = _forward(Q, K, V, a, bt, h0)
    dq, dk, dv, dg, db, R, _ = _backward(Q, K, V, DO, a, bt, S, r, scale, dlast)
    b, L, h, _ = Q.shape
    heads = lambda x: x.reshape(b, L, h // rep, rep, -1).sum(3)
    m = live[..., None, None]
    return {"dq": heads(dq) * m, "dk": heads(dk) * m, "dv": dv * m, "dg": dg * live[..., None],
            "dbeta": db * live[..., None], "dh0": R}


def delta_step(q, k, v, state, g=None, beta=None, scale=1.0):
    """(o, new state) of one token: q, k [b, hk, dk], v [b, h, dv], g, beta [b, h] or None."""
    one = lambda t: None if t is None else _arr(t)[:, None]
    o, S = delta_scan(one(q), one(k), one(v), one(g), one(beta), state, None, scale)
    return o[:, 0], S


def delta_scan_errors(q, k, v, do=None, g=None, beta=None, h0=None, lengths=None, scale=1.0, dlast=None, step=2.0 ** -24,
                      pair=0.0, kept=0.0, chunk=64):
    """What each result may be off by before it is rounded to its own type, by the results' names: a bound on the
    2-norm over d_key or d_value of a token's vector (o, dq, dk, dv), on a number (dg, dbeta) or on the norm of a
    state (last, dh0).

    ``step``: the error of a sum relative to the product of its vectors' norms.  ``pair``: that of a product of values
    held in two parts.  ``kept``: that of the states, r and e as the gradients of q, k, v, g and beta find them (what
    goes on from token to token does not pass through them).  A token's write k r^T is off by |k| (step + pair) times what r is made of, |v| + |k| |S|; these
    errors of different tokens are independent and are decayed with the state, so their squares add up.  A token takes
    a state's error to |I - beta k k^T| = max(1, |1 - beta |k|^2|) of itself at most."""
    Q, K, V, a, bt, live, rep = _prepare(q, k, v, g, beta, lengths)
    b, L, h, _ = Q.shape
    S, r = _forward(Q, K, V, a, bt, h0)
    sign, bt = bt, np.abs(bt)
    n2 = lambda x: np.sqrt((x * x).sum(-1))
    qn, kn, vn, rn = n2(Q), n2(K), n2(V), n2(r)
    amp = np.maximum(1.0, np.abs(1.0 - sign * kn ** 2))
    Sn = np.sqrt((S * S).sum((-1, -2))).transpose(1, 0, 2)  # [b, L + 1, h]
    st, both = step, step + pair
    ES = np.zeros((b, L + 1, h))
    Er = np.zeros((b, L, h))
    for t in range(L):
        made = both * (vn[:, t] + kn[:, t] * a[:, t] * Sn[:, t])
        Er[:, t] = np.sqrt(made ** 2 + (kn[:, t] * a[:, t] * ES[:, t]) ** 2)
        ES[:, t + 1] = np.sqrt((amp[:, t] * a[:, t] * ES[:, t]) ** 2 + (bt[:, t] * kn[:, t] * made) ** 2 +
                               (st * Sn[:, t + 1]) ** 2)
    out = {"o": scale * qn * (ES[:, 1:] + both * (Sn[:, 1:] + kn * bt * rn)), "last": ES[:, -1] + st * Sn[:, -1]}
    if do is None:
        return out
    DO = np.where(live[..., None, None], _arr(do), 0.0)
    dq, dk, dv, dg, db, R, Rn = _backward(Q, K, V, DO, a, sign, S, r, scale, dlast)
    don, en = n2(DO), Rn * kn
    # R~ at a token is R there less what it passed to v
    ER = np.zeros((b, L + 1, h))
    for t in reversed(range(L)):
        made = scale * qn[:, t] * don[:, t] + bt[:, t] * kn[:, t] ** 2 * Rn[:, t]
        after = ER[:, t + 1] * (a[:, t + 1] * amp[:, t + 1] if t + 1 < L else 1.0)
        ER[:, t] = np.sqrt(after ** 2 + (both * made) ** 2 + (st * Rn[:, t]) ** 2)
    Ee = kn * (ER[:, :L] + both * Rn)
    S0, E0 = a * Sn[:, :L], a * ES[:, :L]
    out["dv"] = bt * (Ee + kept * en)
    out["dbeta"] = Ee * rn + en * Er + (both + 2 * kept) * en * rn
    both = both + 4 * kept  # two of them in a product, r and e once more after their product with beta
    eq = scale * don * (ES[:, 1:] + both * (Sn[:, 1:] + kn * bt * rn))
    ek = (bt * (ER[:, :L] * rn + Rn * Er + both * Rn * rn) + bt * (E0 * en + S0 * Ee + both * S0 * en))
    heads = lambda x: x.reshape(b, L, h // rep, rep).sum(3)
    out["dq"], out["dk"] = heads(eq), heads(ek)
    # dg: dots of q with dq and k with dk over the rest of the chunk, and <R, S> at its end
    dots = qn * eq + kn * ek + both * (qn * n2(dq) + kn * n2(dk) + 2 * kn * bt * Rn * rn)
    edge = ER[:, :L] * Sn[:, 1:] + Rn * ES[:, 1:] + both * Rn * Sn[:, 1:]
    pad = -L % chunk
    blocks = np.pad(dots ** 2, ((0, 0), (0, pad), (0, 0))).reshape(b, -1, chunk, h)
    edges = np.pad(edge, ((0, 0), (0, pad), (0, 0))).reshape(b, -1, chunk, h).max(2, keepdims=True)
    total = np.sqrt(blocks[:, :, ::-1].cumsum(2)[:, :, ::-1]) + edges
    out["dg"] = total.reshape(b, -1, h)[:, :L]
    out["dh0"] = ER[:, 0] + st * Rn[:, 0] if L else 0.0
    return out


def delta_scan_spread(q, k, v, do, g=None, beta=None, h0=None, lengths=None, scale=1.0, dlast=None, chunk=64):
    """Root of the sum of the squares of the products that each gradient's numbers are sums of: roundings of their factors
    that are independent of each other add up to so much of the roundings' size.  dq, dk: [b, L, h, d_key], of the heads by
    themselves; dv; dg, dbeta: [b, L, h].  dg as a sum over the rest of a chunk of a token's products with q and k, and
    over the chunk's end of <R, S>."""
    Q, K, V, a, bt, live, _ = _prepare(q, k, v, g, beta, lengths)
    DO = np.where(live[..., None, None], _arr(do), 0.0)
    b, L, h, _ = Q.shape
    S, r = _forward(Q, K, V, a, bt, h0)
    R = np.zeros_like(S[0]) if dlast is None else _arr(dlast).copy()
    out = {"dq": np.zeros_like(Q), "dk": np.zeros_like(K), "dv": np.zeros_like(V), "dg": np.zeros((b, L, h)),
           "dbeta": np.zeros((b, L, h))}
    over = lambda x, m: np.matmul(x[:, :, None, :] ** 2, m * m)[:, :, 0]   # sum over rows of x_i^2 m_ij^2
    along = lambda m, x: np.matmul(m * m, x[..., None] ** 2)[..., 0]       # over columns
    total = np.zeros((b, h))
    for t in reversed(range(L)):
        if t == L - 1 or t % chunk == chunk - 1:
            total = (R * R * S[t + 1] ** 2).sum((-1, -2))
        R = R + scale * Q[:, t, :, :, None] * DO[:, t, :, None, :]
        s = a[:, t, :, None, None] * S[t]
        e = np.matmul(K[:, t, :, None, :], R)[:, :, 0]
        n = bt[:, t, :, None]
        dv = n * e
        dq = scale ** 2 * along(S[t + 1], DO[:, t])
        dk = along(R, n * r[:, t]), along(s, dv)
        e2, r2 = over(K[:, t], R), V[:, t] ** 2 + over(K[:, t], s)
        out["dq"][:, t], out["dk"][:, t], out["dv"][:, t] = np.sqrt(dq), np.sqrt(dk[0] + dk[1]), n * np.sqrt(e2)
        out["dbeta"][:, t] = np.sqrt((e2 * r[:, t] ** 2 + e ** 2 * r2).sum(-1))
        total = total + (Q[:, t] ** 2 * dq + K[:, t] ** 2 * (dk[0] + dk[1])).sum(-1)
        out["dg"][:, t] = np.sqrt(total)
        R = a[:, t, :, None, None] * (R - K[:, t, :, :, None] * dv[:, :, None, :])
    return out
