"""float64 oracle of the head scan (one decay per head, matrix state), token by token from its definition:

    S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t

and its gradients from R_t = scale q_t do_t^T + e^{g_{t+1}} R_{t+1}.  NumPy on the CPU; shares no code with the GPU
path.  q, k: [b, L, hk, dk]; v, do: [b, L, h, dv]; g: [b, L, h] (or [h], or None); h0, dlast: [b, h, dk, dv].
"""
import numpy as np


def _arr(t):
    if t is None:
        return None
    if hasattr(t, "detach"):
        t = t.detach().double().cpu().numpy()
    return np.asarray(t, dtype=np.float64)


def _prepare(q, k, v, g, lengths):
    q, k, v, g = (_arr(t) for t in (q, k, v, g))
    b, L, hk, dk = q.shape
    h, dv = v.shape[2:]
    lens = np.full(b, L) if lengths is None else np.clip(np.asarray([int(n) for n in lengths]), 0, L)
    live = np.arange(L)[None, :] < lens[:, None]
    a = np.ones((b, L, h)) if g is None else np.exp(np.broadcast_to(g, (b, L, h)))
    a = np.where(live[..., None], a, 1.0)
    put = lambda t: np.where(live[..., None, None], t, 0.0)
    rep = h // hk
    return np.repeat(put(q), rep, 2), np.repeat(put(k), rep, 2), put(v), a, live, rep


def head_scan(q, k, v, g=None, h0=None, lengths=None, scale=1.0):
    """(o, last state)."""
    Q, K, V, a, live, _ = _prepare(q, k, v, g, lengths)
    b, L, h, dk = Q.shape
    dv = V.shape[3]
    S = np.zeros((b, h, dk, dv)) if h0 is None else _arr(h0).copy()
    o = np.zeros((b, L, h, dv))
    for t in range(L):
        S = a[:, t, :, None, None] * S + K[:, t, :, :, None] * V[:, t, :, None, :]
        o[:, t] = scale * np.matmul(Q[:, t, :, None, :], S)[:, :, 0]
    return o * live[..., None, None], S


def head_scan_bwd(q, k, v, do, g=None, h0=None, lengths=None, scale=1.0, dlast=None):
    """dict of dq, dk (summed over the heads that share them), dv, dg [b, L, h], dh0.  dg from its definition,
    e^{g_t} <R_t, S_{t-1}>, with every state kept."""
    Q, K, V, a, live, rep = _prepare(q, k, v, g, lengths)
    DO = np.where(live[..., None, None], _arr(do), 0.0)
    b, L, h, dk = Q.shape
    dv = V.shape[3]
    S = np.zeros((L + 1, b, h, dk, dv))
    if h0 is not None:
        S[0] = _arr(h0)
    for t in range(L):
        S[t + 1] = a[:, t, :, None, None] * S[t] + K[:, t, :, :, None] * V[:, t, :, None, :]
    R = np.zeros((b, h, dk, dv)) if dlast is None else _arr(dlast).copy()
    dq, dkk, dvv, dg = np.zeros_like(Q), np.zeros_like(K), np.zeros_like(V), np.zeros((b, L, h))
    for t in reversed(range(L)):
        R = R + scale * Q[:, t, :, :, None] * DO[:, t, :, None, :]
        dq[:, t] = scale * np.matmul(S[t + 1], DO[:, t, :, :, None])[..., 0]
        dkk[:, t] = np.matmul(R, V[:, t, :, :, None])[..., 0]
        dvv[:, t] = np.matmul(K[:, t, :, None, :], R)[:, :, 0]
        aR = a[:, t, :, None, None] * R
        dg[:, t] = (aR * S[t]).sum((-1, -2))
        R = aR
    heads = lambda x: x.reshape(b, L, h // rep, rep, dk).sum(3)
    m = live[..., None, None]
    return {"dq": heads(dq) * m, "dk": heads(dkk) * m, "dv": dvv * m, "dg": dg * live[..., None], "dh0": R}


def head_step(q, k, v, state, g=None, scale=1.0):
    """(o, new state) of one token: q, k [b, hk, dk], v [b, h, dv], g [b, h] (or [h], or None)."""
    g = _arr(g)
    if g is not None and g.ndim == 2:
        g = g[:, None]
    o, S = head_scan(_arr(q)[:, None], _arr(k)[:, None], _arr(v)[:, None], g, state, None, scale)
    return o[:, 0], S
