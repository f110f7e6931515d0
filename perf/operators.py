"""Cases of the head scan, the gated group norm and the token-major linear layer: what is timed and compared.

``run`` computes a case in plain torch operations (``own`` false) or through the library's entry points (``own``
true); ``exact`` computes it in 64 bits from the definitions.  A case's ``op`` says which operator it is:

  scan    o, last state of a prompt                  S_t = e^{g_t} S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t
  train   the same and every gradient
  step    one new token for every sequence
  norm    grouped RMS / mean-variance norm of token rows with a SiLU gate; ``train`` asks for the gradients too
  linear  act(x W^T + bias) + residual on token rows; ``train`` asks for the gradients too
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a short follow-up prompt of one conversation, its state carried on: latency
        {"name": "scan_short", "op": "scan", "dtype": "bf16", "b": 1, "L": 17, "H": 4, "Hk": 4, "dk": 32, "dv": 32,
         "decay": "token", "h0": True, "ragged": False, "fused": False},
        # prompts at the 1.4B-like width (d_inner 4096) in a batch of 8, q, k and v sliced out of one projection
        {"name": "scan_1.4b", "op": "scan", "dtype": "bf16", "b": 8, "L": 2048, "H": 32, "Hk": 32, "dk": 128, "dv": 128,
         "decay": "token", "h0": False, "ragged": True, "fused": True},
        # one long document with few heads: the length is what there is to split
        {"name": "scan_long", "op": "scan", "dtype": "bf16", "b": 1, "L": 65536, "H": 16, "Hk": 16, "dk": 128, "dv": 128,
         "decay": "head", "h0": False, "ragged": False, "fused": False},
        # training at the 1.4B-like width, keys and queries shared by all heads
        {"name": "train_shared", "op": "train", "dtype": "bf16", "b": 4, "L": 2048, "H": 64, "Hk": 1, "dk": 128, "dv": 64,
         "decay": "token", "h0": False, "ragged": False, "fused": False},
        # training in float32 at the 130m-like width (24 heads of 64), a padded batch and a given start state
        {"name": "train_130m_f32", "op": "train", "dtype": "f32", "b": 4, "L": 1999, "H": 24, "Hk": 24, "dk": 64, "dv": 64,
         "decay": "token", "h0": True, "ragged": True, "fused": False},
        # a serving step of few sequences (latency) and of many (the states' traffic)
        {"name": "step_8", "op": "step", "dtype": "f32", "b": 8, "H": 24, "Hk": 24, "dk": 64, "dv": 64, "decay": "token"},
        {"name": "step_256", "op": "step", "dtype": "bf16", "b": 256, "H": 32, "Hk": 8, "dk": 128, "dv": 128,
         "decay": "head"},
        # the norm over each head after the 1.4B-like scan, and the whole-row norm of gated rows in float32 training
        {"name": "norm_1.4b", "op": "norm", "dtype": "bf16", "T": 16384, "C": 4096, "groups": 32, "center": True,
         "gate": "after", "train": False},
        {"name": "norm_130m_f32", "op": "norm", "dtype": "f32", "T": 8191, "C": 1536, "groups": 1, "center": False,
         "gate": "before", "train": True},
        # the output layer of eight sequences' new tokens, and of a training batch
        {"name": "linear_8", "op": "linear", "dtype": "bf16", "T": 8, "K": 4096, "M": 2048, "act": "none", "bias": True,
         "residual": True, "train": False},
        {"name": "linear_130m_f32", "op": "linear", "dtype": "f32", "T": 4099, "K": 768, "M": 1536, "act": "silu",
         "bias": True, "residual": False, "train": False},
        {"name": "linear_1.4b", "op": "linear", "dtype": "bf16", "T": 16384, "K": 4096, "M": 2048, "act": "gelu",
         "bias": True, "residual": True, "train": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "train", "train", "step", "norm", "linear", "linear"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("scan", "train"):
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        H = Hk * rng.choice([1, 1, 2, 4])
        dk, dv = (rng.choice([16, 32, 48, 64, 80, 100, 128, 128, 192, 256]) for _ in range(2))
        b = rng.choice([1, 1, 2, 3, 5, 8])
        most = (2 ** 33 if op == "scan" else 2 ** 31) // (b * H * max(dk * dv, 2048))
        L = max(1, min(_log(rng, 1, 32768 if op == "scan" else 4096), most))
        return {"op": op, "dtype": dtype, "b": b, "L": L, "H": H, "Hk": Hk, "dk": dk, "dv": dv,
                "decay": rng.choice(["token", "token", "head"] if op == "scan" else ["token"]),
                "h0": rng.random() < 0.5, "ragged": rng.random() < 0.5,
                "fused": op == "scan" and dk % 8 == 0 and dv % 8 == 0 and rng.random() < 0.5}
    if op == "step":
        Hk = rng.choice([1, 2, 4, 8, 16])
        H = Hk * rng.choice([1, 2, 4])
        dk, dv = (rng.choice([32, 64, 80, 128, 256]) for _ in range(2))
        return {"op": op, "dtype": dtype, "b": max(1, min(_log(rng, 1, 512), 2 ** 27 // (H * dk * dv))), "H": H, "Hk": Hk,
                "dk": dk, "dv": dv, "decay": rng.choice(["token", "head"])}
    if op == "norm":
        groups = rng.choice([1, 1, 8, 12, 24, 32])
        size = rng.choice([48, 64, 100, 128, 256]) if groups > 1 else _log(rng, 64, 8192)
        C = groups * size
        return {"op": op, "dtype": dtype, "T": max(1, min(_log(rng, 1, 32768), 2 ** 25 // C)), "C": C, "groups": groups,
                "center": rng.random() < 0.5, "gate": rng.choice(["after", "before", "none"]),
                "train": rng.random() < 0.6}
    T = _log(rng, 1, 8192)
    K, M = (rng.choice([96, 200, 512, 768, 1001, 1536, 2048, 4096]) for _ in range(2))
    return {"op": "linear", "dtype": dtype, "T": T, "K": K, "M": M, "act": rng.choice(["none", "silu", "gelu"]),
            "bias": rng.random() < 0.7, "residual": rng.random() < 0.5, "train": rng.random() < 0.4}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def rnd(*shape, by=1.0):
        return torch.randn(shape, generator=g, device=DEV) * by

    s = {"case": dict(case)}
    op = case["op"]
    if op in ("scan", "train", "step"):
        b, H, Hk, dk, dv = (case[n] for n in ("b", "H", "Hk", "dk", "dv"))
        L = 1 if op == "step" else case["L"]
        if case.get("fused"):
            # one projection's rows: q, k and v of a token next to each other, used in place
            row = rnd(b, L, 2 * Hk * dk + H * dv)
            row[..., Hk * dk:2 * Hk * dk] *= dk ** -0.5
            row = row.to(dt)
            q, k, v = row.split([Hk * dk, Hk * dk, H * dv], dim=-1)
            q, k, v = q.unflatten(-1, (Hk, dk)), k.unflatten(-1, (Hk, dk)), v.unflatten(-1, (H, dv))
        else:
            q, k, v = rnd(b, L, Hk, dk).to(dt), rnd(b, L, Hk, dk, by=dk ** -0.5).to(dt), rnd(b, L, H, dv).to(dt)
        s.update(q=q, k=k, v=v, scale=dk ** -0.5, g=None, g_head=None, h0=None, lengths=None)
        rate = torch.logspace(-2.5, 0.5, H, device=DEV)  # slow and fast heads: memories of hundreds of tokens and of one
        if case["decay"] == "token":
            s["g"] = (-rate * torch.nn.functional.softplus(rnd(b, L, H))).to(dt)
        else:
            s["g_head"] = -rate
        if op == "step":
            for n in ("q", "k", "v", "g"):
                s[n] = None if s[n] is None else s[n][:, 0].contiguous()
            s["state"] = rnd(b, H, dk, dv)
            s["state_out"] = torch.empty_like(s["state"])
            return s
        if case["h0"]:
            s["h0"] = rnd(b, H, dk, dv)
        if case["ragged"]:
            s["lengths"] = torch.randint(max(1, L // 4), L + 1, (b,), generator=g, device=DEV).to(torch.int32)
        if op == "train":
            s["do"] = rnd(b, L, H, dv).to(dt)
            s["dlast"] = rnd(b, H, dk, dv) if case["h0"] else None
        return s
    if op == "norm":
        T, C = case["T"], case["C"]
        s.update(x=(rnd(T, C) + 0.25 * rnd(T, 1)).to(dt), w=1 + rnd(C, by=0.1), eps=1e-5,
                 z=rnd(T, C).to(dt) if case["gate"] != "none" else None)
        if case["train"]:
            s["dy"] = rnd(T, C).to(dt)
        return s
    T, K, M = case["T"], case["K"], case["M"]
    s.update(x=rnd(T, K).to(dt), W=rnd(M, K, by=K ** -0.5).to(dt), bias=rnd(M, by=0.5).to(dt) if case["bias"] else None,
             residual=rnd(T, M).to(dt) if case["residual"] else None)
    if case["train"]:
        s["dout"] = rnd(T, M).to(dt)
    return s


# ------------------------------------------------------------------ plain forms, 32 bits
CHUNK = 64


def _plain_scan(q, k, v, g, g_head, h0, lengths, scale):
    """q, k, v, g float32 -> (o, last), by chunks: inside a chunk by pairs, between chunks by the chunks' states."""
    b, L, Hk, dk = q.shape
    H, dv = v.shape[2:]
    n = -(-L // CHUNK)
    at = torch.arange(n * CHUNK, device=q.device)
    live = at[None, :] < (torch.full((b,), L, device=q.device) if lengths is None else lengths)[:, None]  # [b, n C]

    def blocks(x):  # [b, L, h, d] -> [b, h, n, C, d], nothing past a row's length
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, n * CHUNK - L))
        x = torch.where(live[..., None, None], x, torch.zeros((), device=x.device, dtype=x.dtype))
        return x.unflatten(1, (n, CHUNK)).permute(0, 3, 1, 2, 4)

    of = torch.arange(H, device=q.device) // (H // Hk)
    qc, kc, vc = blocks(q)[:, of], blocks(k)[:, of], blocks(v)
    gl = g if g is not None else g_head.expand(b, L, H)
    G = blocks(gl.double()[..., None])[..., 0].cumsum(-1)  # [b, H, n, C]: positions' decays in 64 bits
    end = G[..., -1]
    tri = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    D = torch.where(tri, G[..., :, None] - G[..., None, :], -math.inf).exp().float()
    o = ((qc @ kc.transpose(-1, -2)) * D) @ vc
    U = (kc * (end[..., None] - G).exp().float()[..., None]).transpose(-1, -2) @ vc  # [b, H, n, dk, dv]
    T = torch.nn.functional.pad(end.cumsum(-1), (1, 0))  # decay up to the start of chunk c, c = 0 .. n
    low = torch.ones(n + 1, n, dtype=torch.bool, device=q.device).tril(-1)
    M = torch.where(low, T[..., :, None] - T[..., None, 1:], -math.inf).exp().float()
    S = (M @ U.flatten(-2)).unflatten(-1, (dk, dv))  # the state before chunk c; after all of them
    if h0 is not None:
        S = S + T.exp().float()[..., None, None] * h0[:, :, None]
    o = scale * (o + (qc * G.exp().float()[..., None]) @ S[:, :, :n])
    return o.permute(0, 2, 3, 1, 4).flatten(1, 2)[:, :L] * live[:, :L, None, None], S[:, :, n]


def _plain_train(s):
    names = [n for n in ("q", "k", "v", "g", "h0") if s[n] is not None]
    leaf = {n: s[n].float().requires_grad_() for n in names}
    with torch.enable_grad():
        o, last = _plain_scan(leaf["q"], leaf["k"], leaf["v"], leaf["g"], None, leaf.get("h0"), s["lengths"], s["scale"])
        outs, given = [o], [s["do"].float()]
        if s["dlast"] is not None:
            outs, given = outs + [last], given + [s["dlast"]]
        grads = torch.autograd.grad(outs, [leaf[n] for n in names], given)
    return dict({"o": o.detach().to(s["v"].dtype), "last": last.detach()},
                **{"d" + n: d.to(s[n].dtype) for n, d in zip(names, grads)})


def _plain_step(s):
    of = torch.arange(s["v"].shape[1], device=DEV) // (s["v"].shape[1] // s["q"].shape[1])
    q, k, v = s["q"].float()[:, of], s["k"].float()[:, of], s["v"].float()
    a = (s["g"].float() if s["g"] is not None else s["g_head"][None]).exp()
    S = a[..., None, None] * s["state"] + k[..., :, None] * v[..., None, :]
    o = s["scale"] * (q[..., None, :] @ S)[..., 0, :]
    return {"o": o.to(s["v"].dtype), "state": S}


def _plain_norm(x, w, z, case, eps):
    gate = None if z is None else z * torch.sigmoid(z)
    u = x * gate if case["gate"] == "before" else x
    u = u.unflatten(-1, (case["groups"], -1))
    if case["center"]:
        u = u - u.mean(-1, keepdim=True)
    y = (u * (u.square().mean(-1, keepdim=True) + eps).rsqrt()).flatten(-2) * w
    return y * gate if case["gate"] == "after" else y


def _act(p, act):
    if act == "silu":
        return p * torch.sigmoid(p)
    return 0.5 * p * (1 + torch.erf(p * math.sqrt(0.5))) if act == "gelu" else p


def _plain_linear(x, W, bias, residual, act):
    p = x @ W.t()
    p = _act(p if bias is None else p + bias, act)
    return p if residual is None else p + residual


def _plain_rows(s, names, f, given):
    """f of float32 leaves, its output and, where a gradient is given, the leaves' gradients."""
    names = [n for n in names if s[n] is not None]
    leaf = {n: s[n].float() for n in names}
    if given is None:
        return {"out": f(leaf).to(s["x"].dtype)}
    leaf = {n: t.requires_grad_() for n, t in leaf.items()}
    with torch.enable_grad():
        out = f(leaf)
        grads = torch.autograd.grad(out, list(leaf.values()), given.float())
    return dict({"out": out.detach().to(s["x"].dtype)}, **{"d" + n: d.to(s[n].dtype) for n, d in zip(names, grads)})


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    op = case["op"]
    if op == "scan":
        g = None if s["g"] is None else s["g"].float()
        o, last = _plain_scan(s["q"].float(), s["k"].float(), s["v"].float(), g, s["g_head"], s["h0"], s["lengths"],
                              s["scale"])
        return {"o": o.to(s["v"].dtype), "last": last}
    if op == "train":
        return _plain_train(s)
    if op == "step":
        return _plain_step(s)
    if op == "norm":
        return _plain_rows(s, ("x", "w", "z"), lambda t: _plain_norm(t["x"], t["w"], t.get("z"), case, s["eps"]),
                           s.get("dy"))
    return _plain_rows(s, ("x", "W", "bias"),
                       lambda t: _plain_linear(t["x"], t["W"], t.get("bias"),
                                               None if s["residual"] is None else s["residual"].float(), case["act"]),
                       s.get("dout"))


def _run_own(s):
    import selective_state_space_ssm_amd as ssm
    from selective_state_space_ssm_amd import autograd as ag

    case = s["case"]
    op = case["op"]
    if op == "scan":
        o, last = ssm.ssm_head_scan_fwd(s["q"], s["k"], s["v"], g=s["g"], g_head=s["g_head"], h0=s["h0"],
                                        lengths=s["lengths"], scale=s["scale"])
        return {"o": o, "last": last}
    if op == "step":
        o, state = ssm.ssm_head_step(s["q"], s["k"], s["v"], s["state"], g=s["g"], g_head=s["g_head"], scale=s["scale"],
                                     state_out=s["state_out"])
        return {"o": o, "state": state}
    if op == "norm" and not case["train"]:
        return {"out": ssm.ssm_gate_norm(s["x"], s["w"], s["z"], groups=case["groups"], eps=s["eps"],
                                         center=case["center"], gate_first=case["gate"] == "before")}
    if op == "linear" and not case["train"]:
        return {"out": ssm.ssm_linear(s["x"], s["W"], bias=s["bias"], residual=s["residual"], act=case["act"])}

    names = {"train": ("q", "k", "v", "g", "h0"), "norm": ("x", "w", "z"), "linear": ("x", "W", "bias")}[op]
    names = [n for n in names if s[n] is not None]
    leaf = {n: s[n].detach().requires_grad_() for n in names}
    with torch.enable_grad():
        if op == "train":
            o, last = ag.head_scan(leaf["q"], leaf["k"], leaf["v"], g=leaf["g"], h0=leaf.get("h0"), lengths=s["lengths"],
                                   scale=s["scale"])
            out = {"o": o.detach(), "last": last.detach()}
            outs, given = ([o], [s["do"]]) if s["dlast"] is None else ([o, last], [s["do"], s["dlast"]])
        elif op == "norm":
            y = ag.gate_norm(leaf["x"], leaf["w"], leaf.get("z"), groups=case["groups"], eps=s["eps"],
                             center=case["center"], gate_first=case["gate"] == "before")
            out, outs, given = {"out": y.detach()}, [y], [s["dy"]]
        else:
            y = ag.linear(leaf["x"], leaf["W"], bias=leaf.get("bias"), residual=s["residual"], act=case["act"])
            out, outs, given = {"out": y.detach()}, [y], [s["dout"]]
        grads = torch.autograd.grad(outs, list(leaf.values()), given)
    return dict(out, **{"d" + n: d for n, d in zip(names, grads)})


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    if op in ("scan", "train", "step"):
        b, H, Hk, dk, dv = (case[n] for n in ("b", "H", "Hk", "dk", "dv"))
        T = b * (1 if op == "step" else case["L"])
        rows = T * (2 * Hk * dk + 2 * H * dv) * es + (T * H * es if case["decay"] == "token" else 4 * H)
        state = 4 * b * H * dk * dv
        if op == "step":
            return {"bytes": rows + 2 * state, "flops": 4 * T * H * dk * dv}
        fwd = {"bytes": rows + state * (1 + case["h0"]), "flops": 4 * T * H * dk * dv}
        if op == "scan":
            return fwd
        # the gradients: q, k, v, g, do (and the states' gradients) in, dq, dk, dv, dg out
        more = T * (4 * Hk * dk + 3 * H * dv + 2 * H) * es + state * (3 if case["h0"] else 0)
        return {"bytes": fwd["bytes"] + more, "flops": fwd["flops"] + 10 * T * H * dk * dv}
    if op == "norm":
        n, gated = case["T"] * case["C"] * es, case["gate"] != "none"
        return {"bytes": n * (2 + gated) + (n * (3 + 2 * gated) if case["train"] else 0),
                "flops": 12 * case["T"] * case["C"] * (3 if case["train"] else 1)}
    T, K, M = case["T"], case["K"], case["M"]
    nbytes = (T * K + M * K + T * M * (2 if case["residual"] else 1)) * es
    if case["train"]:
        nbytes += (2 * T * K + 2 * M * K + T * M) * es
    return {"bytes": nbytes, "flops": 2 * T * K * M * (3 if case["train"] else 1)}


# ------------------------------------------------------------------ the definitions, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("scan", "train"):
        return _exact_scan(s, op == "train")
    d = {n: (t.double() if isinstance(t, torch.Tensor) and t.is_floating_point() else t) for n, t in s.items()}
    if op == "step":
        rep = case["H"] // case["Hk"]
        q, k = d["q"].repeat_interleave(rep, 1), d["k"].repeat_interleave(rep, 1)
        a = torch.exp(d["g"] if d["g"] is not None else d["g_head"].expand(case["b"], -1))
        S = a[:, :, None, None] * d["state"] + torch.einsum("bhi,bhj->bhij", k, d["v"])
        return {"o": d["scale"] * torch.einsum("bhi,bhij->bhj", q, S), "state": S}
    return _exact_norm(case, d) if op == "norm" else _exact_linear(case, d)


def _exact_scan(s, train):
    """The recurrence, token by token, forwards and for the gradients backwards."""
    case = s["case"]
    b, L, H, rep = case["b"], case["L"], case["H"], case["H"] // case["Hk"]
    if L * (3 if train else 1) > 70000:
        return None
    dk, dv, scale = case["dk"], case["dv"], s["scale"]
    live = torch.ones(b, L, dtype=torch.bool, device=DEV)
    if s["lengths"] is not None:
        live = torch.arange(L, device=DEV)[None] < s["lengths"][:, None]
    g = (s["g"] if s["g"] is not None else s["g_head"].expand(b, L, H)).double() * live[..., None]
    e = torch.exp(g)[..., None, None]
    put = lambda t: (t.double() * live[:, :, None, None]).repeat_interleave(rep if t.shape[2] != H else 1, 2)  # noqa: E731
    q, k, v = put(s["q"]), put(s["k"]), put(s["v"])
    h0 = torch.zeros(b, H, dk, dv, device=DEV, dtype=torch.float64) if s["h0"] is None else s["h0"].double()
    o, dq = torch.zeros_like(v), torch.zeros_like(q)
    do = put(s["do"]) if train else None
    S = h0.clone()
    for t in range(L):
        S.mul_(e[:, t]).addcmul_(k[:, t, :, :, None], v[:, t, :, None, :])
        o[:, t] = (q[:, t, :, None, :] @ S)[:, :, 0]
        if train:
            dq[:, t] = (S @ do[:, t, :, :, None])[..., 0]
    out = {"o": o.mul_(scale), "last": S}
    if not train:
        return out
    dq.mul_(scale)
    R = torch.zeros_like(S) if s["dlast"] is None else s["dlast"].double().clone()
    tail = (R * S).sum((-1, -2))  # e^{g_t} <R_t, S_{t-1}> summed up from the end
    dk_, dv_, dg = torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(g)
    for t in reversed(range(L)):
        R.addcmul_(q[:, t, :, :, None], do[:, t, :, None, :], value=scale)
        dk_[:, t] = (R @ v[:, t, :, :, None])[..., 0]
        dv_[:, t] = (k[:, t, :, None, :] @ R)[:, :, 0]
        tail = tail + (q[:, t] * dq[:, t]).sum(-1) - (k[:, t] * dk_[:, t]).sum(-1)
        dg[:, t] = tail * live[:, t, None]
        R.mul_(e[:, t])
    heads = lambda t: t.unflatten(2, (-1, rep)).sum(3)  # noqa: E731
    out.update(dq=heads(dq), dk=heads(dk_) * live[:, :, None, None], dv=dv_ * live[:, :, None, None], dg=dg)
    if s["h0"] is not None:
        out["dh0"] = R
    return out


def _exact_norm(case, d):
    T, C, G = case["T"], case["C"], case["groups"]
    x, w, z = d["x"], d["w"], d["z"]
    sg = torch.sigmoid(z) if z is not None else None
    gate = z * sg if z is not None else torch.ones_like(x)
    before, after = case["gate"] == "before", case["gate"] == "after"
    u = (x * gate if before else x).reshape(T, G, C // G)
    mu = u.mean(-1, keepdim=True) if case["center"] else torch.zeros_like(u[..., :1])
    r = 1 / torch.sqrt(((u - mu) ** 2).mean(-1, keepdim=True) + d["eps"])
    xh = (u - mu) * r
    n = xh.reshape(T, C)
    out = {"out": n * w * (gate if after else 1.0)}
    if not case["train"]:
        return out
    dn = d["dy"] * (gate if after else 1.0)
    p = (dn * w).reshape(T, G, C // G)
    du = p - xh * (p * xh).mean(-1, keepdim=True)
    if case["center"]:
        du = du - p.mean(-1, keepdim=True)
    du = (du * r).reshape(T, C)
    out.update(dx=du * gate if before else du, dw=(dn * n).sum(0))
    if z is not None:
        out["dz"] = (du * x if before else d["dy"] * n * w) * sg * (1 + z * (1 - sg))
    return out


def _exact_linear(case, d):
    p = d["x"] @ d["W"].t()
    p = p if d["bias"] is None else p + d["bias"]
    sg, cdf = torch.sigmoid(p), 0.5 * torch.erfc(-p / math.sqrt(2))
    act, slope = {"none": (p, torch.ones_like(p)), "silu": (p * sg, sg * (1 + p * (1 - sg))),
                  "gelu": (p * cdf, cdf + p * torch.exp(-p * p / 2) / math.sqrt(2 * math.pi))}[case["act"]]
    out = {"out": act if d["residual"] is None else act + d["residual"]}
    if case["train"]:
        dp = d["dout"] * slope
        out.update(dx=dp @ d["W"], dW=dp.t() @ d["x"])
        if d["bias"] is not None:
            out["dbias"] = dp.sum(0)
    return out
