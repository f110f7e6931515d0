"""The delta scan and the norm with the residual's addition where things go wrong: rows without tokens, what is stored past
a length, decays of -inf, strides and alignments, offsets past 2^31 bytes, segments, shared heads, other streams, captured
graphs; and a layer made of them."""
import numpy as np
import pytest
import torch

import selective_state_space_ssm_amd as ssm
from oracle import delta, layer
from selective_state_space_ssm_amd import autograd as ag

from test_gpu_delta import DEV, IDS, TYPES, close, errors, f64, make

pytestmark = pytest.mark.gpu

NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dh0")


def equal(a, b):
    assert a.keys() == b.keys()
    for n in a:
        if a[n] is None:
            assert b[n] is None
        else:
            assert torch.equal(a[n], b[n]), n


def both(x, do, dlast=None):
    o, last = ssm.ssm_delta_scan_fwd(**x)
    return dict(ssm.ssm_delta_scan_bwd(do=do, dlast=dlast, **x), o=o, last=last)


def against_oracle(x, do, dlast, dtype, names=NAMES):
    r = both(x, do, dlast)
    torch.cuda.synchronize(DEV)
    y, d = f64(x), do.double().cpu().numpy()
    dl = None if dlast is None else dlast.double().cpu().numpy()
    wo, wl = delta.delta_scan(**y)
    want = delta.delta_scan_bwd(**y, do=d, dlast=dl)
    e = errors(x, dtype, do, dlast)
    close("o", r["o"], wo, e["o"])
    close("last", r["last"], wl, e["last"])
    for n in names:
        if r[n] is not None:
            close(n, r[n], want[n], e[n])
    return r


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_rows_without_tokens(dtype):
    """Lengths 0, 1, a chunk, one past it, all, and out of range (clamped): zeros past them, the state passed through."""
    L = 150
    x, do, dlast = make(7, L, 2, 2, 32, 48, dtype, seed=1)
    x["lengths"] = torch.tensor([0, 1, 64, 65, L, -5, L + 9], dtype=torch.int32, device=DEV)
    r = against_oracle(x, do, dlast, dtype)
    for i in (0, 5):
        assert torch.equal(r["last"][i], x["h0"][i]) and torch.equal(r["dh0"][i], dlast[i])
        for n in ("o", "dq", "dk", "dv", "dg", "dbeta"):
            assert float(r[n][i].abs().max()) == 0


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("dk", [16, 64, 65, 128, 136, 256])
def test_few_tokens_of_every_width(dk, dtype):
    """One chunk and two; column tiles of 64 and of 128, whole and not."""
    for L, dv in ((1, 64), (5, 72), (17, 100), (31, 128), (40, 136), (53, 256), (65, 128), (53, 192)):
        x, do, dlast = make(2, L, 2, 1, dk, dv, dtype, seed=dk + dv)
        torch.full((1 << 24,), float("nan"), device=DEV)  # what the outputs' memory may have held
        against_oracle(x, do, dlast, dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_states_are_kept_to_float32(dtype):
    """Few keys, many tokens, no decay: a token's update of the last state and of dh0 is a few float32 operations, each
    off by 2^-24 at most of the values it works on, and those of different tokens are independent: twice the square
    root of the tokens' number, with either storage type."""
    for case in ((2, 1114, 16, 16, 16, 64), (1, 2000, 2, 2, 48, 64)):
        x, do, dlast = make(*case, dtype, seed=case[1], g=False)
        r = both(x, do, dlast)
        y = f64(x)
        _, last = delta.delta_scan(**y)
        want = delta.delta_scan_bwd(**y, do=do.double().cpu().numpy(), dlast=dlast.double().cpu().numpy())
        most = 2 * 2.0 ** -24 * case[1] ** 0.5
        for got, w in ((r["last"], last), (r["dh0"], want["dh0"])):
            off = np.linalg.norm(got.double().cpu().numpy() - w) / np.linalg.norm(w)
            assert off <= most, (off, most)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("size", [(3, 140, 4, 2, 64, 64), (3, 1300, 2, 1, 32, 96)], ids=["", "segments"])
def test_what_lies_past_a_length_is_not_read(size, dtype):
    x, do, dlast = make(*size, dtype, seed=2)
    L = size[1]
    x["lengths"] = torch.tensor([0, L // 2, L - 11], dtype=torch.int32, device=DEV)
    want = both(x, do, dlast)
    past = torch.arange(L, device=DEV)[None] >= x["lengths"][:, None]
    bad = {n: x[n].clone() for n in ("q", "k", "v", "g", "beta")}
    for v in (float("nan"), float("inf"), torch.finfo(dtype).min):
        for n in bad:
            bad[n][past] = v
        do2 = do.clone()
        do2[past] = v
        equal(both(dict(x, **bad), do2, dlast), want)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_packed_sequences(dtype):
    """g = -inf at a sequence's first token: as if each had been run by itself (the first 17 with the start state)."""
    cuts = [0, 17, 18, 64, 131, 200]
    x, do, _ = make(1, 200, 2, 1, 48, 64, dtype, seed=3)
    for c in cuts[1:-1]:
        x["g"][:, c] = float("-inf")
    r = both(x, do)
    assert all(bool(torch.isfinite(t).all()) for t in r.values())
    for lo, hi in zip(cuts[:-1], cuts[1:]):
        y = dict(x, **{n: x[n][:, lo:hi].contiguous() for n in ("q", "k", "v", "g", "beta")}, h0=x["h0"] if lo == 0 else None)
        if lo:
            y["g"][:, 0] = 0
        d = do[:, lo:hi].contiguous()
        e = errors(y, dtype, d)
        wo, wl = delta.delta_scan(**f64(y))
        want = delta.delta_scan_bwd(**f64(y), do=d.double().cpu().numpy())
        close("o", r["o"][:, lo:hi], wo, e["o"])
        for n in ("dq", "dk", "dv", "dbeta"):
            close(n, r[n][:, lo:hi], want[n], e[n])
        if lo:
            assert float(r["dg"][:, lo].abs().max()) == 0
            close("dg", r["dg"][:, lo + 1:hi], want["dg"][:, 1:], e["dg"][:, 1:])
    close("last", r["last"], wl, e["last"])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_strong_and_absent_decay(dtype):
    """Heads that forget within a token, one that never forgets, one that restarts at every token."""
    x, do, dlast = make(1, 160, 4, 4, 32, 32, dtype, seed=4)
    x["g"][..., 0] = -30.0
    x["g"][..., 1] = 0.0
    x["g"][..., 2] = float("-inf")
    x["g"][:, ::2, 3] = -88.0
    x["beta"][..., 1] = 1.0
    against_oracle(x, do, dlast, dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_keys_that_are_alike(dtype):
    """One key for all tokens and beta 1: every token replaces the value (the powers of N beta pass 1e18 in a chunk of 64,
    what the products hold does not)."""
    x, do, dlast = make(1, 130, 2, 1, 32, 48, dtype, seed=6)
    x["k"][:] = 0
    x["k"][..., 3] = 1
    x["beta"][:] = 1
    x["g"][:] = 0
    r = against_oracle(x, do, dlast, dtype)
    got = r["last"][:, :, 3]
    want = x["v"][:, -1].float()
    assert float((got - want).abs().max()) <= 2.0 ** -20 * float(want.abs().max())


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_no_beta_and_no_decay_are_ones_and_zeros(dtype):
    x, do, dlast = make(2, 100, 2, 2, 64, 64, dtype, seed=7, g=False, beta=False)
    want = both(x, do, dlast)
    ones, zeros = torch.ones(2, 100, 2, dtype=dtype, device=DEV), torch.zeros(2, 100, 2, dtype=dtype, device=DEV)
    got = both(dict(x, beta=ones, g=zeros), do, dlast)
    for n in ("o", "last", "dq", "dk", "dv", "dh0"):
        assert torch.equal(got[n], want[n]), n
    assert want["dg"] is None and want["dbeta"] is None and got["dg"] is not None and got["dbeta"] is not None
    r = ssm.ssm_delta_scan_bwd(do=do, want_dg=False, want_dbeta=False, want_dh0=False, **dict(x, beta=ones, g=zeros))
    assert r["dg"] is None and r["dbeta"] is None and r["dh0"] is None


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("case", [(1, 4000, 1, 1, 32, 32), (2, 1600, 3, 1, 80, 48), (1, 2500, 2, 2, 256, 136), (1, 2000, 1, 1, 129, 256)],
                         ids=lambda c: "x".join(map(str, c)))
def test_segments(case, dtype):
    """Long rows of few heads: cut into segments whose states and transitions are carried."""
    x, do, dlast = make(*case, dtype, seed=case[1], ragged=case[0] > 1)
    against_oracle(x, do, dlast, dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_shared_heads_summed_in_a_workgroup(dtype):
    """Enough chunks and heads that a workgroup adds up all heads of a key head, and some of them."""
    for case in ((4, 2048 if dtype == torch.bfloat16 else 1024, 16, 4, 16, 16), (2, 700, 48, 4, 32, 16)):
        x, do, dlast = make(*case, dtype, seed=case[1])
        against_oracle(x, do, dlast, dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_large_and_small_values(dtype):
    """Values and gradients far from one: what the walks keep is scaled."""
    for by, dby in ((1e15, 1e-12), (1e-15, 1e10)):
        x, do, dlast = make(1, 200, 2, 2, 64, 64, dtype, seed=9)
        want = both(x, do, dlast)
        x["v"], x["h0"] = (x["v"].float() * by).to(dtype), x["h0"] * by
        do, dlast = (do.float() * dby).to(dtype), dlast * dby
        against_oracle(x, do, dlast, dtype)
        assert want["o"].isfinite().all()


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("b", [2, 33, 64, 65])
def test_many_ragged_rows(b, dtype):
    """Rows in the order of their lengths, equal ones among them; more rows than a wavefront has lanes."""
    x, do, dlast = make(b, 100, 5, 5, 16, 16, dtype, seed=b)
    r = torch.Generator().manual_seed(b)
    x["lengths"] = torch.randint(0, 8, (b,), generator=r).mul(15).to(torch.int32).to(DEV)
    against_oracle(x, do, dlast, dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("by", [2.0 ** -6, 2.0 ** 6], ids=["small", "large"])
@pytest.mark.parametrize("case", [(2, 150, 4, 2, 64, 64), (1, 1500, 2, 1, 128, 40)], ids=["", "segments"])
def test_keys_and_beta_far_from_one(case, by, dtype):
    """Keys of any length while beta |k|^2 stays below 2: beta past 1000 and below 2^-12, of either sign; queries too."""
    x, do, dlast = make(*case, dtype, seed=13)
    x["k"], x["q"] = x["k"] * by, x["q"] * by ** -3
    x["beta"] = x["beta"] * by ** -2
    x["beta"][:, 3::7] *= -0.25
    against_oracle(x, do, dlast, dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_views_give_the_bits_of_copies(dtype):
    b, L, h, d = 3, 70, 2, 64
    r = torch.Generator().manual_seed(5)
    big = (0.1 * torch.randn(b, L + 3, 5 * h * d + 8, generator=r)).to(dtype).to(DEV)
    cut = lambda off: big[:, 2:L + 2, off:off + h * d].unflatten(-1, (h, d))
    beta = torch.rand(b, L, h, generator=r).to(dtype).to(DEV)
    for by in (0, 1):  # one element on: no vector is aligned
        q, k, v = cut(by), cut(2 * h * d + by), cut(4 * h * d + by)
        want = ssm.ssm_delta_scan_fwd(*(t.contiguous() for t in (q, k, v)), beta)
        got = ssm.ssm_delta_scan_fwd(q, k, v, beta)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        one = ssm.ssm_delta_scan_fwd(q[:, :1], k[:, :1], v[:, :1], beta[:, :1].contiguous())
        same = ssm.ssm_delta_scan_fwd(*(t[:, :1].contiguous() for t in (q, k, v)), beta[:, :1].contiguous())
        assert torch.equal(one[0], same[0]) and torch.equal(one[1], same[1])
    with pytest.raises(ssm.SSMError):
        ssm.ssm_delta_scan_fwd(q[:1].expand(3, -1, -1, -1), k, v, beta)
    with pytest.raises(ValueError):
        ssm.ssm_delta_scan_fwd(q, k, v, beta.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(TypeError):
        ssm.ssm_delta_scan_fwd(q, k, v, beta.double())


def test_offsets_past_32_bits():
    """v and o of over 2^31 bytes: the tail of the long run and its middle against runs from the states before them."""
    b, L, h, dv = 1, 72 * 1024, 64, 256   # 1.2e9 values, 2.4 GB each
    r = torch.Generator(device=DEV).manual_seed(6)
    q = torch.nn.functional.normalize(torch.randn(b, L, 1, 32, generator=r, device=DEV), dim=-1).bfloat16()
    v = torch.randn(b, L, h, dv, generator=r, device=DEV, dtype=torch.bfloat16)
    g = (-torch.logspace(-2, 0, h, device=DEV)).bfloat16().expand(b, L, h).contiguous()
    beta = torch.rand(b, L, h, generator=r, device=DEV).bfloat16()
    o, last = ssm.ssm_delta_scan_fwd(q, q, v, beta, g=g)
    cut = lambda t, lo, hi: t[:, lo:hi] if t.dim() == 4 else t[:, lo:hi].contiguous()
    mid = 2 ** 31 // (h * dv * 2) // 64 * 64 + 640
    for at, to in ((mid, mid + 64), (L - 192, L)):
        _, state = ssm.ssm_delta_scan_fwd(*(cut(t, 0, at) for t in (q, q, v, beta)), g=cut(g, 0, at))
        o2, last2 = ssm.ssm_delta_scan_fwd(*(cut(t, at, to) for t in (q, q, v, beta)), g=cut(g, at, to), h0=state)
        assert float((o[:, at:to].float() - o2.float()).abs().max()) <= 2 ** -7 * float(o2.float().abs().max())
    assert float((last - last2).norm() / last2.norm()) <= 1e-5


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_repeated_calls_give_the_same_bits(dtype):
    for size in ((2, 1100, 4, 1, 64, 64), (4, 1024, 16, 4, 16, 32)):
        x, do, dlast = make(*size, dtype, seed=7)
        want = both(x, do, dlast)
        for _ in range(3):
            equal(both(x, do, dlast), want)


def test_outputs_given():
    x, do, _ = make(2, 70, 2, 2, 32, 32, torch.bfloat16, seed=8)
    want = ssm.ssm_delta_scan_fwd(**x)
    o, last = torch.full_like(want[0], 7), torch.full_like(want[1], 7)
    got = ssm.ssm_delta_scan_fwd(**x, o=o, last_state=last)
    assert got[0] is o and got[1] is last and torch.equal(o, want[0]) and torch.equal(last, want[1])
    assert ssm.ssm_delta_scan_fwd(**x, return_last_state=False)[1] is None


# ------------------------------------------------------------------ a layer made of them
def _inputs(dtype, seed, b=2, L=300, h=4, hk=2, dk=32, dv=48, m=96):
    r = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=r)
    n = 2 * hk * dk + h * dv
    t = {"x": rnd(b, L, m), "W": rnd(n, m) * m ** -0.5, "Wg": rnd(2 * h, m) * m ** -0.5, "Wo": rnd(m, h * dv) * (h * dv) ** -0.5}
    t = {k: v.to(dtype).to(DEV) for k, v in t.items()}
    t.update(res=rnd(b, L, m).to(DEV), w=(1 + 0.1 * rnd(m)).to(DEV), wn=(1 + 0.1 * rnd(h * dv)).to(DEV),
             wk=torch.full((hk * dk,), dk ** -0.5, device=DEV))
    return t, (h, hk, dk, dv)


def _layer(t, sizes):
    """norm of x + residual, projections, keys and queries to unit length, delta scan, norm, projection."""
    h, hk, dk, dv = sizes
    y, res = ag.add_norm(t["x"], t["res"], t["w"])
    q, k, v = ag.linear(y, t["W"]).split([hk * dk, hk * dk, h * dv], -1)
    q, k = (ag.gate_norm(s.contiguous(), t["wk"], groups=hk, eps=1e-6) for s in (q, k))
    a, c = ag.linear(y, t["Wg"]).split([h, h], -1)
    g, beta = -torch.nn.functional.softplus(a), torch.sigmoid(c)
    o, last = ag.delta_scan(q.unflatten(-1, (hk, dk)), k.unflatten(-1, (hk, dk)), v.unflatten(-1, (h, dv)), beta.contiguous(),
                            g=g.contiguous())
    out = ag.linear(ag.gate_norm(o.flatten(2), t["wn"], groups=h), t["Wo"])
    return (*ag.add_norm(out, res, t["w"]), last)


def _plain_layer(t, sizes):
    """The same in float64 on the host."""
    h, hk, dk, dv = sizes
    rms = lambda x, eps: x * (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    res = t["x"] + t["res"]
    y = rms(res, 1e-5) * t["w"]
    q, k, v = (y @ t["W"].t()).split([hk * dk, hk * dk, h * dv], -1)
    q, k = (rms(s.unflatten(-1, (hk, dk)), 1e-6) * dk ** -0.5 for s in (q, k))
    a, c = (y @ t["Wg"].t()).split([h, h], -1)
    g, beta = -torch.nn.functional.softplus(a), torch.sigmoid(c)
    q, k = (s.repeat_interleave(h // hk, 2) for s in (q, k))
    v = v.unflatten(-1, (h, dv))
    S = torch.zeros(v.shape[0], h, dk, dv, dtype=torch.float64)
    o = []
    for i in range(v.shape[1]):
        S = g[:, i].exp()[..., None, None] * S
        u = beta[:, i, :, None] * (v[:, i] - (k[:, i, :, None] @ S)[:, :, 0])
        S = S + k[:, i, :, :, None] * u[:, :, None]
        o.append(dk ** -0.5 * (q[:, i, :, None] @ S)[:, :, 0])
    o = (rms(torch.stack(o, 1), 1e-5).flatten(2) * t["wn"]) @ t["Wo"].t()
    res = o + res
    return rms(res, 1e-5) * t["w"], res, S


def test_a_layer_and_its_gradients():
    """float32, every weight's and input's gradient against float64: a chain of products, each off by some 1e-6 of its
    norm, far below the 1e-4 asked of the whole."""
    t, sizes = _inputs(torch.float32, 1, L=70)
    a = {n: v.clone().requires_grad_() for n, v in t.items() if n != "wk"}
    a["wk"] = t["wk"]
    b = {n: v.double().cpu().requires_grad_() for n, v in t.items() if n != "wk"}
    got, want = _layer(a, sizes), _plain_layer(b, sizes)
    r = torch.Generator().manual_seed(2)
    w = [torch.randn(s.shape, generator=r) for s in got]
    sum((s * u.to(DEV)).sum() for s, u in zip(got, w)).backward()
    sum((s * u.double()).sum() for s, u in zip(want, w)).backward()
    near = lambda x, y: float((x.double().cpu() - y).norm() / y.norm())
    assert all(near(x.detach(), y.detach()) <= 1e-4 for x, y in zip(got, want))
    for n in b:
        assert near(a[n].grad, b[n].grad) <= 1e-4, n


def _serve(t, sizes):
    """The same without gradients, with the norm in 8 bits and a step behind the prompt."""
    h, hk, dk, dv = sizes
    y, res = ssm.ssm_add_norm(t["x"], t["res"], t["w"])
    y8, scale, _ = ssm.ssm_add_norm_e4m3(t["x"], t["res"], t["w"], group=32)
    row = ssm.ssm_linear(y, t["W"])
    q, k, v = row.split([hk * dk, hk * dk, h * dv], -1)
    k = ssm.ssm_gate_norm(k.contiguous(), t["wk"], groups=hk, eps=1e-6).unflatten(-1, (hk, dk))
    q, v = q.unflatten(-1, (hk, dk)), v.unflatten(-1, (h, dv))
    beta = torch.sigmoid(ssm.ssm_linear(y, t["Wg"])[..., :h]).contiguous()
    o, last = ssm.ssm_delta_scan_fwd(q, k, v, beta)
    d = ssm.ssm_delta_scan_bwd(q, k, v, v.contiguous(), beta)
    s, state = ssm.ssm_delta_step(*(z[:, 0].contiguous() for z in (q, k, v, beta)), last, state_out=torch.empty_like(last))
    n = ssm.ssm_add_norm_bwd(res, y, t["w"], res)
    return dict({m: z for m, z in d.items() if z is not None}, y=y, res=res, y8=y8.view(torch.uint8), scale=scale, o=o, last=last,
                s=s, state=state, dx=n[0], dres=n[1], dw=n[2])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_captured_graphs(dtype):
    """Two captured chains of every call, replayed in turn several times with eager work between: each replay is the
    eager bits (their workspaces are their own)."""
    sets = [_inputs(dtype, s, b=1 + s % 2, L=1500 if s % 2 else 300) for s in (11, 12)]
    graphs, outs = [], []
    for t, sizes in sets:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            _serve(t, sizes)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize(DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_serve(t, sizes))
        graphs.append(g)
    for r in range(3):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize(DEV)
        for (t, sizes), got in zip(sets, outs):
            equal(got, _serve(t, sizes))
        for t, _ in sets:  # the next round's inputs, in place
            t["x"].mul_(0.75)
            t["res"].mul_(-1)
        torch.cuda.synchronize(DEV)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_two_streams(dtype):
    t, sizes = _inputs(dtype, 5, L=1500)
    want = _serve(t, sizes)
    torch.cuda.synchronize(DEV)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got += [_serve(t, sizes) for _ in range(3)]
    torch.cuda.synchronize(DEV)
    for r in got:
        equal(r, want)


def test_gradients_are_not_differentiated_again():
    x, do, _ = make(1, 20, 1, 1, 16, 16, torch.float32, seed=1)
    q = x["q"].clone().requires_grad_()
    (d,) = torch.autograd.grad(ag.delta_scan(q, x["k"], x["v"], x["beta"], g=x["g"])[0].sum(), q, create_graph=True)
    with pytest.raises(RuntimeError):
        d.sum().backward()


def test_gradients_of_any_layout():
    """Incoming gradients that are expanded, transposed or unaligned are taken."""
    x, do, dlast = make(2, 33, 2, 2, 16, 24, torch.float32, seed=2)
    leaf = {n: x[n].clone().requires_grad_() for n in ("q", "k", "v", "g", "beta")}
    o, last = ag.delta_scan(leaf["q"], leaf["k"], leaf["v"], leaf["beta"], g=leaf["g"])
    a = torch.autograd.grad([o, last], list(leaf.values()), [torch.ones(1, 1, 1, 1, device=DEV).expand_as(o), dlast.mT.contiguous().mT],
                            retain_graph=True)
    b = torch.autograd.grad([o, last], list(leaf.values()), [torch.ones_like(o), dlast])
    for u, v in zip(a, b):
        assert torch.equal(u, v)
    w = torch.randn(2 * 33 * 96 + 1, device=DEV)[1:].view(2, 33, 96)
    r, z = torch.randn(2, 33, 96, device=DEV, requires_grad=True), torch.randn(2, 33, 96, device=DEV, requires_grad=True)
    y, h = ag.add_norm(r, z)
    c = torch.autograd.grad([y, h], [r, z], [w, w], retain_graph=True)
    d = torch.autograd.grad([y, h], [r, z], [w.clone(), w.clone()])
    assert all(torch.equal(u, v) for u, v in zip(c, d))


def test_a_gradient_shared_by_two_leaves_is_not_shared_memory():
    """x and a residual of its dtype have one gradient; what is done to one leaf's does not reach the other's."""
    x, r = (torch.randn(3, 5, 64, device=DEV, requires_grad=True) for _ in range(2))
    y, h = ag.add_norm(x, r)
    (y.sum() + h.square().sum()).backward()
    assert torch.equal(x.grad, r.grad)
    kept = r.grad.clone()
    x.grad.zero_()
    assert torch.equal(r.grad, kept)


def test_a_captured_training_step():
    """Forward and backward of the layer captured, replayed with other inputs between eager steps on other leaves."""
    t, sizes = _inputs(torch.bfloat16, 21, L=200)
    leaves = {n: v.clone().requires_grad_() for n, v in t.items() if n != "wk"}
    leaves["wk"] = t["wk"]
    names = [n for n in leaves if n != "wk"]

    def step(a):
        out = _layer(a, sizes)
        return torch.autograd.grad([s.float().square().sum() for s in out], [a[n] for n in names])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(leaves)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize(DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(leaves)
    for i in range(3):
        with torch.no_grad():
            leaves["x"].mul_(0.5)
            leaves["W"].mul_(-1)
        graph.replay()
        torch.cuda.synchronize(DEV)
        want = step({n: v.detach().clone().requires_grad_(n != "wk") for n, v in leaves.items()})
        for n, a, b in zip(names, got, want):
            assert float((a.float() - b.float()).norm()) <= 2.0 ** -7 * float(b.float().norm()), (i, n)
