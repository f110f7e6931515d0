"""The head scan, norm and linear layer where things go wrong: rows without tokens, what is stored past a length,
decays of -inf, strides and alignments, offsets past 2^31 bytes, other streams, captured graphs."""
import numpy as np
import pytest
import torch

import selective_state_space_ssm_amd as ssm
from oracle import head
from selective_state_space_ssm_amd import autograd as ag

from test_gpu_head import TYPES, IDS, DEV, adds, bounds, close, make, oracle_args

pytestmark = pytest.mark.gpu


def equal(a, b):
    assert a.keys() == b.keys()
    for n in a:
        if a[n] is None:
            assert b[n] is None
        else:
            assert torch.equal(a[n], b[n]), n


def both(x, do, dlast):
    o, last = ssm.ssm_head_scan_fwd(**x)
    return dict(ssm.ssm_head_scan_bwd(do=do, dlast=dlast, **x), o=o, last=last)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_rows_without_tokens(dtype):
    """Lengths 0, 1, a chunk, one past it, all, and out of range (clamped): zeros past them, the state passed through."""
    L = 150
    x, do, dlast = make(7, L, 2, 2, 32, 48, dtype, seed=1)
    x["lengths"] = torch.tensor([0, 1, 64, 65, L, -5, L + 9], dtype=torch.int32, device=DEV)
    r = both(x, do, dlast)
    torch.cuda.synchronize(DEV)
    want = head.head_scan_bwd(do=do.double().cpu().numpy(), dlast=dlast.double().cpu().numpy(), **oracle_args(x))
    B = head.head_scan_bwd(do=do.abs().double().cpu().numpy(), dlast=dlast.abs().double().cpu().numpy(), **oracle_args(x, True))
    wo, wl = head.head_scan(**oracle_args(x))
    bo, bl = head.head_scan(**oracle_args(x, True))
    close("o", r["o"], wo, bounds(x, wo, bo, dtype))
    close("last", r["last"], wl, bounds(x, wl, bl, torch.float32))
    for n in ("dq", "dk", "dv"):
        close(n, r[n], want[n], bounds(x, want[n], B[n], dtype))
    close("dh0", r["dh0"], want["dh0"], bounds(x, want["dh0"], B["dh0"], torch.float32))
    for i in (0, 5):
        assert torch.equal(r["last"][i], x["h0"][i]) and torch.equal(r["dh0"][i], dlast[i])
        for n in ("o", "dq", "dk", "dv", "dg"):
            assert float(r[n][i].abs().max()) == 0


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_what_lies_past_a_length_is_not_read(dtype):
    x, do, dlast = make(3, 140, 4, 2, 64, 64, dtype, seed=2)
    x["lengths"] = torch.tensor([0, 70, 129], dtype=torch.int32, device=DEV)
    want = both(x, do, dlast)
    past = torch.arange(140, device=DEV)[None] >= x["lengths"][:, None]
    bad = {n: x[n].clone() for n in ("q", "k", "v", "g")}
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
    o, last = ssm.ssm_head_scan_fwd(**x)
    r = ssm.ssm_head_scan_bwd(do=do, **x)
    assert all(bool(torch.isfinite(t).all()) for t in (o, last, *r.values()))
    for lo, hi in zip(cuts[:-1], cuts[1:]):
        y = dict(x, **{n: x[n][:, lo:hi].contiguous() for n in ("q", "k", "v", "g")}, h0=x["h0"] if lo == 0 else None)
        if lo:
            y["g"][:, 0] = 0
        wo, wl = head.head_scan(**oracle_args(y))
        bo, bl = head.head_scan(**oracle_args(y, True))
        close("o", o[:, lo:hi], wo, bounds(x, wo, bo, dtype))
        d = do[:, lo:hi].double().cpu().numpy()
        want = head.head_scan_bwd(do=d, **oracle_args(y))
        B = head.head_scan_bwd(do=np.abs(d), **oracle_args(y, True))
        for n in ("dq", "dk", "dv"):
            close(n, r[n][:, lo:hi], want[n], bounds(x, want[n], B[n], dtype))
        if lo:
            assert float(r["dg"][:, lo].abs().max()) == 0
    close("last", last, wl, bounds(x, wl, bl, torch.float32))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_strong_and_absent_decay(dtype):
    """Heads that forget within a token (their running decay leaves float32's range inside a chunk), one that never
    forgets, one that restarts at every token: against the recurrence."""
    x, do, dlast = make(1, 160, 4, 4, 32, 32, dtype, seed=4)
    x["g"][..., 0] = -30.0
    x["g"][..., 1] = 0.0
    x["g"][..., 2] = float("-inf")
    x["g"][:, ::2, 3] = -88.0
    r = both(x, do, dlast)
    wo, wl = head.head_scan(**oracle_args(x))
    bo, bl = head.head_scan(**oracle_args(x, True))
    close("o", r["o"], wo, bounds(x, wo, bo, dtype))
    close("last", r["last"], wl, bounds(x, wl, bl, torch.float32))
    d = do.double().cpu().numpy()
    want = head.head_scan_bwd(do=d, dlast=dlast.double().cpu().numpy(), **oracle_args(x))
    B = head.head_scan_bwd(do=np.abs(d), dlast=dlast.abs().double().cpu().numpy(), **oracle_args(x, True))
    for n in ("dq", "dk", "dv"):
        close(n, r[n], want[n], bounds(x, want[n], B[n], dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_views_give_the_bits_of_copies(dtype):
    """Token and batch strides, a batch row used twice (stride 0 is refused), one token, an unaligned start."""
    b, L, h, d = 3, 70, 2, 64
    r = torch.Generator().manual_seed(5)
    big = torch.randn(b, L + 3, 5 * h * d + 8, generator=r).to(dtype).to(DEV)
    cut = lambda off: big[:, 2:L + 2, off:off + h * d].unflatten(-1, (h, d))
    q, k, v = cut(0), cut(2 * h * d), cut(4 * h * d)
    kw = dict(g_head=torch.tensor([-0.1, -1.0], device=DEV))
    want = ssm.ssm_head_scan_fwd(q.contiguous(), k.contiguous(), v.contiguous(), **kw)
    got = ssm.ssm_head_scan_fwd(q, k, v, **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    one = ssm.ssm_head_scan_fwd(q[:, :1], k[:, :1], v[:, :1], **kw)
    same = ssm.ssm_head_scan_fwd(*(t[:, :1].contiguous() for t in (q, k, v)), **kw)
    assert torch.equal(one[0], same[0]) and torch.equal(one[1], same[1])
    # one element on: no vector is aligned; the same sums in the same order
    q1, k1, v1 = cut(1), cut(2 * h * d + 1), cut(4 * h * d + 1)
    want = ssm.ssm_head_scan_fwd(q1.contiguous(), k1.contiguous(), v1.contiguous(), **kw)
    got = ssm.ssm_head_scan_fwd(q1, k1, v1, **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(ssm.SSMError):
        ssm.ssm_head_scan_fwd(q[:1].expand(3, -1, -1, -1), k, v, **kw)
    with pytest.raises(ValueError):
        ssm.ssm_head_scan_fwd(q.transpose(2, 3).contiguous().transpose(2, 3), k, v, **kw)


def test_offsets_past_32_bits():
    """v and o of over 2^31 bytes and 2^31 elements past a batch row: the tail of the long run is the bits of a run over
    the tail alone from the state before it."""
    b, L, h, dv = 1, 72 * 1024, 64, 256   # 1.2e9 values, 2.4 GB each
    r = torch.Generator(device=DEV).manual_seed(6)
    q = torch.randn(b, L, 1, 32, generator=r, device=DEV).bfloat16()
    v = torch.randn(b, L, h, dv, generator=r, device=DEV, dtype=torch.bfloat16)
    gh = -torch.logspace(-2, 0, h, device=DEV)
    o, last = ssm.ssm_head_scan_fwd(q, q, v, g_head=gh)
    at = L - 192
    _, state = ssm.ssm_head_scan_fwd(q[:, :at], q[:, :at], v[:, :at], g_head=gh, o=torch.empty_like(v[:, :at]))
    o2, last2 = ssm.ssm_head_scan_fwd(q[:, at:], q[:, at:], v[:, at:], g_head=gh, h0=state)
    torch.cuda.synchronize(DEV)
    # the splits into segments differ: equal up to float32 sums, then one rounding
    assert float((o[:, at:].float() - o2.float()).abs().max()) <= 2 ** -7 * float(o2.float().abs().max())
    assert float((last - last2).norm() / last2.norm()) <= 1e-5
    # the middle, past 2^31 bytes from the start
    mid = 2 ** 31 // (h * dv * 2) + 640
    mid -= mid % 64
    _, state = ssm.ssm_head_scan_fwd(q[:, :mid], q[:, :mid], v[:, :mid], g_head=gh, o=torch.empty_like(v[:, :mid]))
    o3, _ = ssm.ssm_head_scan_fwd(q[:, mid:mid + 64], q[:, mid:mid + 64], v[:, mid:mid + 64], g_head=gh, h0=state)
    assert float((o[:, mid:mid + 64].float() - o3.float()).abs().max()) <= 2 ** -7 * float(o3.float().abs().max())


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_repeated_calls_give_the_same_bits(dtype):
    x, do, dlast = make(2, 1100, 4, 1, 64, 64, dtype, seed=7)
    want = both(x, do, dlast)
    for _ in range(3):
        equal(both(x, do, dlast), want)


def _chain(t, dout):
    """Every new entry point once, forwards and backwards."""
    o, last = ssm.ssm_head_scan_fwd(t["q"], t["k"], t["v"], g=t["g"])
    rows = o.flatten(2)
    y = ssm.ssm_gate_norm(rows, t["w"], t["z"], groups=2, center=True)
    out, pre = ssm.ssm_linear(y, t["W"], t["b"], t["r"], "gelu", return_pre=True)
    dy, dW, db = ssm.ssm_linear_bwd(y, t["W"], dout, pre, "gelu")
    dx, dw, dz = ssm.ssm_gate_norm_bwd(rows, dy, t["w"], t["z"], groups=2, center=True)
    h = ssm.ssm_head_scan_bwd(t["q"], t["k"], t["v"], dx.view(o.shape), g=t["g"])
    so, state = ssm.ssm_head_step(t["q"][:, 0].contiguous(), t["k"][:, 0].contiguous(), t["v"][:, 0].contiguous(), last,
                                  g=t["g"][:, 0].contiguous(), state_out=torch.empty_like(last))
    few = ssm.ssm_linear(y[:, 0].contiguous(), t["W"], t["b"], None, "silu")
    return dict(h, o=o, last=last, y=y, out=out, pre=pre, dy=dy, dW=dW, db=db, dx=dx, dw=dw, dz=dz, so=so, state=state, few=few)


def _chain_inputs(dtype, seed, b=2, L=1300, hk=1, h=2, dk=48, dv=64, m=96):
    r = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=r)
    t = {"q": rnd(b, L, hk, dk), "k": rnd(b, L, hk, dk), "v": rnd(b, L, h, dv), "g": -rnd(b, L, h).abs(), "z": rnd(b, L, h * dv),
         "W": rnd(m, h * dv) * 0.1, "b": rnd(m), "r": rnd(b, L, m)}
    t = {n: v.to(dtype).to(DEV) for n, v in t.items()}
    t["w"] = rnd(h * dv).to(DEV)
    return t, rnd(b, L, m).to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_captured_graphs(dtype):
    """Two captured chains of every call, replayed in turn several times with eager work between: each replay is the
    eager bits (their workspaces are their own)."""
    sets = [_chain_inputs(dtype, s) for s in (11, 12)]
    graphs, outs = [], []
    for t, d in sets:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            _chain(t, d)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize(DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_chain(t, d))
        graphs.append(g)
    for r in range(3):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize(DEV)
        for (t, d), got in zip(sets, outs):
            equal(got, _chain(t, d))
        for t, d in sets:  # the next round's inputs, in place
            for n in ("q", "v", "z"):
                t[n].mul_(0.75)
            t["g"].mul_(0.9)
            d.mul_(-1)
        torch.cuda.synchronize(DEV)


def test_another_stream():
    """On a side stream behind slow work that makes the inputs, at the same time as the same call on the first one."""
    t, d = _chain_inputs(torch.bfloat16, 13)
    t2, d2 = _chain_inputs(torch.bfloat16, 14)
    want, want2 = _chain(t, d), _chain(t2, d2)
    torch.cuda.synchronize(DEV)
    slow = torch.randn(4096, 4096, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        late = {n: torch.zeros_like(v) for n, v in t.items()}
        for _ in range(20):
            slow = slow @ slow * 1e-3
        for n in t:
            late[n].copy_(t[n])
        got = _chain(late, d)
    got2 = _chain(t2, d2)
    torch.cuda.synchronize(DEV)
    equal(got, want)
    equal(got2, want2)


def test_gradients_asked_for_in_part():
    x, do, dlast = make(2, 90, 4, 2, 32, 64, torch.bfloat16, seed=15)
    want = ssm.ssm_head_scan_bwd(do=do, dlast=dlast, **x)
    less = ssm.ssm_head_scan_bwd(do=do, dlast=dlast, want_dg=False, want_dh0=False, **x)
    assert less["dg"] is None and less["dh0"] is None
    for n in ("dq", "dk", "dv"):
        a, b = less[n].float(), want[n].float()
        # the same products; without dots the same scores too
        assert torch.equal(a, b), n
    leaves = [x[n].detach().requires_grad_() for n in ("q", "v")]
    o, last = ag.head_scan(leaves[0], x["k"], leaves[1], g=x["g"], h0=x["h0"], scale=x["scale"])
    got = torch.autograd.grad([last], leaves, [dlast], retain_graph=True)  # no gradient of o
    zero = ssm.ssm_head_scan_bwd(do=torch.zeros_like(do), dlast=dlast, **x)
    assert torch.equal(got[0], zero["dq"]) and torch.equal(got[1], zero["dv"])
    with pytest.raises(RuntimeError):
        (g,) = torch.autograd.grad([o], [leaves[0]], [do], create_graph=True)
        g.float().sum().backward()
