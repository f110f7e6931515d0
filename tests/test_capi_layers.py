"""Refusals of the head scan's, norm's and linear layer's entry points (CPU): every bad argument is turned away on the
host.  The addresses are made up and never reach the GPU: each call breaks exactly one rule."""
import ctypes

import pytest
import torch

import selective_state_space_ssm_amd as ssm

G = 1 << 32  # made-up, aligned addresses far from each other
INF, NAN = float("inf"), float("nan")


def status(fn, *args):
    lib = ssm.load_library()
    rc = getattr(lib, fn)(*args)
    return rc, lib.ssm_last_error().decode()


FWD = dict(q=G, qb=8192, qt=128, k=2 * G, kb=8192, kt=128, v=3 * G, vb=16384, vt=256, g=4 * G, gh=None, h0=None, lens=None,
           scale=1.0, o=5 * G, last=6 * G, ws=None, nws=0, b=2, L=64, h=4, hk=2, dk=64, dv=64, dtype=1)


def fwd(**kw):
    a = {**FWD, **kw}
    return status("ssm_head_scan_fwd", *(a[n] for n in FWD), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), ssm.SSM_EINVAL), (dict(o=None), ssm.SSM_EINVAL), (dict(b=0), ssm.SSM_EINVAL), (dict(L=-1), ssm.SSM_EINVAL),
    (dict(dk=0), ssm.SSM_EINVAL), (dict(h=5), ssm.SSM_EINVAL), (dict(dk=257), ssm.SSM_EUNSUPPORTED),
    (dict(dv=257), ssm.SSM_EUNSUPPORTED), (dict(dtype=2), ssm.SSM_EUNSUPPORTED), (dict(gh=9 * G), ssm.SSM_EINVAL),
    (dict(scale=INF), ssm.SSM_EINVAL), (dict(scale=NAN), ssm.SSM_EINVAL),
    (dict(qt=127), ssm.SSM_EINVAL), (dict(vb=100), ssm.SSM_EINVAL), (dict(kt=-128), ssm.SSM_EINVAL),
    (dict(vt=1 << 23, vb=1 << 40), ssm.SSM_EUNSUPPORTED),
    (dict(q=G + 1), ssm.SSM_EINVAL), (dict(o=5 * G + 8), ssm.SSM_EINVAL), (dict(h0=7 * G + 4), ssm.SSM_EINVAL),
    (dict(o=3 * G + 256), ssm.SSM_EINVAL), (dict(last=G + 16), ssm.SSM_EINVAL), (dict(last=5 * G + 64), ssm.SSM_EINVAL),
    (dict(h0=6 * G), ssm.SSM_EINVAL), (dict(L=1 << 31), ssm.SSM_EUNSUPPORTED), (dict(b=1 << 15, h=4), ssm.SSM_EUNSUPPORTED),
    (dict(b=1, L=4096, h=2, hk=1), ssm.SSM_EINVAL),  # needs a workspace
    (dict(b=1, L=4096, h=2, hk=1, ws=8 * G, nws=16), ssm.SSM_EINVAL),
])
def test_head_scan_fwd_refusals(kw, code):
    rc, msg = fwd(**kw)
    assert rc == code and msg, (rc, msg)


def workspace(*a):
    n = ctypes.c_int64(-1)
    rc = ssm.load_library().ssm_head_scan_workspace(*a, ctypes.byref(n))
    return rc, n.value


def test_head_scan_workspace():
    assert workspace(2, 64, 4, 2, 64, 64, 1, 0) == (ssm.SSM_OK, 0)
    rc, n = workspace(1, 4096, 2, 1, 64, 64, 1, 0)
    assert rc == ssm.SSM_OK and n >= 2 * 4096 // 256 * 64 * 64 * 4
    rc, n = workspace(2, 64, 4, 2, 64, 64, 1, 1)
    assert rc == ssm.SSM_OK and n > 0
    assert workspace(2, 64, 4, 3, 64, 64, 1, 1)[0] == ssm.SSM_EINVAL
    assert ssm.load_library().ssm_head_scan_workspace(2, 64, 4, 2, 64, 64, 1, 0, None) == ssm.SSM_EINVAL


BWD = dict(q=G, qb=8192, qt=128, k=2 * G, kb=8192, kt=128, v=3 * G, vb=16384, vt=256, g=4 * G, gh=None, h0=None, lens=None,
           scale=1.0, do=5 * G, dlast=None, dq=7 * G, dk=8 * G, dv=9 * G, dg=10 * G, dh0=11 * G, ws=12 * G, nws=G, b=2, L=64,
           h=4, hk=2, d_k=64, d_v=64, dtype=1)


@pytest.mark.parametrize("kw,code", [
    (dict(do=None), ssm.SSM_EINVAL), (dict(dq=None), ssm.SSM_EINVAL), (dict(g=None), ssm.SSM_EINVAL),
    (dict(ws=None), ssm.SSM_EINVAL), (dict(nws=64), ssm.SSM_EINVAL), (dict(do=5 * G + 2), ssm.SSM_EINVAL),
    (dict(dq=8 * G + 16), ssm.SSM_EINVAL), (dict(dv=5 * G), ssm.SSM_EINVAL), (dict(ws=3 * G), ssm.SSM_EINVAL),
    (dict(dh0=12 * G), ssm.SSM_EINVAL), (dict(d_v=300), ssm.SSM_EUNSUPPORTED), (dict(hk=3), ssm.SSM_EINVAL),
])
def test_head_scan_bwd_refusals(kw, code):
    a = {**BWD, **kw}
    rc, msg = status("ssm_head_scan_bwd", *(a[n] for n in BWD), None)
    assert rc == code and msg, (rc, msg)


STEP = dict(q=G, k=2 * G, v=3 * G, g=None, gh=None, scale=1.0, si=4 * G, so=4 * G, o=5 * G, b=2, h=4, hk=2, dk=64, dv=64,
            dtype=0)


@pytest.mark.parametrize("kw,code", [
    (dict(si=None), ssm.SSM_EINVAL), (dict(so=4 * G + 64), ssm.SSM_EINVAL), (dict(o=4 * G + 64), ssm.SSM_EINVAL),
    (dict(o=3 * G), ssm.SSM_EINVAL), (dict(q=G + 4), ssm.SSM_EINVAL), (dict(g=6 * G, gh=7 * G), ssm.SSM_EINVAL),
    (dict(h=3), ssm.SSM_EINVAL), (dict(dk=512), ssm.SSM_EUNSUPPORTED), (dict(scale=NAN), ssm.SSM_EINVAL),
    (dict(dtype=9), ssm.SSM_EUNSUPPORTED), (dict(b=-1), ssm.SSM_EINVAL),
])
def test_head_step_refusals(kw, code):
    a = {**STEP, **kw}
    rc, msg = status("ssm_head_step", *(a[n] for n in STEP), None)
    assert rc == code and msg, (rc, msg)


NORM = dict(x=G, z=2 * G, w=3 * G, y=4 * G, rows=4, c=64, groups=2, eps=1e-5, center=0, first=0, dtype=0)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), ssm.SSM_EINVAL), (dict(y=None), ssm.SSM_EINVAL), (dict(rows=0), ssm.SSM_EINVAL),
    (dict(groups=3), ssm.SSM_EINVAL), (dict(groups=0), ssm.SSM_EINVAL), (dict(c=8193, groups=1), ssm.SSM_EUNSUPPORTED),
    (dict(eps=-1.0), ssm.SSM_EINVAL), (dict(eps=NAN), ssm.SSM_EINVAL), (dict(eps=INF), ssm.SSM_EINVAL),
    (dict(center=2), ssm.SSM_EINVAL), (dict(first=-1), ssm.SSM_EINVAL), (dict(dtype=3), ssm.SSM_EUNSUPPORTED),
    (dict(x=G + 8), ssm.SSM_EINVAL), (dict(y=G), ssm.SSM_EINVAL), (dict(y=2 * G + 16), ssm.SSM_EINVAL),
    (dict(rows=1 << 40, c=8192, groups=1), ssm.SSM_EUNSUPPORTED),
])
def test_gate_norm_refusals(kw, code):
    a = {**NORM, **kw}
    rc, msg = status("ssm_gate_norm", *(a[n] for n in NORM), None)
    assert rc == code and msg, (rc, msg)


NBWD = dict(x=G, z=2 * G, w=3 * G, dy=4 * G, dx=5 * G, dz=6 * G, dw=7 * G, ws=8 * G, nws=G, rows=4, c=64, groups=2, eps=1e-5,
            center=0, first=0, dtype=0)


@pytest.mark.parametrize("kw", [dict(dy=None), dict(dx=None), dict(dz=None), dict(z=None), dict(ws=None), dict(nws=8),
                                dict(dx=4 * G), dict(dw=3 * G), dict(dx=6 * G + 16), dict(ws=G)])
def test_gate_norm_bwd_refusals(kw):
    a = {**NBWD, **kw}
    rc, msg = status("ssm_gate_norm_bwd", *(a[n] for n in NBWD), None)
    assert rc == ssm.SSM_EINVAL and msg, (rc, msg)


LIN = dict(x=G, W=2 * G, bias=3 * G, res=4 * G, act=1, out=5 * G, pre=6 * G, ws=7 * G, nws=G, rows=64, k=512, m=64, dtype=1)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), ssm.SSM_EINVAL), (dict(W=None), ssm.SSM_EINVAL), (dict(out=None), ssm.SSM_EINVAL),
    (dict(act=3), ssm.SSM_EINVAL), (dict(rows=0), ssm.SSM_EINVAL), (dict(k=-4), ssm.SSM_EINVAL),
    (dict(k=1 << 21), ssm.SSM_EUNSUPPORTED), (dict(m=1 << 21), ssm.SSM_EUNSUPPORTED), (dict(rows=1 << 40), ssm.SSM_EUNSUPPORTED),
    (dict(dtype=5), ssm.SSM_EUNSUPPORTED), (dict(bias=3 * G + 2), ssm.SSM_EINVAL), (dict(out=4 * G), ssm.SSM_EINVAL),
    (dict(pre=5 * G + 32), ssm.SSM_EINVAL), (dict(ws=None), ssm.SSM_EINVAL), (dict(nws=3), ssm.SSM_EINVAL), (dict(ws=G), ssm.SSM_EINVAL),
])
def test_linear_refusals(kw, code):
    a = {**LIN, **kw}
    rc, msg = status("ssm_linear", *(a[n] for n in LIN), None)
    assert rc == code and msg, (rc, msg)


LBWD = dict(x=G, W=2 * G, pre=3 * G, act=1, dout=4 * G, dx=5 * G, dW=6 * G, db=7 * G, ws=8 * G, nws=G, rows=64, k=512, m=64,
            dtype=1)


@pytest.mark.parametrize("kw", [dict(pre=None), dict(dout=None), dict(dx=None, dW=None, db=None), dict(dx=4 * G),
                                dict(dW=2 * G), dict(db=6 * G + 16), dict(ws=None), dict(nws=0), dict(dW=6 * G + 4), dict(act=-1)])
def test_linear_bwd_refusals(kw):
    a = {**LBWD, **kw}
    rc, msg = status("ssm_linear_bwd", *(a[n] for n in LBWD), None)
    assert rc == ssm.SSM_EINVAL and msg, (rc, msg)


def test_python_refuses_what_is_not_on_a_gpu():
    t = torch.zeros(1, 2, 1, 4)
    for f in (lambda: ssm.ssm_head_scan_fwd(t, t, t), lambda: ssm.ssm_head_scan_bwd(t, t, t, t),
              lambda: ssm.ssm_head_step(t[:, 0], t[:, 0], t[:, 0], torch.zeros(1, 1, 4, 4)), lambda: ssm.ssm_gate_norm(t),
              lambda: ssm.ssm_gate_norm_bwd(t, t), lambda: ssm.ssm_linear(t, torch.zeros(4, 4)),
              lambda: ssm.ssm_linear_bwd(t, torch.zeros(4, 4), t)):
        with pytest.raises(ValueError):
            f()
