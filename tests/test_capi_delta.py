"""Refusals of the delta scan's and the add norm's entry points (CPU): every bad argument is turned away on the host.  The
addresses are made up and never reach the GPU: each call breaks exactly one rule."""
import ctypes

import pytest
import torch

import selective_state_space_ssm_amd as ssm

G = 1 << 36  # made-up, aligned addresses far from each other
INF, NAN = float("inf"), float("nan")
EINVAL, EUNSUPPORTED = ssm.SSM_EINVAL, ssm.SSM_EUNSUPPORTED


def status(fn, *args):
    lib = ssm.load_library()
    rc = getattr(lib, fn)(*args)
    return rc, lib.ssm_last_error().decode()


FWD = dict(q=G, qb=8192, qt=128, k=2 * G, kb=8192, kt=128, v=3 * G, vb=16384, vt=256, g=4 * G, beta=10 * G, h0=None, lens=None,
           scale=1.0, o=5 * G, last=6 * G, ws=8 * G, nws=G, b=2, L=64, h=4, hk=2, dk=64, dv=64, dtype=1)
BWD = dict(q=G, qb=8192, qt=128, k=2 * G, kb=8192, kt=128, v=3 * G, vb=16384, vt=256, g=4 * G, beta=10 * G, h0=None, lens=None,
           scale=1.0, do=5 * G, dlast=None, dq=6 * G, d_k=7 * G, d_v=9 * G, dg=11 * G, db=12 * G, dh0=13 * G, ws=14 * G, nws=G,
           b=2, L=64, h=4, hk=2, dk=64, dv=64, dtype=1)

SHARED = [
    (dict(q=None), EINVAL), (dict(v=None), EINVAL), (dict(b=0), EINVAL), (dict(L=-1), EINVAL), (dict(dk=0), EINVAL),
    (dict(h=5), EINVAL), (dict(dk=257), EUNSUPPORTED), (dict(dv=257), EUNSUPPORTED), (dict(dtype=2), EUNSUPPORTED),
    (dict(scale=INF), EINVAL), (dict(scale=NAN), EINVAL), (dict(qt=127), EINVAL), (dict(vb=100), EINVAL), (dict(kt=-128), EINVAL),
    (dict(vt=1 << 23, vb=1 << 40), EUNSUPPORTED), (dict(q=G + 1), EINVAL), (dict(g=4 * G + 1), EINVAL), (dict(beta=10 * G + 1), EINVAL),
    (dict(L=1 << 31), EUNSUPPORTED), (dict(b=1 << 15, h=4), EUNSUPPORTED), (dict(ws=None), EINVAL), (dict(nws=16), EINVAL),
    (dict(ws=G + 64), EINVAL), (dict(h0=20 * G + 4), EINVAL), (dict(lens=20 * G + 4), EINVAL),
]


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(o=None), EINVAL), (dict(o=5 * G + 8), EINVAL), (dict(o=3 * G + 256), EINVAL), (dict(last=G + 16), EINVAL),
    (dict(last=5 * G + 64), EINVAL), (dict(h0=6 * G), EINVAL), (dict(last=10 * G), EINVAL), (dict(ws=5 * G), EINVAL)])
def test_scan_fwd_refusals(kw, code):
    a = {**FWD, **kw}
    rc, msg = status("ssm_delta_scan_fwd", *(a[n] for n in FWD), None)
    assert rc == code and msg, (rc, msg)


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(do=None), EINVAL), (dict(dq=None), EINVAL), (dict(d_k=None), EINVAL), (dict(d_v=None), EINVAL), (dict(g=None), EINVAL),
    (dict(beta=None), EINVAL), (dict(dq=5 * G), EINVAL), (dict(dg=6 * G + 16), EINVAL), (dict(db=10 * G), EINVAL),
    (dict(dh0=9 * G), EINVAL), (dict(dlast=13 * G), EINVAL), (dict(db=12 * G + 2), EINVAL), (dict(do=5 * G + 2), EINVAL)])
def test_scan_bwd_refusals(kw, code):
    a = {**BWD, **kw}
    rc, msg = status("ssm_delta_scan_bwd", *(a[n] for n in BWD), None)
    assert rc == code and msg, (rc, msg)


def workspace(*a):
    n = ctypes.c_int64(-1)
    rc = ssm.load_library().ssm_delta_scan_workspace(*a, ctypes.byref(n))
    return rc, n.value


def test_scan_workspace():
    for dtype in (0, 1):
        last = 0
        for L in (1, 64, 65, 1000, 100000):
            rc, f = workspace(2, L, 4, 2, 64, 64, dtype, 0)
            assert rc == ssm.SSM_OK and f > 0
            rc, b = workspace(2, L, 4, 2, 64, 64, dtype, 1)
            assert rc == ssm.SSM_OK and b > f and b >= last
            last = b
    assert workspace(2, 64, 4, 3, 64, 64, 1, 1)[0] == EINVAL
    assert workspace(2, 0, 4, 2, 64, 64, 1, 1)[0] == EINVAL
    assert ssm.load_library().ssm_delta_scan_workspace(2, 64, 4, 2, 64, 64, 1, 0, None) == EINVAL


def test_too_many_workgroups():
    a = {**FWD, "q": G, "b": 65535, "h": 1, "hk": 1, "dk": 1, "dv": 1, "L": 1 << 19, "qt": 1, "kt": 1, "vt": 1, "qb": 1 << 19,
         "kb": 1 << 19, "vb": 1 << 19, "dtype": 0, "g": None, "beta": None, "last": None}
    big = 1 << 46
    a.update(q=big, k=2 * big, v=3 * big, o=4 * big, ws=5 * big, nws=big)
    rc, msg = status("ssm_delta_scan_fwd", *(a[n] for n in FWD), None)
    assert rc == EUNSUPPORTED and "workgroups" in msg, (rc, msg)


STEP = dict(q=G, k=2 * G, v=3 * G, g=4 * G, beta=5 * G, scale=1.0, sin=6 * G, sout=6 * G, o=7 * G, b=2, h=4, hk=2, dk=64, dv=64,
            dtype=1)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), EINVAL), (dict(sin=None), EINVAL), (dict(o=None), EINVAL), (dict(h=3), EINVAL), (dict(dk=300), EUNSUPPORTED),
    (dict(dtype=7), EUNSUPPORTED), (dict(scale=NAN), EINVAL), (dict(beta=5 * G + 8), EINVAL), (dict(sout=6 * G + 64), EINVAL),
    (dict(o=6 * G + 64), EINVAL), (dict(sout=5 * G), EINVAL), (dict(o=G), EINVAL), (dict(b=0), EINVAL)])
def test_step_refusals(kw, code):
    a = {**STEP, **kw}
    rc, msg = status("ssm_delta_step", *(a[n] for n in STEP), None)
    assert rc == code and msg, (rc, msg)


NORM = dict(x=G, res=2 * G, w=3 * G, y=4 * G, h=5 * G, rows=4, c=64, eps=1e-5, dtype=1, rdtype=0)
NORM8 = dict(x=G, res=2 * G, w=3 * G, y=4 * G, scale=6 * G, group=32, h=5 * G, rows=4, c=64, eps=1e-5, dtype=1, rdtype=0)
NORMS = [
    (dict(x=None), EINVAL), (dict(y=None), EINVAL), (dict(rows=0), EINVAL), (dict(c=0), EINVAL), (dict(c=8256), EUNSUPPORTED),
    (dict(eps=-1.0), EINVAL), (dict(eps=NAN), EINVAL), (dict(dtype=2), EUNSUPPORTED), (dict(rdtype=2), EUNSUPPORTED),
    (dict(dtype=0, rdtype=1), EUNSUPPORTED), (dict(x=G + 8), EINVAL), (dict(w=3 * G + 4), EINVAL), (dict(h=2 * G + 64), EINVAL),
    (dict(h=G), EINVAL), (dict(y=G), EINVAL), (dict(y=2 * G), EINVAL), (dict(y=5 * G), EINVAL), (dict(rows=1 << 40), EUNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", NORMS)
def test_add_norm_refusals(kw, code):
    for name, base in (("ssm_add_norm", NORM), ("ssm_add_norm_e4m3", NORM8)):
        a = {**base, **kw}
        if "rows" in kw and kw["rows"] > 1:  # far enough from each other for that size
            a.update({n: v * 1024 for n, v in a.items() if n in ("x", "res", "w", "y", "h", "scale")})
        rc, msg = status(name, *(a[n] for n in base), None)
        assert rc == code and msg, (name, rc, msg)


@pytest.mark.parametrize("kw,code", [
    (dict(scale=None), EINVAL), (dict(group=48), EUNSUPPORTED), (dict(group=-32), EUNSUPPORTED), (dict(group=128), EINVAL),
    (dict(c=65, group=64), EINVAL), (dict(scale=6 * G + 4), EINVAL), (dict(scale=4 * G), EINVAL), (dict(scale=3 * G), EINVAL)])
def test_add_norm_e4m3_refusals(kw, code):
    a = {**NORM8, **kw}
    rc, msg = status("ssm_add_norm_e4m3", *(a[n] for n in NORM8), None)
    assert rc == code and msg, (rc, msg)


NBWD = dict(h=G, w=2 * G, dy=3 * G, dh=4 * G, dx=5 * G, dres=6 * G, dw=7 * G, ws=8 * G, nws=G, rows=4, c=64, eps=1e-5, dtype=1,
            rdtype=0)


@pytest.mark.parametrize("kw,code", [
    (dict(h=None), EINVAL), (dict(dy=None), EINVAL), (dict(dx=None, dres=None, dw=None), EINVAL), (dict(ws=None), EINVAL),
    (dict(nws=8), EINVAL), (dict(dx=3 * G), EINVAL), (dict(dres=4 * G), EINVAL), (dict(dw=2 * G), EINVAL), (dict(ws=G), EINVAL),
    (dict(dx=6 * G + 16), EINVAL), (dict(c=9000), EUNSUPPORTED), (dict(rdtype=1, dtype=0), EUNSUPPORTED), (dict(dh=4 * G + 2), EINVAL)])
def test_add_norm_bwd_refusals(kw, code):
    a = {**NBWD, **kw}
    rc, msg = status("ssm_add_norm_bwd", *(a[n] for n in NBWD), None)
    assert rc == code and msg, (rc, msg)


def test_add_norm_workspace():
    n = ctypes.c_int64(-1)
    lib = ssm.load_library()
    for rows, c in ((1, 1), (1, 8192), (100000, 64), (3, 513)):
        assert lib.ssm_add_norm_workspace(rows, c, ctypes.byref(n)) == ssm.SSM_OK and 4 * c <= n.value <= 4096 * c
    assert lib.ssm_add_norm_workspace(1, 9000, ctypes.byref(n)) == EUNSUPPORTED
    assert lib.ssm_add_norm_workspace(1, 10, None) == EINVAL


def test_python_refuses_what_is_not_on_a_gpu():
    t = torch.zeros(1, 2, 1, 4)
    for f in (lambda: ssm.ssm_delta_scan_fwd(t, t, t), lambda: ssm.ssm_delta_scan_bwd(t, t, t, t),
              lambda: ssm.ssm_delta_step(t[:, 0], t[:, 0], t[:, 0], None, torch.zeros(1, 1, 4, 4)), lambda: ssm.ssm_add_norm(t),
              lambda: ssm.ssm_add_norm_e4m3(t), lambda: ssm.ssm_add_norm_bwd(t, t)):
        with pytest.raises(ValueError):
            f()
