"""Refusals of sizes whose launch would have 2^32 threads or more (CPU): on the host, before any launch.  The addresses
are made up and never reach the GPU."""
import pytest

import selective_state_space_ssm_amd as ssm

import test_capi_layers as base

G = 1 << 46  # far enough from each other for these sizes


def norm(**kw):
    a = {**base.NORM, "x": G, "z": None, "w": None, "y": 2 * G, **kw}
    return base.status("ssm_gate_norm", *(a[n] for n in base.NORM), None)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("rows,c,groups", [(1 << 31, 1, 1), (1 << 24, 128, 128), (1 << 30, 128, 2), (1 << 29, 1 << 9, 1),
                                           (1 << 25, 1 << 13, 1)])
def test_gate_norm(rows, c, groups, dtype):
    # groups side by side in a workgroup of 256 (8 lanes or more each), four times that where they are small
    lanes = 8
    n = c // groups * (2 if dtype else 4)
    while lanes < 64 and lanes * 16 < n:
        lanes *= 2
    per = 1 if n > 2048 else 256 // lanes * (2 if n > 1024 else 4)
    assert rows * groups >= per * (1 << 24)
    rc, msg = norm(rows=rows, c=c, groups=groups, dtype=dtype)
    assert rc == ssm.SSM_EUNSUPPORTED and "workgroups" in msg, (rc, msg)


@pytest.mark.parametrize("kw", [dict(rows=8, c=1 << 31, groups=1 << 31), dict(rows=1, c=1 << 35, groups=1 << 30)])
def test_gate_norm_of_many_groups(kw):
    a = {**base.NBWD, "x": G, "z": None, "w": None, "dy": 2 * G, "dx": 3 * G, "dz": None, "dw": None, **kw}
    rc, msg = base.status("ssm_gate_norm_bwd", *(a[n] for n in base.NBWD), None)
    assert rc == ssm.SSM_EUNSUPPORTED and "workgroups" in msg, (rc, msg)


def test_head_scan():
    a = {**base.FWD, "q": G, "k": 2 * G, "v": 3 * G, "o": 4 * G, "last": None, "g": None, "b": 65535, "h": 1, "hk": 1, "dk": 1,
         "dv": 1, "L": 1 << 19, "qt": 1, "kt": 1, "vt": 1, "qb": 1 << 19, "kb": 1 << 19, "vb": 1 << 19, "dtype": 0,
         "ws": 5 * G, "nws": G}
    bwd = dict(a, do=6 * G, dlast=None, dq=7 * G, dv=9 * G, dg=None, dh0=None)
    bwd.update(d_k=1, d_v=1, dk=8 * G)
    rc, msg = base.status("ssm_head_scan_bwd", *(bwd[n] for n in base.BWD), None)
    assert rc == ssm.SSM_EUNSUPPORTED and "workgroups" in msg, (rc, msg)
