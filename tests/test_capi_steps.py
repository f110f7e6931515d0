"""How many (sequence, head) pairs the single-token steps take (CPU): as many as one launch has workgroups for.  The
addresses are made up and never reach the GPU."""
import pytest

import selective_state_space_ssm_amd as ssm

from test_capi_delta import STEP, status

# far enough from each other for the sizes below
FAR = {n: 1024 * v for n, v in STEP.items() if n in ("q", "k", "v", "g", "beta", "sin", "sout", "o")}


@pytest.mark.parametrize("sizes", [dict(b=1 << 19, h=32, dv=32), dict(b=1 << 18, h=32, dv=64), dict(b=1 << 18, h=32, dv=33)], ids=str)
def test_one_workgroup_too_many(sizes):
    a = {**STEP, **FAR, "hk": 32, "dk": 1, **sizes}
    rc, msg = status("ssm_delta_step", *(a[n] for n in STEP), None)
    assert rc == ssm.SSM_EUNSUPPORTED and "workgroups" in msg, (rc, msg)
    b = dict(a, beta=None)
    rc, msg = status("ssm_head_step", *(b[n] for n in STEP), None)
    assert rc == ssm.SSM_EUNSUPPORTED and "workgroups" in msg, (rc, msg)


def test_more_than_a_scan_takes_is_not_refused_for_that():
    """The next check, for a scale that is not finite, is reached."""
    a = {**STEP, **FAR, "b": 4096, "h": 32, "hk": 32, "dk": 128, "dv": 128, "scale": float("nan")}
    rc, msg = status("ssm_delta_step", *(a[n] for n in STEP), None)
    assert rc == ssm.SSM_EINVAL and "scale" in msg, (rc, msg)
    rc, msg = status("ssm_head_step", *(dict(a, beta=None)[n] for n in STEP), None)
    assert rc == ssm.SSM_EINVAL and "scale" in msg, (rc, msg)
