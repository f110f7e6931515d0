"""Gradients of the delta scan where a workgroup adds up the heads that share a key head: against the same call with every
head's own copy of its keys and queries, which takes the kernel of one head that the oracle's tests hold.

dv, dg, dbeta and dh0 are of one head alone.  dq and dk are sums over the heads: the copies' are each rounded to their type
(half a step, 2^-8 in bfloat16 and 2^-24 in float32 of each), the sum once more, and n float32 additions are off by n 2^-24
of what they add.
"""
import ctypes

import pytest
import torch

import selective_state_space_ssm_amd as ssm
from oracle import delta

from test_gpu_delta import DEV, IDS, TYPES, close, errors, f64, make

pytestmark = pytest.mark.gpu


def heads_of_a_workgroup(b, L, h, hk, dk, dv, dtype):
    """From the size of the workspace, which holds float32 parts of dq and dk for every group that is not all heads of a
    key head."""
    def size(key_heads):
        n = ctypes.c_int64()
        code = ssm.SSM_F32 if dtype == torch.float32 else ssm.SSM_BF16
        assert ssm.load_library().ssm_delta_scan_workspace(b, L, h, key_heads, dk, dv, code, 1, ctypes.byref(n)) == ssm.SSM_OK
        return n.value

    parts = size(hk) - size(h)
    return h // hk if parts == 0 else round(8 * b * h * L * dk / parts)


def own_keys(x):
    rep = x["v"].shape[2] // x["q"].shape[2]
    return dict(x, q=x["q"].repeat_interleave(rep, 2), k=x["k"].repeat_interleave(rep, 2))


def check(x, do, dlast, dtype, names=("dv", "dg", "dbeta", "dh0")):
    got = ssm.ssm_delta_scan_bwd(do=do, dlast=dlast, **x)
    one = ssm.ssm_delta_scan_bwd(do=do, dlast=dlast, **own_keys(x))
    torch.cuda.synchronize(DEV)
    for n in names:
        assert bool(torch.isfinite(got[n]).all())
        # the same products; what the compiler makes of the two kernels may differ in the order of a sum
        half = 2.0 ** -8 if got[n].dtype == torch.bfloat16 else 2.0 ** -24
        off, size = (got[n].double() - one[n].double()).abs(), one[n].double().abs()
        most = 2 * half * size + 2.0 ** -20 * size.max()
        assert bool((off <= most).all()), (n, float((off / most).max()))
    hk = x["q"].shape[2]
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    for n in ("dq", "dk"):
        parts = one[n].double().unflatten(2, (hk, -1))
        want, size = parts.sum(3), parts.abs().sum(3)
        off = (got[n].double() - want).abs()
        # the two kernels' own sums: float32, over d_value and a chunk's tokens
        most = half * (want.abs() + size) + 2.0 ** -20 * parts.norm(dim=-1, keepdim=True).sum(3) + 1e-30
        assert bool((off <= most).all()), (n, float((off / most).max()))


# b, L, h, hk, dk, dv; heads a workgroup adds up, float32 (chunks of 32 tokens) and bfloat16 (of 64)
CASES = [
    ((8, 1030, 8, 4, 128, 128), (2, 2)),   # two slabs of columns
    ((12, 700, 16, 4, 100, 72), (4, 4)),   # no whole vectors in bfloat16; a slab of eight columns
    ((26, 600, 8, 2, 72, 200), (4, 4)),    # four slabs
    ((4, 1100, 16, 2, 128, 80), (4, 2)),   # some of eight: parts
    ((16, 1030, 8, 4, 37, 130), (2, 2)),   # up to 64 keys
]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("case,n", CASES, ids=lambda c: "x".join(map(str, c)) if len(c) == 6 else "")
@pytest.mark.parametrize("fused", [False, True], ids=["dense", "views"])
def test_heads_added_up_in_a_workgroup(case, n, dtype, fused):
    b, L = case[:2]
    took = heads_of_a_workgroup(*case, dtype)
    assert took == n[TYPES.index(dtype)], took
    x, do, dlast = make(*case, dtype, seed=L, fused=fused)
    if fused:  # one value on: no row is a whole vector
        x["q"], x["k"], x["v"] = (torch.cat([t.flatten(2), t.new_zeros(b, L, 1)], -1)[..., :-1].unflatten(2, t.shape[2:])
                                  for t in (x["q"], x["k"], x["v"]))
    lens = [0, L, 64, 65, L - 1, 1, L // 2, -3]
    x["lengths"] = torch.tensor((lens * b)[:b], dtype=torch.int32, device=DEV)
    print(f"[delta shared] {case} {dtype} {took}", flush=True)
    check(x, do, dlast, dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_many_short_rows_against_the_oracle(dtype):
    case = (256, 5, 4, 2, 128, 128)
    assert heads_of_a_workgroup(*case, dtype) == 2
    x, do, dlast = make(*case, dtype, seed=3)
    x["lengths"] = torch.arange(256, dtype=torch.int32, device=DEV) % 6
    got = ssm.ssm_delta_scan_bwd(do=do, dlast=dlast, **x)
    y = f64(x)
    want = delta.delta_scan_bwd(**y, do=do.double().cpu().numpy(), dlast=dlast.double().cpu().numpy())
    e = errors(x, dtype, do, dlast)
    for n in ("dq", "dk", "dv", "dg", "dbeta", "dh0"):
        close(n, got[n], want[n], e[n])
    check(x, do, dlast, dtype)
