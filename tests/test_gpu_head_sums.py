"""The sums of dq and dk over the heads that share them where their workgroups take more than one turn: the bits of the
heads' own gradients added (float32, two heads)."""
import pytest
import torch

import selective_state_space_ssm_amd as ssm

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.mark.parametrize("b,L,hk,dk", [(4, 2049, 16, 64), (2, 2050, 17, 33)])
def test_many_values(b, L, hk, dk):
    r = torch.Generator(device=DEV).manual_seed(61)
    rnd = lambda *s: torch.randn(s, generator=r, device=DEV)
    q, k, v, do = rnd(b, L, hk, dk), rnd(b, L, hk, dk), rnd(b, L, 2 * hk, 16), rnd(b, L, 2 * hk, 16)
    g = -rnd(b, L, 2 * hk).abs()
    print(f"[head sums] {b} {L} {hk} {dk}", flush=True)
    got = ssm.ssm_head_scan_bwd(q, k, v, do, g=g)
    own = ssm.ssm_head_scan_bwd(q.repeat_interleave(2, 2), k.repeat_interleave(2, 2), v, do, g=g)
    for n in ("dq", "dk"):
        parts = own[n].unflatten(2, (hk, 2))
        assert torch.equal(got[n], parts[:, :, :, 0] + parts[:, :, :, 1]), n
    assert torch.equal(got["dv"], own["dv"]) and torch.equal(got["dg"], own["dg"])
