"""Single-token steps of more (sequence, head) pairs than a scan takes: the bits of the same sequences a part at a time."""
import pytest
import torch

import selective_state_space_ssm_amd as ssm

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("b,h,hk,dk,dv", [(4096, 32, 16, 16, 40), (70000, 1, 1, 8, 8)], ids=["", "one head"])
def test_steps_of_many_sequences(b, h, hk, dk, dv, dtype):
    r = torch.Generator(device=DEV).manual_seed(b)
    rnd = lambda *s: torch.randn(s, generator=r, device=DEV)
    q, k, v, g = rnd(b, hk, dk).to(dtype), rnd(b, hk, dk).to(dtype), rnd(b, h, dv).to(dtype), (-rnd(b, h).abs()).to(dtype)
    beta, state = torch.rand(b, h, generator=r, device=DEV).to(dtype), rnd(b, h, dk, dv)
    delta = lambda i, s: ssm.ssm_delta_step(q[i], k[i], v[i], beta[i], s, g=g[i])
    head = lambda i, s: ssm.ssm_head_step(q[i], k[i], v[i], s, g=g[i])
    for f in (delta, head):
        o, s = f(slice(None), state.clone())
        n = b // 8 * 4
        for part in (slice(0, n), slice(n, None)):
            o2, s2 = f(part, state[part].clone())
            assert torch.equal(o[part], o2) and torch.equal(s[part], s2)
