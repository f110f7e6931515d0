"""The head scan's C entry points with strides over a size of one (one token, one batch row): they address nothing, so
that every value of them gives the bits of the dense call."""
import pytest
import torch

import selective_state_space_ssm_amd as ssm

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def run(x, token, batch, backward):
    lib = ssm.load_library()
    q, k, v, do = x
    b, L, hk, dk = q.shape
    h, dv = v.shape[2:]
    code = ssm.SSM_F32 if q.dtype == torch.float32 else ssm.SSM_BF16
    ops = []
    for t, row in ((q, hk * dk), (k, hk * dk), (v, h * dv)):  # the dense strides where none is given
        ops += [t.data_ptr(), L * row if batch is None else batch, row if token is None else token]
    new = lambda *shape, dtype=q.dtype: torch.full(shape, 7.0, device=DEV, dtype=dtype)
    ws, nws = ssm._workspace("ssm_head_scan_workspace", DEV, b, L, h, hk, dk, dv, code, int(backward))
    stream = torch.cuda.current_stream(DEV).cuda_stream
    tail = [ssm._addr(ws), nws, b, L, h, hk, dk, dv, code, stream]
    if not backward:
        out = [new(b, L, h, dv), new(b, h, dk, dv, dtype=torch.float32)]
        rc = lib.ssm_head_scan_fwd(*ops, None, None, None, None, 0.5, *(t.data_ptr() for t in out), *tail)
    else:
        out = [new(b, L, hk, dk), new(b, L, hk, dk), new(b, L, h, dv), None, new(b, h, dk, dv, dtype=torch.float32)]
        rc = lib.ssm_head_scan_bwd(*ops, None, None, None, None, 0.5, do.data_ptr(), None, *(ssm._addr(t) for t in out), *tail)
    torch.cuda.synchronize(DEV)
    assert rc == ssm.SSM_OK, lib.ssm_last_error()
    return [t for t in out if t is not None]


@pytest.mark.parametrize("backward", [False, True], ids=["fwd", "bwd"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("b,L,token,batch", [(2, 1, 0, None), (2, 1, 1, None), (2, 1, 63, None), (1, 1, 0, 0), (1, 1, 3, 5),
                                             (1, 1, -7, -9), (1, 1, 1 << 40, 1 << 61), (1, 70, None, 0), (1, 70, None, -3)])
def test_a_stride_over_a_size_of_one_means_nothing(b, L, token, batch, dtype, backward):
    r = torch.Generator().manual_seed(21)
    x = [torch.randn(b, L, n, d, generator=r).to(dtype).to(DEV) for n, d in ((2, 32), (2, 32), (4, 32), (4, 32))]
    want = run(x, None, None, backward)
    got = run(x, token, batch, backward)
    assert all(torch.equal(a, w) for a, w in zip(got, want))
    assert all(float(a.float().abs().min()) < 7 for a in got)


def test_empty_sizes_are_refused_as_such():
    """No token, no sequence, no key, no value: the library's own refusal, for every call."""
    new = lambda *s: torch.zeros(*s, device=DEV)
    for b, L, h, dk, dv in ((0, 3, 2, 4, 4), (1, 0, 2, 4, 4), (1, 3, 0, 4, 4), (1, 3, 2, 0, 4), (1, 3, 2, 4, 0)):
        q, v = new(b, L, h, dk), new(b, L, h, dv)
        with pytest.raises(ssm.SSMError, match="sizes must be positive"):
            ssm.ssm_head_scan_fwd(q, q.clone(), v)
        with pytest.raises(ssm.SSMError, match="sizes must be positive"):
            ssm.ssm_head_scan_bwd(q, q.clone(), v, v.clone())
        if L:
            with pytest.raises(ssm.SSMError):
                ssm.ssm_head_step(new(b, h, dk), new(b, h, dk), new(b, h, dv), new(b, h, dk, dv))
