"""The larger variants in captured graphs (two heads a workgroup, many segments; copied operands, k in parts, 256 x 256
tiles), replayed several times with eager work between, and at the same time on two streams: the eager bits each time."""
import pytest
import torch

import selective_state_space_ssm_amd as ssm
from test_gpu_head import make

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def head(b, L, h, hk, dk, dv, dtype):
    x, do, dlast = make(b, L, h, hk, dk, dv, dtype, seed=L, ragged=True)

    def run():
        o, last = ssm.ssm_head_scan_fwd(**x)
        r = ssm.ssm_head_scan_bwd(do=do, dlast=dlast, **x)
        return [o, last, *r.values()]
    return run, [x["q"], x["v"], do]


def linear(rows, k, m, dtype):
    r = torch.Generator().manual_seed(rows)
    x, W, bias, res, dout = (torch.randn(*s, generator=r).to(dtype).to(DEV) for s in ((rows, k), (m, k), (m,), (rows, m),
                                                                                     (rows, m)))

    def run():
        out, pre = ssm.ssm_linear(x, W, bias, res, "silu", return_pre=True)
        return [out, pre, *ssm.ssm_linear_bwd(x, W, dout, pre, "silu")]
    return run, [x, W, dout]


VARIANTS = {
    "pairs": lambda: head(16, 130, 32, 4, 64, 32, torch.bfloat16),
    "segments": lambda: head(1, 1500, 4, 2, 100, 48, torch.float32),
    "copies": lambda: linear(700, 1536, 1001, torch.bfloat16),
    "copies_f32": lambda: linear(333, 1111, 770, torch.float32),
    "parts": lambda: linear(300, 4096, 2048, torch.float32),
    "large": lambda: linear(3336, 1928, 3592, torch.bfloat16),
}


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b) if x is not None)


@pytest.mark.parametrize("name", VARIANTS)
def test_captured(name):
    run, inputs = VARIANTS[name]()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize(DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run()
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize(DEV)
        assert same(got, run())
        for t in inputs:
            t.mul_(-0.75)
        torch.cuda.synchronize(DEV)


@pytest.mark.parametrize("name", VARIANTS)
def test_two_streams(name):
    run, _ = VARIANTS[name]()
    want = run()
    torch.cuda.synchronize(DEV)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got += [run() for _ in range(3)]
    torch.cuda.synchronize(DEV)
    assert all(same(r, want) for r in got)
