"""The delta scan past 128 keys where its tiles of 64 columns are more than the CUs, so that (bfloat16) a workgroup takes 128:
against the oracle, and long rows, whose length is then cut, against fewer of them at a time."""
import pytest
import torch

import selective_state_space_ssm_amd as ssm

from test_gpu_delta import DEV, IDS, TYPES, make
from test_gpu_delta_edges import against_oracle, both

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("case", [(43, 70, 3, 3, 136, 72), (33, 33, 4, 2, 160, 136), (130, 9, 1, 1, 256, 256), (260, 3, 1, 1, 130, 65)],
                         ids=lambda c: "x".join(map(str, c)))
def test_against_the_oracle(case, dtype):
    x, do, dlast = make(*case, dtype, seed=case[1], ragged=True)
    print(f"[delta wide] {case} {dtype}", flush=True)
    against_oracle(x, do, dlast, dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_long_rows(dtype):
    """Every result rounded once to its type on either side, and sums in float32: 2^-7 of a token's vector (float32: 1e-5)."""
    b, L, h, dk, dv = 44, 1500, 3, 136, 72
    x, do, dlast = make(b, L, h, h, dk, dv, dtype, seed=7)
    x["lengths"] = torch.randint(0, L + 1, (b,), generator=torch.Generator().manual_seed(1)).to(torch.int32).to(DEV)
    got = both(x, do, dlast)
    for lo in range(0, b, 11):
        part = {n: t[lo:lo + 11].clone() if isinstance(t, torch.Tensor) else t for n, t in x.items()}
        want = both(part, do[lo:lo + 11].contiguous(), dlast[lo:lo + 11].clone())
        for n, w in want.items():
            by = 2.0 ** -7 if w.dtype == torch.bfloat16 else 1e-5
            off, size = (got[n][lo:lo + 11].double() - w.double()).flatten(2).norm(dim=2), w.double().flatten(2).norm(dim=2)
            assert bool((off <= by * size + 1e-6 * size.max()).all()), (n, lo, float((off / size).nan_to_num().max()))
