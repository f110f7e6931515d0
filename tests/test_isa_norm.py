"""The norm's compiled kernels (CPU): none for groups that no call can have."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "selective_state_space_ssm_amd", "csrc")

pytestmark = pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="hipcc not available")


def test_no_kernel_is_made_for_groups_past_the_limit(tmp_path):
    """A kernel of LANES lanes with NV vectors of 16 bytes serves groups of up to LANES * NV vectors; the one of half
    that size serves the rest, so that it must not pass the 8192 values a group may have."""
    out = tmp_path / "norm.s"
    subprocess.run(["/opt/rocm/bin/hipcc", "-O1", "--offload-arch=gfx950", "-std=c++17", "-I", os.path.join(ROOT, "include"),
                    "-I", CSRC, "-x", "hip", "--cuda-device-only", "-S", os.path.join(CSRC, "ssm_norm.hip"), "-o", str(out)],
                   check=True, stderr=subprocess.DEVNULL)
    names = set(re.findall(r"^(_Z\w*ssm_gate_norm_\w*kernel\w*):", out.read_text(), flags=re.M))
    sizes = [re.search(r"dev\d*(BF16|F32)ELi(\d+)ELi(\d+)E", n) for n in names]
    assert len(names) >= 60 and all(sizes)
    for n, m in zip(names, sizes):
        values = int(m[2]) * int(m[3]) * (8 if m[1] == "BF16" else 4)
        assert values <= 8192, (n, values)
