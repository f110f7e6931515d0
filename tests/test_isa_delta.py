"""Static checks of the generated gfx950 code of the delta scan and of the norm with the residual's addition (CPU): no write
through the scalar data cache, no packed float32 arithmetic."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "selective_state_space_ssm_amd", "csrc")
SOURCES = ["ssm_delta.hip", "ssm_delta_bf16.hip", "ssm_delta_f32.hip", "ssm_delta_grad.hip", "ssm_addnorm.hip"]

pytestmark = pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="hipcc not available")


def test_no_scalar_cache_writes_and_no_packed_float32(tmp_path):
    flags = ["-O3", "--offload-arch=gfx950", "-std=c++17", "-ffp-contract=off", "-Xclang", "-target-feature", "-Xclang",
             "-packed-fp32-ops", "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-x", "hip", "--cuda-device-only", "-S"]
    run = {s: subprocess.Popen(["/opt/rocm/bin/hipcc", *flags, os.path.join(CSRC, s), "-o", str(tmp_path / (s + ".s"))],
                               stderr=subprocess.DEVNULL) for s in SOURCES}
    bad = re.compile(r"^\s*(s_store|s_buffer_store|s_scratch_store|s_atomic|s_buffer_atomic|s_dcache_wb|s_dcache_discard|"
                     r"v_pk_(add|mul|fma)_f32)\S*.*", re.M)
    for s, p in run.items():
        assert p.wait() == 0, s
        found = bad.search((tmp_path / (s + ".s")).read_text())
        assert found is None, (s, found[0])
