"""Static checks of the generated gfx950 code of the head scan, the norm and the linear layer (CPU): no write through the
scalar data cache, no packed float32 arithmetic, and the linear layer's loads into LDS as their kernel counts on."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "selective_state_space_ssm_amd", "csrc")
SOURCES = ["ssm_head.hip", "ssm_head_bf16.hip", "ssm_head_f32.hip", "ssm_norm.hip", "ssm_linear.hip"]

pytestmark = pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="hipcc not available")


@pytest.fixture(scope="module")
def isa(tmp_path_factory):
    d = tmp_path_factory.mktemp("isa")
    flags = ["-O3", "--offload-arch=gfx950", "-std=c++17", "-ffp-contract=off", "-Xclang", "-target-feature", "-Xclang",
             "-packed-fp32-ops", "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-x", "hip", "--cuda-device-only", "-S"]
    run = {s: subprocess.Popen(["/opt/rocm/bin/hipcc", *flags, os.path.join(CSRC, s), "-o", str(d / (s + ".s"))],
                               stderr=subprocess.DEVNULL) for s in SOURCES}
    for s, p in run.items():
        assert p.wait() == 0, s
    return {s: (d / (s + ".s")).read_text() for s in SOURCES}


def instructions(text):
    out = []
    for line in text.splitlines():
        line = line.split(";")[0].strip()
        if line and not line.endswith(":") and not line.startswith((".", "#")):
            parts = line.split(None, 1)
            out.append((parts[0], parts[1] if len(parts) > 1 else ""))
    return out


def test_no_scalar_cache_writes_and_no_packed_float32(isa):
    bad = re.compile(r"^(s_store|s_buffer_store|s_scratch_store|s_atomic|s_buffer_atomic|s_dcache_wb|s_dcache_discard|"
                     r"v_pk_(add|mul|fma)_f32)")
    for src, text in isa.items():
        for op, args in instructions(text):
            assert not bad.match(op), f"{src}: {op} {args}"


def test_lds_loads_of_the_linear_layer(isa):
    """Every load into LDS has its own M0 write and a wait state before it, nothing else touches M0, and no full wait
    stands between the first and the last of them (it would empty the pipeline every step)."""
    text = isa["ssm_linear.hip"]
    kernels = re.findall(r"^(_Z\w*ssm_linear_dma_kernel\w*):", text, flags=re.M)
    assert len(kernels) >= 4
    for k in kernels:
        ins = instructions(text.split("\n" + k + ":", 1)[1].split("s_endpgm", 1)[0])
        loads = [i for i, (op, a) in enumerate(ins) if op.startswith("buffer_load") and a.rstrip().endswith("lds")]
        assert loads, k
        for i in loads:
            assert ins[i - 1][0] == "s_nop" and ins[i - 2][0] == "s_mov_b32" and ins[i - 2][1].startswith("m0,"), (k, ins[i - 2:i])
        m0 = {i for i, (op, a) in enumerate(ins) if re.search(r"\bm0\b", a)}
        assert m0 == {i - 2 for i in loads}, k
        full = [i for i, (op, a) in enumerate(ins) if op == "s_waitcnt" and "vmcnt(0)" in a and loads[0] < i < loads[-1]]
        assert not full, (k, full)
