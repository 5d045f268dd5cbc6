"""What the routed-field calls hand to their launchers (no GPU): the pairs'
quotient for every number of choices, and no refusal of sizes that fit the card.
``tests/native/host_expert_limits.cpp`` with ``csrc/experts_abi.cpp``."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "volume_rendering_amd", "csrc")


def test_quotients_and_limits(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "host_expert_limits")
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, "-fsanitize=undefined", "-fno-sanitize-recover=all",
           os.path.join(ROOT, "tests", "native", "host_expert_limits.cpp"), os.path.join(CSRC, "experts_abi.cpp"),
           "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-4000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, (run.stdout + run.stderr)[-4000:]
    assert "checks passed" in run.stdout
