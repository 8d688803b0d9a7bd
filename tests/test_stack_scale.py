"""Exponents and factors of the stacks' float16 pairs on the host (no GPU): first iterates of
every size, from the smallest float32 number's on."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_exponents_and_factors(tmp_path):
    exe = tmp_path / "stack_scale_check"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-D__HIP_PLATFORM_AMD__",
                    "-fsanitize=undefined", "-isystem", os.path.join(ROCM, "include"),
                    f"-I{os.path.join(ROOT, 'include')}",
                    f"-I{os.path.join(ROOT, 'newton_schulz_flat_amd', 'csrc')}",
                    os.path.join(ROOT, "tests", "stack_scale_check.cpp"), "-o", str(exe)],
                   check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout + out.stderr
    assert out.stdout.strip() == "ok"
