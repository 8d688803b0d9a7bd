"""What the host works out for stacks (no GPU): exponents and factors of the float16 pairs, for first
iterates of every size from the smallest float32 number's on, and how stages are divided among
workgroups."""

import math
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


def build(tmp_path, name, *flags):
    exe = tmp_path / name
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-D__HIP_PLATFORM_AMD__", *flags,
                    "-isystem", os.path.join(ROCM, "include"),
                    f"-I{os.path.join(ROOT, 'include')}",
                    f"-I{os.path.join(ROOT, 'newton_schulz_flat_amd', 'csrc')}",
                    os.path.join(ROOT, "tests", name + ".cpp"), "-o", str(exe)],
                   check=True)
    return str(exe)


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_exponents_and_factors(tmp_path):
    exe = build(tmp_path, "stack_scale_check", "-fsanitize=undefined")
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout + out.stderr
    assert out.stdout.strip() == "ok"


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_gpu_tests_take_every_tiling(tmp_path):
    pytest.importorskip("torch")
    from tests.test_gpu_stack import EVERY_TILING
    exe = build(tmp_path, "stack_tiling_check")

    def tilings(shapes):
        out = subprocess.run([exe], input="\n".join("%d %d %d" % s for s in shapes), capture_output=True,
                             text=True, check=True).stdout
        return set(out.splitlines())

    rng = random.Random(1)

    def log(lo, hi):
        return round(math.exp(rng.uniform(math.log(lo), math.log(hi))))

    shapes = [(log(1, 600), log(129, 20000), log(129, 20000)) for _ in range(30000)]
    found = tilings(shapes)
    assert len(found) >= 15
    assert found - tilings(EVERY_TILING) == set()
