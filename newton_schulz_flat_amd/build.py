"""Build the gfx950 shared library ``libmuon_step.so`` from ``csrc/``.

Every source is compiled by ``hipcc --offload-arch=gfx950`` into ``_build/``
at the repository root (in parallel), then linked into
``newton_schulz_flat_amd/libmuon_step.so``.  Cross-compiles without a GPU.

    python -m newton_schulz_flat_amd.build
"""

from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmuon_step.so")

SOURCES = [
    "muon_abi.cpp",
    "muon_validate.cpp",
    "muon_plan.cpp",
    "muon_profile.cpp",
    "k_elementwise.hip",
    "k_norm_cast.hip",
    "k_ns_gemm.hip",
    "muon_noalloc.hip",
    "muon_clip.cpp",
    "k_clip.hip",
    "k_adamw.hip",
    "muon_fp8.cpp",
    "k_fp8_cast.hip",
    "k_fp8_gemm.hip",
    "muon_stack.cpp",
    "k_stack.hip",
    "k_stack_small.hip",
]
# Sources whose arithmetic must round every operation separately.
NO_CONTRACT = {"k_elementwise.hip", "k_norm_cast.hip", "k_clip.hip", "k_adamw.hip",
               "k_fp8_cast.hip"}

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
COMMON = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall",
    # packed float32 instructions stay off: ordinary float code only
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    f"-I{INCLUDE}", f"-I{CSRC}",
]


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, src + ".o")
    cmd = [HIPCC, *COMMON, "-c", os.path.join(CSRC, src), "-o", obj]
    if src in NO_CONTRACT:
        cmd.append("-ffp-contract=off")
    if src.endswith(".cpp"):
        cmd[1:1] = ["-x", "hip"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling {src} failed:\n{r.stdout}\n{r.stderr}")
    return obj


def build(verbose: bool = False, jobs: int = 6) -> str:
    """Compile every source and link the library; returns the library path."""
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=jobs) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
