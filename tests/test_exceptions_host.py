"""Nothing is thrown across the C ABI: an entry point that runs out of host memory
returns MUON_ERR_INTERNAL.  Each call runs in a child process whose address space is
limited to little more than it holds, with more descriptors (or slices) than
the rest of it can take; none of them reaches a HIP call."""

import os
import subprocess
import sys

import pytest

import newton_schulz_flat_amd as nsf

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import ctypes, resource, sys
import numpy as np
import newton_schulz_flat_amd as nsf
lib = nsf.load_library()
P, G, M, U, T, C, W = (k << 40 for k in range(1, 8))       # never dereferenced
BIG = 1 << 62

# one matrix in very many slices: the list of slices does not fit
slices = nsf.descs_array([(0, 1 << 16, 1 << 17, 0, 32, 1 << 28)])
# very many matrices of one element: the list of matrices does not fit
n = 1 << 22
rows = np.zeros((n, 12), np.int32)
rows[:, 0] = 4 * np.arange(n)           # offset
rows[:, 2] = rows[:, 4] = rows[:, 10] = 1  # rows, cols, n_shards
rows[:, 6] = 8 * np.arange(n)           # param_offset
many = (nsf.MatrixDescC * n).from_buffer(rows)
assert (many[5].offset, many[5].rows, many[5].cols, many[5].n_shards) == (20, 1, 1, 1)
out = ctypes.c_size_t(0)
ranges = (nsf.RangeC * n)()
calls = {
    "muon_step": lambda: lib.muon_step(P, 0, BIG, G, M, BIG, slices, 1, 0., 0., 0., 1, 5, 0, W,
                                       1 << 40, None),
    "muon_step_noalloc": lambda: lib.muon_step_noalloc(P, 0, BIG, G, M, BIG, slices, 1, 0., 0., 0.,
                                                       1, 5, 0, None),
    "muon_step_grouped": lambda: lib.muon_step_grouped(P, 0, BIG, None, G, M, BIG, slices, 1, T, 1, 5,
                                                       0, W, 1 << 40, None),
    "muon_step_clipped": lambda: lib.muon_step_clipped(P, 0, BIG, None, G, M, BIG, slices, 1, T, 1, C,
                                                       5, 0, W, 1 << 40, None),
    "muon_apply": lambda: lib.muon_apply(P, 0, BIG, U, BIG, slices, 1, 0., 0., None),
    "muon_momentum": lambda: lib.muon_momentum(G, M, U, BIG, many, n, 0., 1, None),
    "muon_orthogonalize": lambda: lib.muon_orthogonalize(U, U, BIG, many, n, 5, 0, W, 1 << 40, None),
    "muon_workspace_bytes": lambda: lib.muon_workspace_bytes(many, n, 0, ctypes.byref(out)),
    "muon_adamw": lambda: lib.muon_adamw(P, 0, BIG, None, G, 0, M, U, BIG, ranges, n, T, 1, C, None),
}
name = sys.argv[1]
held = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (held + (48 << 20),) * 2)
rc = calls[name]()
print("status", rc, lib.muon_last_error().decode())
"""


@pytest.mark.parametrize("name", ["muon_step", "muon_step_noalloc", "muon_step_grouped",
                                  "muon_step_clipped", "muon_apply", "muon_momentum",
                                  "muon_orthogonalize", "muon_workspace_bytes", "muon_adamw"])
def test_out_of_host_memory_is_a_status(name):
    if not os.path.exists(nsf.LIB_PATH):
        from newton_schulz_flat_amd import build
        build.build()
    r = subprocess.run([sys.executable, "-c", CHILD, name], cwd=ROOT, capture_output=True, text=True,
                       timeout=120)
    assert r.returncode == 0, (r.returncode, r.stderr[-400:])
    assert "status -10 exception" in r.stdout, r.stdout
