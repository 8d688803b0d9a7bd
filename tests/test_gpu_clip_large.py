"""GPU tests of norm, clipping and AdamW on sets that one launch grid does not cover, so that
workgroups take a second unit: clipping past 2^34 elements (34 GB of bfloat16),
AdamW past 2^33 (103 GB of weights, gradients and moments).  Every element has one
value, so that one left out or taken twice shows."""

import numpy as np
import pytest

from oracle import adamw_oracle as ao
from oracle import same_order as so
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

PIECE = 1 << 30


@pytest.fixture(scope="module")
def nsf():
    import newton_schulz_flat_amd as m
    m.load_library()
    return m


@pytest.fixture()
def torch():
    import torch as t
    assert t.cuda.is_available()
    t.cuda.empty_cache()
    yield t
    t.cuda.empty_cache()


def all_equal(t, value, lo=0, hi=None):
    hi = t.numel() if hi is None else hi
    return all(bool((t[i:min(i + PIECE, hi)] == value).all()) for i in range(lo, hi, PIECE))


def test_clipping_over_two_passes_of_the_grid(nsf, torch):
    """Three adjacent tensors: the first two are one run of exactly 2^34 elements, the longest
    that is made, and the third stays by itself."""
    say("clip past 2^34")
    half, rest = 1 << 33, (1 << 20) + 5
    n = 2 * half + rest
    t = torch.ones(n + 3, dtype=torch.bfloat16, device="cuda")
    parts = [t[:half], t[half:2 * half], t[2 * half:n]]
    clip = nsf.clip_state("cuda")
    nsf.muon_grad_norm(parts, 1.0, clip)
    # whole numbers below 2^53 add up exactly in any order
    assert float(clip.sumsq) == n
    norms = torch.zeros(3, device="cuda")
    nsf.muon_grad_norm(parts, 1.0, clip, tensor_norms=norms)
    assert float(clip.sumsq) == n
    assert norms.tolist() == [float(np.float32(np.sqrt(float(p.numel())))) for p in parts]
    nsf.clip_coef(clip).fill_(0.5)
    nsf.muon_clip_grads(parts, clip)
    torch.cuda.synchronize()
    assert all_equal(t, 0.5, 0, n)
    assert all_equal(t, 1.0, n)


def test_adamw_over_two_passes_of_the_grid(nsf, torch):
    """One range of 2^33 elements and a few more, in another group, behind a gap."""
    say("adamw past 2^33")
    long, gap, more = 1 << 33, 64, 300_007
    n = long + gap + more + 9
    groups = [(3e-2, 0.1, 0.9, 0.999, 1e-8, 3), (2e-2, 0.01, 0.5, 0.95, 1e-6, 7)]
    start = dict(w=1.0, g=0.25, m=0.03125, v=0.015625)
    kinds = dict(w=torch.bfloat16, g=torch.bfloat16, m=torch.float32, v=torch.float32)
    s = {k: torch.full((n,), x, dtype=kinds[k], device="cuda") for k, x in start.items()}
    nsf.muon_adamw(s["w"], s["g"], s["m"], s["v"],
                   [(0, long, 0, 0), (long + gap, more, long + gap, 1)],
                   nsf.adamw_group_table(groups, "cuda"))
    torch.cuda.synchronize()
    one = {k: np.array([x], np.float32) for k, x in start.items()}
    bits = {k: so.f32_to_bf16_bits(one[k]) for k in "wg"}
    for grp, lo, hi in ((groups[0], 0, long), (groups[1], long + gap, long + gap + more)):
        w, m, v = ao.adamw_same_order(bits["w"], bits["g"], one["m"], one["v"], grp)
        want = dict(w=so.bf16_bits_to_f32(w)[0], m=m[0], v=v[0])
        assert all(want[k] != start[k] for k in "wmv")
        for k in "wmv":
            assert all_equal(s[k], float(want[k]), lo, hi), (k, lo)
    for lo, hi in ((long, long + gap), (long + gap + more, n)):
        for k in "wmv":
            assert all_equal(s[k], start[k], lo, hi), (k, lo)
    assert all_equal(s["g"], start["g"])
