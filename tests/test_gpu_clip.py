"""GPU tests of the global gradient norm, clipping and AdamW.

* Norm: against exact sums of squares (float64 squares of float32 values are
  exact).  The device's sum has at most N float64 roundings, so sumsq is within
  N 2^-53 of it, and norm and coef are within half a float32 step of the exact
  ones beside that: 2^-24 (1 + tiny).
* Clipping and AdamW: bit for bit against the same-order float32 chains, and
  AdamW against the float64 definition within the chain's roundings.
* The chain as used: norm, Muon step and AdamW on the clipped gradient,
  eagerly and in a captured graph replayed with other gradients.
"""

import dataclasses
import math

import numpy as np
import pytest

import workloads as wlm
from oracle import adamw_oracle as ao
from oracle import same_order as so
from tests.gpu_helpers import bits, host, say

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -24       # half a float32 step, relative
DT = {"f32": 4, "bf16": 2}


@pytest.fixture(scope="module")
def nsf():
    import newton_schulz_flat_amd as m
    m.load_library()
    return m


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available()
    return t


def tdtype(torch, name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def values(t):
    """float32 values of a tensor on the host."""
    a = host(t)
    return ao.widen(a)


def make_list(torch, sizes, seed, std=1.0, shift=0, dtypes=("f32", "bf16")):
    """Tensors of the given lengths inside larger buffers of NaN, at element offset
    `shift` + 0..7, types in turn."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out, owners = [], []
    for k, n in enumerate(sizes):
        off = (shift + k) % 8
        buf = torch.full((n + 24,), math.nan, dtype=tdtype(torch, dtypes[k % len(dtypes)]),
                         device="cuda")
        t = buf[off:off + n]
        t.copy_(torch.randn(n, generator=gen, device="cuda") * std)
        out.append(t)
        owners.append(buf)
    return out, owners


def read(nsf, clip):
    c = clip.record.cpu()
    f = c.numpy().view(np.float32)
    return float(c[0]), float(f[2]), float(f[3])


def check_record(nsf, clip, arrays, max_norm):
    s, norm, coef = read(nsf, clip)
    n = sum(a.size for a in arrays)
    want = ao.sumsq(arrays)
    assert abs(s - want) <= n * 2.0 ** -53 * want, (s, want)
    root = math.sqrt(want)
    eps = n * 2.0 ** -53 + 2.0 ** -50
    assert abs(norm - root) <= (HALF + eps) * root, (norm, root)
    c = ao.coefficient(want, max_norm)
    assert abs(coef - c) <= (HALF + eps) * c, (coef, c)
    return s


SIZES = {
    "solo_full": [2048] * 47 + [2048],      # the longest list that one workgroup takes,
    "solo_over": [2048] * 47 + [2049],      # and one element more
    "single": [1],
    "empty": [0],
    "edges": [0, 1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 31, 33, 63, 65, 255, 257, 1023, 1025],
    "units": [8191, 8192, 8193, 16384, 0, 1, 24577, 8192, 8192],
    "launches": [300] * 241 + [259, 256, 5],
    "many_small": [1 + (7 * k) % 23 for k in range(700)],
    "mixed": [300000, 1, 0, 77777, 131072, 5, 1 << 20],
}


@pytest.mark.parametrize("dtypes", [("f32",), ("bf16",), ("f32", "bf16")])
@pytest.mark.parametrize("name", sorted(SIZES))
def test_norm(nsf, torch, name, dtypes):
    say("grad norm", name, dtypes)
    ts, _ = make_list(torch, SIZES[name], 5, std=0.3, shift=len(name), dtypes=dtypes)
    clip = nsf.clip_state("cuda")
    norms = torch.full((len(ts),), -1.0, device="cuda")
    ws = torch.full((nsf.muon_clip_workspace_bytes(ts),), 255, dtype=torch.uint8, device="cuda")
    nsf.muon_grad_norm(ts, 0.75, clip, tensor_norms=norms, workspace=ws)
    torch.cuda.synchronize()
    arrays = [values(t) for t in ts]
    check_record(nsf, clip, arrays, 0.75)
    got = host(norms)
    for a, x in zip(arrays, got):
        want = math.sqrt(ao.sumsq([a]))
        assert abs(float(x) - want) <= (HALF + a.size * 2.0 ** -53 + 2.0 ** -50) * want
    # without norms and in the default workspace the sum may take another order (short
    # lists go to one workgroup, adjacent tensors are one): two sums of the same N
    # terms, each within N 2^-53 of the exact one, check_record's bound for both
    again, third = nsf.clip_state("cuda"), nsf.clip_state("cuda")
    nsf.muon_grad_norm(nsf.tensor_list(ts), 0.75, again)
    nsf.muon_grad_norm(ts, 0.75, third)
    torch.cuda.synchronize()
    check_record(nsf, again, arrays, 0.75)
    # the same call twice: the same bits
    assert torch.equal(again.record, third.record)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("count,n", [(5, 8), (40, 2001), (300, 9001), (700, 513)])
def test_packed_lists(nsf, torch, count, n, dtype):
    """Tensors one behind the other, in their order and shuffled: norm (with and
    without each one's own), clipping into another buffer and in place."""
    say("packed", count, n, dtype)
    flat = torch.randn(count * n + 3, device="cuda").to(tdtype(torch, dtype))
    out = torch.full((count * n + 3,), math.nan, device="cuda")
    before = host(flat).copy()
    parts = [flat[1 + k * n:1 + (k + 1) * n] for k in range(count)]
    outs = [out[1 + k * n:1 + (k + 1) * n] for k in range(count)]
    order = np.random.default_rng(count).permutation(count)
    clip, norms = nsf.clip_state("cuda"), torch.zeros(count, device="cuda")
    inner = values(flat)[1:-2]
    for idx in (range(count), order):
        nsf.muon_grad_norm([parts[k] for k in idx], 1.0, clip)
        check_record(nsf, clip, [inner], 1.0)
        nsf.muon_grad_norm([parts[k] for k in idx], 1.0, clip, tensor_norms=norms)
        check_record(nsf, clip, [inner], 1.0)
        got = host(norms)
        for j, k in enumerate(idx):
            want = math.sqrt(ao.sumsq([inner[k * n:(k + 1) * n]]))
            assert abs(float(got[j]) - want) <= (HALF + n * 2.0 ** -53 + 2.0 ** -50) * want
        out.fill_(math.nan)
        nsf.muon_clip_grads([parts[k] for k in idx], clip, out=[outs[k] for k in idx])
        coef = read(nsf, clip)[2]
        want = ao.clip_same_order(before[1:-2], coef, "f32")
        assert np.array_equal(bits(host(out)[1:-2]), bits(want))
        assert np.isnan(host(out)[[0, -2, -1]]).all()
    nsf.muon_clip_grads([parts[k] for k in order], clip)
    want = before.copy()
    want[1:-2] = ao.clip_same_order(before[1:-2], coef, dtype)
    assert np.array_equal(bits(host(flat)), bits(want))


def test_norm_of_an_empty_list(nsf, torch):
    clip = nsf.clip_state("cuda")
    clip.record.fill_(7.0)
    nsf.muon_grad_norm([], 1.0, clip)
    torch.cuda.synchronize()
    assert read(nsf, clip) == (0.0, 0.0, 1.0)
    nsf.muon_clip_grads([], clip)


@pytest.mark.parametrize("n", [4096, 8192 * 2048, 8192 * 2048 + 1, 8192 * 4096 - 3])
def test_norm_where_workgroups_and_tensors_end_together(nsf, torch, n):
    """Tensors of whole units, before and behind one that fills every workgroup."""
    say("norm of whole units", n)
    ts, _ = make_list(torch, [8192, n, 8192, 16384], 3, dtypes=("f32",))
    clip = nsf.clip_state("cuda")
    ws = torch.full((nsf.muon_clip_workspace_bytes(ts),), 255, dtype=torch.uint8, device="cuda")
    norms = torch.zeros(4, device="cuda")
    nsf.muon_grad_norm(ts, 1.0, clip, tensor_norms=norms, workspace=ws)
    each = [t.double().square().sum() for t in ts]
    want = float(sum(each))
    s, norm, _ = read(nsf, clip)
    assert abs(s - want) <= 2 * 2.0 ** -53 * sum(t.numel() for t in ts) * want
    for e, x in zip(each, host(norms)):
        assert abs(float(x) - math.sqrt(float(e))) <= 2 * HALF * math.sqrt(float(e))


def test_norm_range(nsf, torch):
    """Squares beyond float32 at both ends; infinities and NaN."""
    say("norm range")
    clip = nsf.clip_state("cuda")

    def norm_of(vals, max_norm=1.0):
        t = torch.tensor(vals, dtype=torch.float32, device="cuda")
        nsf.muon_grad_norm([t], max_norm, clip)
        return read(nsf, clip), np.array(vals, np.float32)

    for vals in ([3e30, 4e30], [3e-30, 4e-30], [1e38, 1e-40], [1e-45], [0.0, -0.0]):
        (s, norm, coef), a = norm_of(vals)
        check_record(nsf, clip, [a], 1.0)
    # norms past float32's largest: infinite in float32, the coefficient still right
    (s, norm, coef), a = norm_of([3e38] * 4)
    assert math.isinf(norm) and math.isfinite(s)
    c = ao.coefficient(ao.sumsq([a]), 1.0)
    assert abs(coef - c) <= max(HALF * c, 2.0 ** -150)
    (s, norm, coef), _ = norm_of([1.0, math.inf])
    assert math.isinf(s) and math.isinf(norm) and coef == 0.0
    (s, norm, coef), _ = norm_of([math.inf, -math.inf, math.nan])
    assert math.isnan(s) and math.isnan(norm) and math.isnan(coef)
    (s, norm, coef), _ = norm_of([2.0] * 100, math.inf)
    assert (norm, coef) == (20.0, 1.0)
    (s, norm, coef), _ = norm_of([2.0] * 100, 0.0)
    assert (norm, coef) == (20.0, 0.0)
    (s, norm, coef), _ = norm_of([0.0] * 100, 0.0)
    assert (norm, coef) == (0.0, 0.0)
    (s, norm, coef), _ = norm_of([2.0] * 100, 19.0)
    assert coef == np.float32(19.0 / (20.0 + 1e-6))


def test_parts_add_up(nsf, torch):
    """The ranks' way: sums of squares of two parts added, then finished."""
    say("norm of parts")
    ts, _ = make_list(torch, [50000, 333, 8192, 70001], 11)
    whole, a, b = (nsf.clip_state("cuda") for _ in range(3))
    nsf.muon_grad_norm(ts, 2.0, whole)
    nsf.muon_grad_norm(ts[:2], math.inf, a)
    nsf.muon_grad_norm(ts[2:], math.inf, b)
    nsf.clip_sumsq(a).add_(nsf.clip_sumsq(b))
    nsf.muon_clip_finish(a, 2.0)
    torch.cuda.synchronize()
    check_record(nsf, a, [values(t) for t in ts], 2.0)
    # one rounding of the sum apart
    assert abs(read(nsf, a)[0] - read(nsf, whole)[0]) <= 4 * 2.0 ** -53 * 130000 * read(nsf, whole)[0]


def test_overlapping_tensors_count_each(nsf, torch):
    t = torch.randn(5000, device="cuda")
    clip = nsf.clip_state("cuda")
    nsf.muon_grad_norm([t, t[100:300], t], 1.0, clip)
    torch.cuda.synchronize()
    a = values(t)
    check_record(nsf, clip, [a, a[100:300], a], 1.0)


@pytest.mark.parametrize("out", [None, "f32", "bf16"])
@pytest.mark.parametrize("dtypes", [("f32",), ("bf16",), ("f32", "bf16")])
@pytest.mark.parametrize("name", sorted(SIZES))
def test_clip(nsf, torch, name, dtypes, out):
    say("clip", name, dtypes, out)
    sizes = SIZES[name]
    ts, owners = make_list(torch, sizes, 9, std=1.0, dtypes=dtypes)
    clip = nsf.clip_state("cuda")
    nsf.muon_grad_norm(ts, 0.5, clip)
    before = [host(t).copy() for t in ts]
    if out is None:
        nsf.muon_clip_grads(ts, clip)
        res, bufs = ts, owners
    else:
        # half of the destinations reach their vector boundary where their source does
        res, bufs = make_list(torch, sizes, 1, shift=0 if len(name) % 2 else 3, dtypes=(out,))
        nsf.muon_clip_grads(nsf.tensor_list(ts), clip, out=res)
    torch.cuda.synchronize()
    coef = read(nsf, clip)[2]
    for k, (b, t, buf) in enumerate(zip(before, res, bufs)):
        to = "bf16" if t.dtype == torch.bfloat16 else "f32"
        assert np.array_equal(bits(host(t)), bits(ao.clip_same_order(b, coef, to))), k
        if out is not None:
            assert np.array_equal(bits(host(ts[k])), bits(b)), k
        lo = t.storage_offset()
        assert torch.isnan(buf[:lo]).all() and torch.isnan(buf[lo + t.numel():]).all(), k


@pytest.mark.parametrize("sdt", ["f32", "bf16"])
@pytest.mark.parametrize("ddt", ["f32", "bf16"])
def test_clip_long_lists(nsf, torch, sdt, ddt):
    """Lists past the size up to which the source stays cached, odd lengths and
    offsets; one product in float32, rounded once, is torch's too."""
    say("clip long", sdt, ddt)
    sizes = [40_000_003, 8192 * 700, 13]
    ts, _ = make_list(torch, sizes, 13, dtypes=(sdt,))
    res, bufs = make_list(torch, sizes, 1, dtypes=(ddt,))
    clip = nsf.clip_state("cuda")
    nsf.muon_grad_norm(ts, 3.0, clip)
    nsf.muon_clip_grads(ts, clip, out=res)
    for t, r, buf in zip(ts, res, bufs):
        want = (t.float() * clip.coef).to(r.dtype)
        assert torch.equal(r, want)
        lo = r.storage_offset()
        assert torch.isnan(buf[:lo]).all() and torch.isnan(buf[lo + r.numel():]).all()
    total = sum(t.double().square().sum() for t in ts)
    s, norm, coef = read(nsf, clip)
    n = sum(sizes)
    assert abs(s - float(total)) <= 2 * n * 2.0 ** -53 * s
    assert abs(norm - math.sqrt(s)) <= HALF * (1 + 1e-6) * norm
    assert abs(coef - 3.0 / (math.sqrt(s) + 1e-6)) <= HALF * (1 + 1e-6) * coef


@pytest.mark.parametrize("sp", range(8))
def test_clip_alignments(nsf, torch, sp):
    """Every pair of element offsets and types, lengths around the vectors'."""
    say("clip alignments", sp)
    clip = nsf.clip_state("cuda")
    nsf.clip_coef(clip).fill_(1 / 3)
    src, dst = [], []
    for td in ("f32", "bf16"):
        for ts in ("f32", "bf16"):
            for dp in range(8):
                for n in (1, 6, 8, 13, 40, 3001):
                    a = torch.randn(n + 16, device="cuda").to(tdtype(torch, ts))
                    b = torch.full((n + 16,), math.nan, dtype=tdtype(torch, td), device="cuda")
                    src.append(a[sp:sp + n])
                    dst.append(b[dp:dp + n])
    nsf.muon_clip_grads(src, clip, out=dst)
    torch.cuda.synchronize()
    for s, d in zip(src, dst):
        to = "bf16" if d.dtype == torch.bfloat16 else "f32"
        assert np.array_equal(bits(host(d)), bits(ao.clip_same_order(host(s), 1 / 3, to)))


def test_clip_special_values(nsf, torch):
    say("clip specials")
    vals = [0.0, -0.0, 1e-45, -1e-38, 3e38, math.inf, -math.inf, math.nan, 1.0]
    clip = nsf.clip_state("cuda")
    for c in (1.0, 0.0, 0.25, math.nan):
        nsf.clip_coef(clip).fill_(c)
        for inplace in (True, False):
            t = torch.tensor(vals * 5, device="cuda")
            o = t if inplace else torch.empty_like(t)
            nsf.muon_clip_grads([t], clip, out=None if inplace else [o])
            want = ao.clip_same_order(np.array(vals * 5, np.float32), c, "f32")
            got = host(o)
            assert np.array_equal(np.isnan(got), np.isnan(want))
            ok = ~np.isnan(want)
            assert np.array_equal(bits(got)[ok], bits(want)[ok])


def test_clip_by_one(nsf, torch):
    """A coefficient of 1: in place nothing changes (the bits of NaN among it), into
    other tensors everything arrives, also where a list has both."""
    say("clip by one")
    clip = nsf.clip_state("cuda")
    nsf.clip_coef(clip).fill_(1.0)
    raw = torch.tensor([0x7f800001, 0x7fc12345, 0x3f800000, 0xff812345 - (1 << 32)] * 5000,
                       dtype=torch.int32, device="cuda").view(torch.float32)
    a, b = raw.clone(), torch.randn(9001, device="cuda").bfloat16()
    nsf.muon_clip_grads([a, b], clip)
    assert torch.equal(a.view(torch.int32), raw.view(torch.int32))
    c, d = b.clone(), torch.zeros(9001, device="cuda")
    nsf.muon_clip_grads([c, b], clip, out=[c, d])
    assert torch.equal(c, b) and torch.equal(d, b.float())


# ---------------------------------------------------------------------- AdamW

GROUPS = [(1e-3, 0.1, 0.9, 0.999, 1e-8, 1), (2e-2, 0.0, 0.5, 0.95, 1e-6, 7),
          (5e-4, 0.01, 0.95, 0.9999, 1e-12, 123456)]


def adamw_setup(torch, sizes, wdt, gdt, seed, align=8, gap=16, reverse_params=False):
    """Ranges with gaps in flat buffers, groups in turn; params laid out in another order if
    asked."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ranges, off = [], 8
    for k, n in enumerate(sizes):
        ranges.append([off, n, off, k % len(GROUPS)])
        off = -(-(off + n) // align) * align + gap * (k % 2)
    if reverse_params:
        at = 0
        for r in reversed(ranges):
            r[2] = at
            at = -(-(at + r[1]) // 8) * 8
    size = off + 8

    def rnd(std, dt=torch.float32):
        return (torch.randn(size, generator=gen, device="cuda") * std).to(dt)
    w = rnd(0.05, tdtype(torch, wdt))
    g = rnd(0.1, tdtype(torch, gdt))
    m = rnd(0.03)
    v = (torch.rand(size, generator=gen, device="cuda") + 1e-3) * 0.01
    return [tuple(r) for r in ranges], w, g, m, v


def adamw_want(ranges, w, g, m, v, coef):
    w, g, m, v = (host(x).copy() for x in (w, g, m, v))
    for off, n, poff, grp in ranges:
        s, p = slice(off, off + n), slice(poff, poff + n)
        w[p], m[s], v[s] = ao.adamw_same_order(w[p], g[s], m[s], v[s], GROUPS[grp], coef)
    return w, m, v


@pytest.mark.parametrize("clipped", [True, False])
@pytest.mark.parametrize("gdt", ["f32", "bf16"])
@pytest.mark.parametrize("wdt", ["f32", "bf16"])
@pytest.mark.parametrize("name", sorted(SIZES))
def test_adamw(nsf, torch, name, wdt, gdt, clipped):
    say("adamw", name, wdt, gdt, clipped)
    ranges, w, g, m, v = adamw_setup(torch, SIZES[name], wdt, gdt, 17, align=4 if wdt == "f32" else 8,
                                     reverse_params=name in ("edges", "mixed"))
    clip = None
    coef = None
    if clipped:
        clip = nsf.clip_state("cuda")
        nsf.clip_coef(clip).fill_(0.37)
        coef = np.float32(0.37)
    copy = None
    if wdt == "f32":
        copy = torch.full((w.numel(),), math.nan, dtype=torch.bfloat16, device="cuda")
    want = adamw_want(ranges, w, g, m, v, coef)
    gb = host(g).copy()
    nsf.muon_adamw(w, g, m, v, ranges, nsf.adamw_group_table(GROUPS, "cuda"), clip=clip,
                   model_copy=copy)
    torch.cuda.synchronize()
    for got, ref, what in zip((w, m, v), want, "wmv"):
        # gaps between ranges included: those stay as they were
        assert np.array_equal(bits(host(got)), bits(ref)), what
    assert np.array_equal(bits(host(g)), bits(gb))
    if copy is not None:
        c = host(copy)
        inside = np.zeros(w.numel(), bool)
        for off, n, poff, _ in ranges:
            inside[poff:poff + n] = True
        assert np.array_equal(c[inside], so.f32_to_bf16_bits(want[0])[inside])
        assert np.isnan(so.bf16_bits_to_f32(c[~inside])).all()


@pytest.mark.parametrize("wdt", ["f32", "bf16"])
def test_adamw_adjacent_ranges(nsf, torch, wdt):
    """Ranges one behind the other (some of one group, empty ones among them, one that
    is adjacent in the state alone), in any order: the same as each alone."""
    say("adamw adjacent", wdt)
    n = 4000
    w = (torch.randn(n, device="cuda") * 0.05).to(tdtype(torch, wdt))
    g, m = (torch.randn(n, device="cuda") * 0.1 for _ in range(2))
    v = torch.rand(n, device="cuda") * 0.01
    ranges = [(0, 64, 0, 0), (64, 128, 64, 0), (192, 0, 192, 0), (192, 800, 192, 0),
              (992, 8, 992, 1), (1000, 1000, 1000, 1), (2000, 40, 2400, 1), (2040, 13, 2440, 1),
              (2056, 5, 2000, 2), (2064, 1200, 2600, 2)]
    want = adamw_want(ranges, w, g, m, v, None)
    table = nsf.adamw_group_table(GROUPS, "cuda")
    for idx in (range(len(ranges)), reversed(range(len(ranges)))):
        w1, m1, v1 = w.clone(), m.clone(), v.clone()
        nsf.muon_adamw(w1, g, m1, v1, [ranges[k] for k in idx], table)
        torch.cuda.synchronize()
        for got, ref in zip((w1, m1, v1), want):
            assert np.array_equal(bits(host(got)), bits(ref))


def test_adamw_against_the_definition(nsf, torch):
    """30 steps from zero state against float64.  The moments' relative error grows by
    at most 6 half steps a step; each update's is within (6 + 6) t of its own size
    (lr here, |m_hat| / sqrt(v_hat) <= 1 / sqrt(1 - beta2) at most), and the weights
    add 4 half steps of their size a step."""
    say("adamw definition")
    n, steps = 4099, 30
    lr, wd, b1, b2, eps = 1e-2, 0.1, 0.9, 0.99, 1e-8
    gen = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randn(n, generator=gen, device="cuda")
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    W, M, V = (host(x).astype(np.float64) for x in (w, m, v))
    tab = nsf.adamw_group_table([(lr, wd, b1, b2, eps)], "cuda")
    clip = nsf.clip_state("cuda")
    for t in range(1, steps + 1):
        g = torch.randn(n, generator=gen, device="cuda")
        nsf.muon_grad_norm([g], 1.0, clip)
        nsf.muon_adamw(w, g, m, v, [(0, n)], tab, clip=clip)
        nsf.adamw_steps(tab).add_(1)
        W, M, V = ao.adamw(W, host(g), M, V, (lr, wd, b1, b2, eps, t), read(nsf, clip)[2])
    torch.cuda.synchronize()
    scale_m = float(np.abs(M).max())
    assert np.abs(host(m) - M).max() <= 6 * steps * HALF * max(scale_m, 1.0 / 30)
    assert (np.abs(host(v) - V) <= 6 * steps * HALF * V).all()
    per = lr * 12 * steps * HALF / math.sqrt(1 - b2) + 4 * HALF * (np.abs(W).max() + 1)
    assert np.abs(host(w) - W).max() <= steps * per
    assert np.abs(W).max() > 1.0 and np.abs(host(w) - W).max() < 1e-4


def test_adamw_nonfinite_stays_where_it_is(nsf, torch):
    say("adamw non-finite")
    n = 1000
    ranges, w, g, m, v = adamw_setup(torch, [n], "f32", "f32", 4)
    off = ranges[0][0]
    g[off + 3], g[off + 500], g[off + 501] = math.nan, math.inf, -math.inf
    want = adamw_want(ranges, w, g, m, v, None)
    nsf.muon_adamw(w, g, m, v, ranges, nsf.adamw_group_table(GROUPS, "cuda"))
    torch.cuda.synchronize()
    for got, ref in zip((w, m, v), want):
        a = host(got)
        assert np.array_equal(np.isnan(a), np.isnan(ref))
        ok = ~np.isnan(ref)
        assert np.array_equal(bits(a)[ok], bits(ref)[ok])


# ------------------------------------------------------- the step on clipped gradients

@pytest.mark.parametrize("mode", ["f32", "bf16"])
@pytest.mark.parametrize("ns_steps", [5, 0])
@pytest.mark.parametrize("max_norm", [1e-2, 1e9])
def test_step_clipped_equals_clip_then_step(nsf, torch, mode, ns_steps, max_norm):
    wl = wlm.small_mixed(41, count=7, max_side=300, param_dtype="bf16", shards=2)
    say("step_clipped == clip + step", mode, ns_steps, max_norm)
    params, grads, mom = wlm.make_tensors(wl, "cuda", momentum_std=1e-3)
    p2, m2, g2 = params.clone(), mom.clone(), grads.clone()
    before = grads.clone()
    views = [grads[d.offset:d.offset + d.rows * d.cols] for d in wl.descs]
    clip = nsf.clip_state("cuda")
    table = nsf.group_table([(0.02, 0.01, 0.95, True)], "cuda")
    nsf.muon_grad_norm(views, max_norm, clip)
    nsf.muon_step_clipped(params, grads, mom, wl.descs, table, clip, ns_steps=ns_steps, mode=mode)
    nsf.muon_clip_grads([g2], clip)
    nsf.muon_step_grouped(p2, g2, m2, wl.descs, table, ns_steps=ns_steps, mode=mode)
    torch.cuda.synchronize()
    assert torch.equal(grads, before)
    assert np.array_equal(bits(host(params)), bits(host(p2)))
    assert np.array_equal(bits(host(mom)), bits(host(m2)))
    coef = read(nsf, clip)[2]
    assert (coef == 1.0) == (max_norm > 1)


@pytest.mark.parametrize("coef", [0.3, math.nan])
def test_step_clipped_groups_copy_and_waves(nsf, torch, coef):
    """float32 weights with model copy, three groups, tall and wide and unaligned rows, in
    one wave and in several."""
    wl = wlm.small_mixed(43, count=8, max_side=330, param_dtype="f32")
    say("step_clipped groups, copy, waves", coef)
    descs = [dataclasses.replace(d, group=k % 3) for k, d in enumerate(wl.descs)]
    params, grads, mom = wlm.make_tensors(wl, "cuda", momentum_std=1e-3)
    table = nsf.group_table([(0.02, 0.01, 0.95, True), (0.005, 0.0, 0.9, False),
                             (0.05, 0.1, 0.8, True)], "cuda")
    clip = nsf.clip_state("cuda")
    nsf.clip_coef(clip).fill_(coef)
    p0, m0, g0 = params.clone(), mom.clone(), grads.clone()
    c0 = torch.zeros(params.numel(), dtype=torch.bfloat16, device="cuda")
    nsf.muon_clip_grads([g0], clip)
    nsf.muon_step_grouped(p0, g0, m0, descs, table, model_copy=c0)
    for size in (nsf.muon_workspace_bytes(descs), nsf.muon_workspace_min_bytes(descs)):
        p1, m1, c1 = params.clone(), mom.clone(), torch.zeros_like(c0)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        nsf.muon_step_clipped(p1, grads, m1, descs, table, clip, model_copy=c1, workspace=ws)
        torch.cuda.synchronize()
        for a, b in ((p0, p1), (m0, m1), (c0, c1)):
            x, y = ao.widen(host(a)), ao.widen(host(b))
            assert np.array_equal(x, y, equal_nan=True)


def small_training(nsf, torch, seed):
    wl = wlm.small_mixed(seed, count=5, max_side=200, param_dtype="f32")
    params, grads, mom = wlm.make_tensors(wl, "cuda", momentum_std=1e-3)
    ranges, w, g, m, v = adamw_setup(torch, [3000, 17, 70000, 1], "f32", "bf16", seed)
    views = [grads[d.offset:d.offset + d.rows * d.cols] for d in wl.descs]
    views += [g[o:o + n] for o, n, _, _ in ranges]
    return dict(wl=wl, params=params, grads=grads, mom=mom, ranges=ranges, w=w, g=g, m=m, v=v,
                tensors=nsf.tensor_list(views), clip=nsf.clip_state("cuda"),
                groups=nsf.group_table([(0.02, 0.01, 0.95, True)], "cuda"),
                agroups=nsf.adamw_group_table(GROUPS, "cuda"),
                copy=torch.zeros(w.numel(), dtype=torch.bfloat16, device="cuda"),
                ws=torch.empty(nsf.muon_workspace_bytes(wl.descs), dtype=torch.uint8,
                               device="cuda"),
                cws=torch.empty(nsf.muon_clip_workspace_bytes(views), dtype=torch.uint8,
                                device="cuda"))


def training_step(nsf, s):
    nsf.muon_grad_norm(s["tensors"], 1.0, s["clip"], workspace=s["cws"])
    nsf.muon_step_clipped(s["params"], s["grads"], s["mom"], s["wl"].descs, s["groups"], s["clip"],
                          workspace=s["ws"])
    nsf.muon_adamw(s["w"], s["g"], s["m"], s["v"], s["ranges"], s["agroups"], clip=s["clip"],
                   model_copy=s["copy"])
    nsf.adamw_steps(s["agroups"]).add_(1)


def state_of(s):
    return [host(x).copy() for x in (*(s[k] for k in ("params", "mom", "w", "m", "v", "copy",
                                                       "agroups")), s["clip"].record)]


def new_gradients(torch, s, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s["grads"].normal_(0.0, 1e-2 / seed, generator=gen)
    s["g"].normal_(0.0, 0.1, generator=gen)


def test_training_step_in_a_graph(nsf, torch):
    """Norm, Muon step and AdamW together, captured once and replayed on new
    gradients, equal to the eager calls after every replay (bit for bit); the norm
    is that of all gradients, and AdamW's part equals the same-order chain."""
    say("training step in a graph")
    eager, graphed = (small_training(nsf, torch, 51) for _ in range(2))
    side = torch.cuda.Stream()
    # the Muon step's plan is built outside the capture
    warm = small_training(nsf, torch, 51)
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        training_step(nsf, warm)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        training_step(nsf, graphed)
    for rep in range(1, 5):
        for s in (eager, graphed):
            new_gradients(torch, s, rep)
        torch.cuda.synchronize()
        w, g, m, v = (eager[k].clone() for k in "wgmv")
        steps = host(nsf.adamw_steps(eager["agroups"])).tolist()
        training_step(nsf, eager)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(state_of(eager), state_of(graphed)):
            assert np.array_equal(a, b), rep
        coef = read(nsf, eager["clip"])[2]
        check_record(nsf, eager["clip"], [values(t) for t in eager["tensors"].tensors], 1.0)
        wn, gn, mn, vn = (host(x).copy() for x in (w, g, m, v))
        for off, n, poff, grp in eager["ranges"]:
            sl, pl = slice(off, off + n), slice(poff, poff + n)
            grow = GROUPS[grp][:5] + (steps[grp],)
            wn[pl], mn[sl], vn[sl] = ao.adamw_same_order(wn[pl], gn[sl], mn[sl], vn[sl], grow, coef)
        for k, ref in zip("wmv", (wn, mn, vn)):
            assert np.array_equal(bits(host(eager[k])), bits(ref)), (rep, k)


@pytest.mark.parametrize("sizes", [[300, 5, 77], [200000, 3, 8192, 70001]])
def test_norm_and_clip_in_graphs(nsf, torch, sizes):
    """Norm and clipping captured as their first calls on their tensors: in place and into
    other tensors, two graphs over one record and workspace, replayed in turn."""
    say("norm and clip in graphs", sizes)
    ts, _ = make_list(torch, sizes, 21)
    clip = nsf.clip_state("cuda")
    outs = [torch.zeros(n, device="cuda") for n in sizes]
    tl = nsf.tensor_list(ts)
    ws = torch.empty(nsf.muon_clip_workspace_bytes(tl), dtype=torch.uint8, device="cuda")
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        nsf.muon_grad_norm(tl, 2.0, clip, workspace=ws)
        nsf.muon_clip_grads(tl, clip, out=outs)
    with torch.cuda.graph(second):
        nsf.muon_grad_norm(tl, 1.0, clip, workspace=ws)
        nsf.muon_clip_grads(tl, clip)
    gen = torch.Generator(device="cuda").manual_seed(1)
    for rep in range(4):
        for t in ts:
            t.copy_(torch.randn(t.numel(), generator=gen, device="cuda"))
        before = [host(t).copy() for t in ts]
        torch.cuda.synchronize()
        first.replay()
        torch.cuda.synchronize()
        check_record(nsf, clip, [ao.widen(b) for b in before], 2.0)
        coef = read(nsf, clip)[2]
        for b, o in zip(before, outs):
            assert np.array_equal(bits(host(o)), bits(ao.clip_same_order(b, coef, "f32"))), rep
        second.replay()
        torch.cuda.synchronize()
        coef = read(nsf, clip)[2]
        for b, t in zip(before, ts):
            to = "bf16" if t.dtype == torch.bfloat16 else "f32"
            assert np.array_equal(bits(host(t)), bits(ao.clip_same_order(b, coef, to))), rep


def test_default_workspace_is_refused_under_capture(nsf, torch):
    t = torch.ones(8, device="cuda")
    clip = nsf.clip_state("cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError, match="workspace"):
            nsf.muon_grad_norm([t], 1.0, clip)
        nsf.muon_clip_grads([t], clip)


def test_two_streams_at_once(nsf, torch):
    """Calls on two streams, each with its own record and (default) workspace."""
    say("two streams")
    streams = [torch.cuda.Stream() for _ in range(2)]
    lists = [make_list(torch, [70000 + 5000 * k, 3, 400000], 60 + k)[0] for k in range(2)]
    clips = [nsf.clip_state("cuda") for _ in range(2)]
    outs = [[torch.empty(t.numel(), device="cuda") for t in ts] for ts in lists]
    torch.cuda.synchronize()
    for rep in range(5):
        for st, ts, c, o in zip(streams, lists, clips, outs):
            with torch.cuda.stream(st):
                nsf.muon_grad_norm(ts, 1.0, c)
                nsf.muon_clip_grads(ts, c, out=o)
    torch.cuda.synchronize()
    for ts, c, o in zip(lists, clips, outs):
        check_record(nsf, c, [values(t) for t in ts], 1.0)
        coef = read(nsf, c)[2]
        for t, x in zip(ts, o):
            assert np.array_equal(bits(host(x)), bits(ao.clip_same_order(host(t), coef, "f32")))


def test_binding_refusals_on_the_device(nsf, torch):
    clip = nsf.clip_state("cuda")
    t = torch.zeros(64, device="cuda")
    with pytest.raises(TypeError):
        nsf.tensor_list([t.half()])
    with pytest.raises(ValueError, match="contiguous"):
        nsf.tensor_list([t[::2]])
    with pytest.raises(TypeError):
        nsf.tensor_list([1.0])
    with pytest.raises(TypeError, match="clip_state"):
        nsf.muon_grad_norm([t], 1.0, torch.zeros(2, dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError, match="GPU"):
        nsf.muon_grad_norm([], 1.0, nsf.clip_state("cpu"))
    with pytest.raises(ValueError, match="one element per tensor"):
        nsf.muon_grad_norm([t], 1.0, clip, tensor_norms=torch.zeros(2, device="cuda"))
    with pytest.raises(nsf.MuonError) as e:
        nsf.muon_grad_norm([t], 1.0, clip, workspace=torch.zeros(0, dtype=torch.uint8, device="cuda"))
    assert e.value.name in ("MUON_ERR_NULL_POINTER", "MUON_ERR_WORKSPACE_TOO_SMALL")
    with pytest.raises(ValueError, match="in out"):
        nsf.muon_clip_grads([t], clip, out=[t, t])
    tab = nsf.adamw_group_table(GROUPS, "cuda")
    with pytest.raises(ValueError, match="as many elements"):
        nsf.muon_adamw(t, t, t[:32], t, [(0, 8)], tab)
    with pytest.raises(ValueError, match="adamw_group_table"):
        nsf.muon_adamw(t, t, t, t, [(0, 8)], tab[:, :3].contiguous())
    with pytest.raises(nsf.MuonError) as e:
        nsf.muon_adamw(t, t, t, t, [(0, 8)], tab)
    assert e.value.name == "MUON_ERR_ALIAS"


def test_kernel_timing_names(nsf, torch):
    t, long = torch.ones(100, device="cuda"), torch.ones(1 << 18, device="cuda")
    clip = nsf.clip_state("cuda")
    z = [torch.zeros(100, device="cuda") for _ in range(3)]
    table = nsf.adamw_group_table(GROUPS, "cuda")
    nsf.muon_profile_begin()
    nsf.muon_grad_norm([t], 1.0, clip, tensor_norms=torch.zeros(1, device="cuda"))
    nsf.muon_grad_norm([t], 1.0, clip)
    nsf.muon_grad_norm([long], 1.0, clip)
    nsf.muon_clip_finish(clip, 1.0)
    nsf.muon_clip_grads([t], clip)
    nsf.muon_adamw(z[0], t, z[1], z[2], [(0, 100)], table, clip=clip)
    got = {k: n for k, (_, n) in nsf.muon_profile_end().items()}
    assert got == {"grad_norm": 2, "tensor_norms": 1, "norm_solo": 1, "norm_finish": 1,
                   "clip_finish": 1, "clip": 1, "adamw": 1}


# ---------------------------------------------------------- past 32 bits

def test_past_two_to_the_31(nsf, torch):
    """bfloat16 and float32 tensors of more than 2^31 elements: values at their very
    ends and at 2^31 reach the norm, and are clipped in place."""
    say("past 2^31")
    n = (1 << 31) + 8192 * 3 + 5
    for dt in (torch.bfloat16, torch.float32):
        t = torch.zeros(n, dtype=dt, device="cuda")
        at = [0, (1 << 31) - 1, 1 << 31, (1 << 31) + 1, n - 1]
        for k, i in enumerate(at):
            t[i] = float(k + 1)
        clip = nsf.clip_state("cuda")
        nsf.muon_grad_norm([t], 1.0, clip)
        assert read(nsf, clip)[0] == 55.0
        nsf.clip_coef(clip).fill_(0.5)
        nsf.muon_clip_grads([t], clip)
        assert [float(t[i]) for i in at] == [0.5, 1.0, 1.5, 2.0, 2.5]
        assert int(torch.count_nonzero(t[: 1 << 30])) + int(torch.count_nonzero(t[1 << 30:])) == 5
        del t


def test_adamw_past_two_to_the_31(nsf, torch):
    """Ranges that begin beyond 2^31 and one that spans it, against the chain at
    sampled places."""
    say("adamw past 2^31")
    size = (1 << 31) + 40000
    w = torch.zeros(size, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(size, dtype=torch.bfloat16, device="cuda")
    m, v = torch.zeros(size, device="cuda"), torch.zeros(size, device="cuda")
    ranges = [(0, (1 << 31) + 13, 0, 0), ((1 << 31) + 16, 39000, (1 << 31) + 16, 1)]
    spots = [0, 2047, 2048, (1 << 31) - 64, (1 << 31) + 16, (1 << 31) + 30000]
    gen = torch.Generator(device="cuda").manual_seed(5)
    for i in spots:
        for x, std in ((w, 0.05), (g, 0.1), (m, 0.03)):
            x[i:i + 64] = (torch.randn(64, generator=gen, device="cuda") * std).to(x.dtype)
        v[i:i + 64] = torch.rand(64, generator=gen, device="cuda") + 0.01
    part = {i: [host(x[i:i + 64]).copy() for x in (w, g, m, v)] for i in spots}
    nsf.muon_adamw(w, g, m, v, ranges, nsf.adamw_group_table(GROUPS, "cuda"))
    torch.cuda.synchronize()
    for i, (wb, gb, mb, vb) in part.items():
        want = [a.copy() for a in (wb, mb, vb)]
        for off, n, _, grp in ranges:
            lo, hi = max(off - i, 0), min(off + n - i, 64)
            if lo < hi:
                s = slice(lo, hi)
                want[0][s], want[1][s], want[2][s] = ao.adamw_same_order(wb[s], gb[s], mb[s], vb[s],
                                                                         GROUPS[grp])
        for x, ref in zip((w, m, v), want):
            assert np.array_equal(bits(host(x[i:i + 64])), bits(ref)), i
