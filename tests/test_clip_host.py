"""Host-side tests of the gradient norm, clipping and AdamW: every refusal of
the C ABI (none of these calls reaches a HIP call), workspace sizes, the
binding's own checks, and the pins of their oracles."""

import ctypes
import fractions
import math
import os

import numpy as np
import pytest

import newton_schulz_flat_amd as nsf
from oracle import adamw_oracle as ao
from oracle import same_order as so

ERR = {"NULL_POINTER": -1, "BAD_SHAPE": -2, "OUT_OF_BOUNDS": -3, "MISALIGNED": -4, "OVERLAP": -5,
       "ALIAS": -6, "BAD_ARG": -7, "WORKSPACE_TOO_SMALL": -8}
F32, BF16 = 0, 1
# fake device addresses, compared as integers and never dereferenced
A, B, C, D, E, G, W = (k * 0x10_0000_0000 for k in range(1, 8))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(nsf.LIB_PATH):
        from newton_schulz_flat_amd import build
        build.build()
    return nsf.load_library()


def tensors(*items):
    arr = (nsf.TensorC * max(1, len(items)))()
    for k, (ptr, numel, dtype) in enumerate(items):
        arr[k] = nsf.TensorC(ptr, numel, dtype, 0)
    return arr


def need(lib, *items):
    out = ctypes.c_size_t(0)
    rc = lib.muon_clip_workspace_bytes(tensors(*items), len(items), ctypes.byref(out))
    return rc, out.value


def test_structs_have_the_header_sizes():
    assert ctypes.sizeof(nsf.TensorC) == 24
    assert ctypes.sizeof(nsf.RangeC) == 32


def test_workspace_bytes(lib):
    assert need(lib) == (0, 0)
    rc, one = need(lib, (A, 1, F32))
    assert rc == 0 and one == 256
    # lengths alone decide: neither address nor type
    many = [(A + 4096 * k, 1000, F32) for k in range(700)]
    other = [(B + 2 + 4096 * k, 1000, BF16) for k in range(700)]
    assert need(lib, *many) == need(lib, *other)
    assert need(lib, *many)[1] >= 700 * 8
    # one partial for each workgroup and tensor, not one for each piece of a long tensor
    rc, long = need(lib, (A, 1 << 34, F32))
    assert rc == 0 and long < 1 << 20
    assert lib.muon_clip_workspace_bytes(tensors((A, 1, F32)), 1, None) == ERR["NULL_POINTER"]


@pytest.mark.parametrize("items,code", [
    ([(A, 4, 2)], "BAD_ARG"),
    ([(A, 4, -1)], "BAD_ARG"),
    ([(A, -1, F32)], "BAD_SHAPE"),
    ([(A, (1 << 34) + 1, F32)], "BAD_SHAPE"),
    ([(A + (k << 36), 1 << 34, F32) for k in range(4)] + [(W, 1, F32)], "BAD_SHAPE"),
    ([(None, 4, F32)], "NULL_POINTER"),
    ([(A + 2, 4, F32)], "MISALIGNED"),
    ([(A + 1, 4, BF16)], "MISALIGNED"),
])
def test_tensor_lists_are_checked(lib, items, code):
    assert need(lib, *items)[0] == ERR[code]
    arr, n = tensors(*items), len(items)
    assert lib.muon_grad_norm(arr, n, 1.0, C, None, D, 1 << 20, None) == ERR[code]
    assert lib.muon_clip_grads(arr, arr, n, C, None) == ERR[code]
    assert lib.muon_last_error() != b""


def test_counts_and_lists(lib):
    arr = tensors((A, 4, F32))
    for n, code in ((-1, "BAD_ARG"), ((1 << 24) + 1, "BAD_ARG")):
        assert lib.muon_grad_norm(arr, n, 1.0, C, None, D, 1 << 20, None) == ERR[code]
        assert lib.muon_clip_grads(arr, arr, n, C, None) == ERR[code]
    assert lib.muon_grad_norm(None, 1, 1.0, C, None, D, 1 << 20, None) == ERR["NULL_POINTER"]
    assert lib.muon_clip_grads(None, arr, 1, C, None) == ERR["NULL_POINTER"]
    assert lib.muon_clip_grads(arr, None, 1, C, None) == ERR["NULL_POINTER"]
    assert lib.muon_clip_grads(None, None, 0, None, None) == 0  # nothing to do


@pytest.mark.parametrize("kw,code", [
    (dict(max_norm=-1.0), "BAD_ARG"),
    (dict(max_norm=math.nan), "BAD_ARG"),
    (dict(clip=None), "NULL_POINTER"),
    (dict(clip=C + 8), "MISALIGNED"),
    (dict(norms=E + 2), "MISALIGNED"),
    (dict(ws=None), "NULL_POINTER"),
    (dict(ws=D + 128), "MISALIGNED"),
    (dict(ws_bytes=255), "WORKSPACE_TOO_SMALL"),
    (dict(clip=A + 16), "ALIAS"),           # the record inside a tensor
    (dict(norms=A + 4 * 99), "ALIAS"),
    (dict(ws=A - 256 + 256), "ALIAS"),
    (dict(norms=C + 12), "ALIAS"),          # the norms over the record
    (dict(clip=D + 64), "ALIAS"),           # the record in the workspace
])
def test_grad_norm_refuses(lib, kw, code):
    a = dict(max_norm=1.0, clip=C, norms=E, ws=D, ws_bytes=256)
    a.update(kw)
    rc = lib.muon_grad_norm(tensors((A, 100, F32)), 1, a["max_norm"], a["clip"], a["norms"],
                            a["ws"], a["ws_bytes"], None)
    assert rc == ERR[code], lib.muon_last_error()


def test_clip_finish_refuses(lib):
    assert lib.muon_clip_finish(None, 1.0, None) == ERR["NULL_POINTER"]
    assert lib.muon_clip_finish(C + 4, 1.0, None) == ERR["MISALIGNED"]
    assert lib.muon_clip_finish(C, math.nan, None) == ERR["BAD_ARG"]


@pytest.mark.parametrize("src,dst,code", [
    ([(A, 8, F32)], [(A, 8, BF16)], "ALIAS"),                 # in place, but another type
    ([(A, 8, F32)], [(A + 4, 8, F32)], "ALIAS"),              # shifted
    ([(A, 8, F32)], [(B, 7, F32)], "BAD_SHAPE"),
    ([(A, 8, F32), (B, 8, F32)], [(D, 8, F32), (D + 28, 8, F32)], "OVERLAP"),
    ([(A, 8, F32), (A, 8, F32)], [(A, 8, F32), (A, 8, F32)], "OVERLAP"),   # the same one twice
    ([(A, 8, F32), (B, 8, F32)], [(B, 8, F32), (A, 8, F32)], "ALIAS"),     # crosswise
    ([(A, 800, F32), (A + 8, 2, F32), (B, 8, F32)],
     [(D, 800, F32), (E, 2, F32), (A + 3000, 8, F32)], "ALIAS"),  # behind a short source
    ([(A, 8, F32)], [(C - 16, 8, F32)], "ALIAS"),             # over the record
])
def test_clip_grads_refuses(lib, src, dst, code):
    rc = lib.muon_clip_grads(tensors(*src), tensors(*dst), len(src), C, None)
    assert rc == ERR[code], lib.muon_last_error()


def test_clip_grads_needs_a_record(lib):
    arr = tensors((A, 8, F32))
    assert lib.muon_clip_grads(arr, arr, 1, None, None) == ERR["NULL_POINTER"]
    assert lib.muon_clip_grads(arr, arr, 1, C + 8, None) == ERR["MISALIGNED"]


def adamw(lib, ranges, *, params=A, pdt=F32, n_params=1 << 20, copy=None, grads=B, gdt=F32, m=C,
          v=D, n_state=1 << 20, groups=E, n_groups=2, clip=G):
    arr = nsf.ranges_array(ranges)
    return lib.muon_adamw(params, pdt, n_params, copy, grads, gdt, m, v, n_state, arr, len(arr),
                          groups, n_groups, clip, None)


@pytest.mark.parametrize("kw,code", [
    (dict(params=None), "NULL_POINTER"),
    (dict(grads=None), "NULL_POINTER"),
    (dict(m=None), "NULL_POINTER"),
    (dict(v=None), "NULL_POINTER"),
    (dict(groups=None), "NULL_POINTER"),
    (dict(params=A + 4), "MISALIGNED"),
    (dict(grads=B + 8), "MISALIGNED"),
    (dict(m=C + 4), "MISALIGNED"),
    (dict(v=D + 4), "MISALIGNED"),
    (dict(groups=E + 4), "MISALIGNED"),
    (dict(clip=G + 8), "MISALIGNED"),
    (dict(copy=W + 2), "MISALIGNED"),
    (dict(pdt=2), "BAD_ARG"),
    (dict(gdt=3), "BAD_ARG"),
    (dict(pdt=BF16, copy=W), "BAD_ARG"),
    (dict(n_groups=0), "BAD_ARG"),
    (dict(n_groups=65537), "BAD_ARG"),
    (dict(n_state=-1), "BAD_ARG"),
    (dict(n_state=99), "OUT_OF_BOUNDS"),
    (dict(n_params=99), "OUT_OF_BOUNDS"),
    (dict(m=B + 400), "ALIAS"),
    (dict(v=C), "ALIAS"),
    (dict(grads=A), "ALIAS"),
    (dict(copy=A + 16), "ALIAS"),
    (dict(clip=C + 16), "ALIAS"),
    (dict(groups=D + 8), "ALIAS"),
])
def test_adamw_refuses(lib, kw, code):
    assert adamw(lib, [(0, 100, 0, 1)], **kw) == ERR[code], lib.muon_last_error()


@pytest.mark.parametrize("ranges,kw,code", [
    ([(0, -1)], {}, "BAD_SHAPE"),
    ([(0, (1 << 34) + 1)], {}, "BAD_SHAPE"),
    ([(1 << 36, 8, 0)], dict(n_state=1 << 37), "BAD_SHAPE"),
    ([(0, 8, 1 << 36)], dict(n_params=1 << 37), "BAD_SHAPE"),
    ([(2, 8, 0)], {}, "MISALIGNED"),
    ([(0, 8, 2)], {}, "MISALIGNED"),
    ([(4, 8, 4)], dict(pdt=BF16), "MISALIGNED"),
    ([(-4, 8, 0)], {}, "OUT_OF_BOUNDS"),
    ([(0, 8, -4)], {}, "OUT_OF_BOUNDS"),
    ([(0, 8, 0, 2)], {}, "BAD_ARG"),
    ([(0, 8, 0, -1)], {}, "BAD_ARG"),
    ([(0, 8, 0), (4, 8, 100)], {}, "OVERLAP"),
    ([(0, 8, 0), (100, 8, 4)], {}, "OVERLAP"),
    ([(0, 8), (0, 8)], {}, "OVERLAP"),
])
def test_adamw_refuses_ranges(lib, ranges, kw, code):
    assert adamw(lib, ranges, **kw) == ERR[code], lib.muon_last_error()


def test_adamw_with_nothing_to_do(lib):
    empty = dict(params=None, grads=None, m=None, v=None, groups=None, clip=None, n_state=0,
                 n_params=0)
    assert adamw(lib, [], **empty) == 0
    assert adamw(lib, [(0, 0), (0, 0)], **empty) == 0


def test_step_clipped_refuses(lib):
    arr = nsf.descs_array([(0, 64, 32)])

    def call(clip=G, groups=E, n_groups=1, ws=W):
        return lib.muon_step_clipped(A, 0, 1 << 20, None, B, C, 1 << 20, arr, 1, groups, n_groups,
                                     clip, 5, 0, ws, 1 << 30, None)
    assert call(clip=None) == ERR["NULL_POINTER"]
    assert call(clip=G + 8) == ERR["MISALIGNED"]
    assert call(clip=C + 64) == ERR["ALIAS"]
    assert call(clip=W + 64) == ERR["ALIAS"]
    assert call(groups=None) == ERR["NULL_POINTER"]
    assert call(n_groups=0) == ERR["BAD_ARG"]
    assert call(ws=None) == ERR["NULL_POINTER"]
    # no matrices: nothing is needed
    assert lib.muon_step_clipped(None, 0, 0, None, None, None, 0, arr, 0, None, 1, None, 5, 0, None,
                                 0, None) == 0


def test_binding_refuses_host_tensors():
    import torch
    clip = nsf.clip_state("cpu")
    t = torch.zeros(8)
    for call in (lambda: nsf.tensor_list([t]), lambda: nsf.muon_grad_norm([t], 1.0, clip),
                 lambda: nsf.muon_clip_grads([t], clip), lambda: nsf.muon_clip_finish(clip, 1.0),
                 lambda: nsf.muon_adamw(t, t, t, t, [(0, 8)], None)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_binding_tables():
    import torch
    tab = nsf.adamw_group_table([(1e-3, 0.1, 0.9, 0.999, 1e-8), (1, 2, 3, 4, 5, 7)], "cpu")
    assert tab.shape == (2, 4) and tab.dtype == torch.int64
    assert nsf.adamw_steps(tab).tolist() == [1, 7]
    f = tab.view(torch.float32)
    assert f[0, :5].tolist() == [float(np.float32(x)) for x in (1e-3, 0.1, 0.9, 0.999, 1e-8)]
    with pytest.raises(ValueError):
        nsf.adamw_group_table([(1, 2, 3)], "cpu")
    arr = nsf.ranges_array([(4, 8), (16, 3, 32, 1)])
    assert nsf.ranges_array(arr) is arr
    assert [(r.offset, r.numel, r.param_offset, r.group) for r in arr] == [(4, 8, 4, 0), (16, 3, 32, 1)]
    clip = nsf.clip_state("cpu")
    clip.sumsq[0] = 9.0
    nsf.clip_norm(clip).fill_(3.0)
    nsf.clip_coef(clip).fill_(0.5)
    assert nsf.clip_sumsq(clip).tolist() == [9.0]
    raw = clip.record.numpy().view(np.float32)
    assert raw[2] == 3.0 and raw[3] == 0.5


# --------------------------------------------------------------- oracle pins

def test_oracle_sumsq_and_coefficient():
    a = np.array([3.0, 4.0], np.float32)
    assert ao.sumsq([a]) == 25.0
    # exact rational sum, rounded once
    rng = np.random.default_rng(3)
    x = (rng.standard_normal(200) * 10.0 ** rng.integers(-30, 30, 200)).astype(np.float32)
    want = float(sum(fractions.Fraction(float(v)) ** 2 for v in x))
    assert ao.sumsq([x[:77], x[77:]]) == want
    assert ao.coefficient(25.0, 1.0) == 1.0 / (5.0 + 1e-6)
    assert ao.coefficient(25.0, 6.0) == 1.0
    assert ao.coefficient(math.inf, 1.0) == 0.0
    assert math.isnan(ao.coefficient(math.nan, 1.0))


def adamw_pins(step):
    """Closed forms that a step function (w, g, m, v, group, coef) has to meet."""
    z = np.zeros(1, np.float64)
    one = np.ones(1, np.float64)
    # from zero state, the first update is lr * sign(g) up to eps, whatever the size of g
    for g in (1e-3, -7.0, 1e4):
        w, m, v = step(z, one * g, z, z, (0.5, 0.0, 0.875, 0.75, 0.0, 1), 1.0)
        assert abs(w[0] + 0.5 * math.copysign(1, g)) < 1e-12
        assert m[0] == 0.125 * g and v[0] == 0.25 * g * g
    # no gradient, no state: decay alone
    w, _, _ = step(one, z, z, z, (0.5, 0.25, 0.875, 0.75, 0.5, 3), 1.0)
    assert w[0] == 1 - 0.125
    # decay acts on the old weight alone: w (1 - lr wd) - lr sign(g)
    w, _, _ = step(one * 4, one, z, z, (0.5, 0.25, 0.875, 0.75, 0.0, 1), 1.0)
    assert abs(w[0] - (4 * 0.875 - 0.5)) < 1e-12
    # eps beside the root of the corrected moment: g / (|g| + eps)
    w, _, _ = step(z, one, z, z, (0.5, 0.0, 0.875, 0.75, 3.0, 1), 1.0)
    assert abs(w[0] + 0.5 / 4) < 1e-12
    # constant gradient: m and v are 1 - beta^t of g and g^2, so every step is lr * sign(g)
    w, m, v = z, z, z
    for t in range(1, 30):
        w, m, v = step(w, one * 2.0, m, v, (0.25, 0.0, 0.875, 0.75, 0.0, t), 0.5)
    assert abs(m[0] - (1 - 0.875 ** 29)) < 1e-12 and abs(v[0] - (1 - 0.75 ** 29)) < 1e-12
    assert abs(w[0] + 0.25 * 29) < 1e-12


def test_oracle_adamw_closed_forms():
    adamw_pins(ao.adamw)


def planted(mistake):
    def step(w, g, m, v, group, coef):
        lr, wd, b1, b2, eps, t = group
        raw = g
        if mistake != "coefficient dropped":
            g = g * coef
        if mistake == "decay in the gradient":
            g = g + wd * w
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * (raw if mistake == "coefficient once in v" else g) * g
        h = m / (1 - b1 ** (t - 1 if mistake == "step off by one" and t > 1 else t))
        if mistake == "m not corrected":
            h = m
        u = v if mistake == "v not corrected" else v / (1 - b2 ** t)
        root = np.sqrt(u + eps) if mistake == "eps in the root" else np.sqrt(u) + eps
        with np.errstate(all="ignore"):
            upd = np.nan_to_num(h / root)
        if mistake == "decay after the update":
            w = (w - lr * upd) * (1 - lr * wd)
        elif mistake == "decay without lr":
            w = w - wd * w - lr * upd
        elif mistake == "decay in the gradient":
            w = w - lr * upd
        elif mistake == "betas swapped":
            return planted("")(w, raw, m, v, (lr, wd, b2, b1, eps, t), coef)
        else:
            w = w - lr * wd * w - lr * upd
        return w, m, v
    return step


MISTAKES = ["coefficient dropped", "decay in the gradient", "coefficient once in v",
            "step off by one", "m not corrected", "v not corrected", "eps in the root",
            "decay after the update", "decay without lr", "betas swapped"]


@pytest.mark.parametrize("mistake", MISTAKES)
def test_oracle_adamw_pins_find_mistakes(mistake):
    adamw_pins(planted(""))
    with pytest.raises(AssertionError):
        adamw_pins(planted(mistake))


def test_oracle_same_order_is_near_the_definition():
    """Each of its values is within the roundings of its own chain.  m: two products
    and a sum, at most 3 half steps of the larger terms; v: one product more, and
    1 - beta2 exact (beta >= 1/2).  The update: m (3), v under a root (4/2 + 1), r, the
    sum with eps, the quotient, a, the product: below 12; the weight: decay
    factor (2), product, difference (and bfloat16's own)."""
    rng = np.random.default_rng(8)
    n = 20000
    w = rng.standard_normal(n).astype(np.float32)
    g = rng.standard_normal(n).astype(np.float32)
    m = rng.standard_normal(n).astype(np.float32)
    v = (rng.random(n) + 0.05).astype(np.float32)
    u = 2.0 ** -24
    for t in (1, 2, 1000, 10 ** 6):
        grp = (1e-2, 0.1, 0.9, 0.999, 1e-8, t)
        coef = np.float32(0.37)
        w1, m1, v1 = ao.adamw_same_order(w, g, m, v, grp, coef)
        W, M, V = ao.adamw(w, g, m, v, grp, float(coef))
        # terms before they cancel
        tm = 0.9 * abs(m) + 0.1 * 0.37 * abs(g)
        assert (abs(m1 - M) <= 4 * u * tm).all()
        assert (abs(v1 - V) <= 6 * u * V).all()
        upd = 1e-2 / (1 - 0.9 ** t) * tm / np.sqrt(V / (1 - 0.999 ** t))
        assert (abs(w1 - W) <= 14 * u * upd + 4 * u * abs(w) + u * abs(W)).all()
        wb, mb, vb = ao.adamw_same_order(so.f32_to_bf16_bits(w), g, m, v, grp, coef)
        assert wb.dtype == np.uint16 and np.array_equal(mb, m1) and np.array_equal(vb, v1)


def test_oracle_clip_rounds_once():
    x = np.array([1.0, -3.0, 1e-40, np.inf, np.nan], np.float32)
    c = np.float32(1 / 3)
    y = ao.clip_same_order(x, c, "f32")
    exact = [float(np.float32(float(c) * float(v))) for v in x[:4]]  # product exact in float64
    assert y[:4].tolist() == exact and np.isnan(y[4])
    assert np.array_equal(ao.clip_same_order(x, c, "bf16"), so.f32_to_bf16_bits(y))
