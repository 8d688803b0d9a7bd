"""Host-side tests of the 8-bit casts, products and stacks: every refusal of the C ABI (none
of these calls reaches a HIP call), the binding's own checks, and the pins of their oracle."""

import ctypes
import os

import numpy as np
import pytest

import newton_schulz_flat_amd as nsf
from oracle import fp8_oracle as fo

ERR = {"OK": 0, "NULL_POINTER": -1, "BAD_SHAPE": -2, "MISALIGNED": -4, "OVERLAP": -5, "ALIAS": -6,
       "BAD_ARG": -7, "WORKSPACE_TOO_SMALL": -8}
F32, BF16 = 0, 1
# fake device addresses, compared as integers and never dereferenced
A, B, C, D, E, G, W = (k * 0x10_0000_0000 for k in range(1, 8))
FIELDS = ("codes", "scales", "rows", "cols", "row_stride", "scale_row", "scale_col", "format",
          "block_rows")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(nsf.LIB_PATH):
        from newton_schulz_flat_amd import build
        build.build()
    return nsf.load_library()


def fp8(codes=A, scales=B, rows=256, cols=512, row_stride=None, scale_row=1, scale_col=None, format=0,
        block_rows=1):
    return nsf.Fp8C(codes, scales, rows, cols, cols if row_stride is None else row_stride, scale_row,
                    max(1, rows) if scale_col is None else scale_col, format, block_rows)


def stack(src=A, dst=B, count=2, rows=30, cols=40, in_stride=1200, in_row=40, out_stride=1200,
          out_row=40, in_dtype=F32, out_dtype=F32):
    return nsf.StackC(src, dst, count, rows, cols, in_stride, in_row, out_stride, out_row, in_dtype,
                      out_dtype)


def cast(lib, out, out_t=None, x=C, dtype=F32, rows=256, cols=512, row_stride=512):
    return lib.muon_fp8_cast(x, dtype, rows, cols, row_stride, None if out is None else ctypes.byref(out),
                             None if out_t is None else ctypes.byref(out_t), None)


def product(lib, a, b, out=G, dtype=BF16, stride=None, accumulate=0, ws=W, ws_bytes=1 << 40):
    stride = (0 if b is None else b.rows) if stride is None else stride
    return lib.muon_fp8_matmul(None if a is None else ctypes.byref(a), None if b is None else ctypes.byref(b),
                               out, dtype, stride, accumulate, ws, ws_bytes, None)


def ortho(lib, s, steps=nsf.QUINTIC, n=None, scale=1.0, ws=W, ws_bytes=1 << 40, coefs=True):
    flat = (ctypes.c_float * max(1, 3 * len(steps)))(*[v for c in steps for v in c])
    return lib.muon_orthogonalize_stack(None if s is None else ctypes.byref(s), flat if coefs else None,
                                        len(steps) if n is None else n, scale, ws, ws_bytes, None)


def test_structs_have_the_header_sizes():
    assert ctypes.sizeof(nsf.Fp8C) == 64
    assert ctypes.sizeof(nsf.StackC) == 80


@pytest.mark.parametrize("change,code", [
    ({"format": 2}, "BAD_ARG"), ({"format": -1}, "BAD_ARG"), ({"block_rows": 64}, "BAD_ARG"),
    ({"block_rows": 0}, "BAD_ARG"), ({"codes": None}, "NULL_POINTER"), ({"scales": None}, "NULL_POINTER"),
    ({"scales": B + 2}, "MISALIGNED"), ({"row_stride": 511}, "BAD_SHAPE"),
    ({"row_stride": -512}, "BAD_SHAPE"), ({"row_stride": (1 << 26) + 1}, "BAD_SHAPE"),
    ({"scale_row": 0}, "BAD_SHAPE"), ({"scale_col": 0}, "BAD_SHAPE"), ({"scale_col": 255}, "BAD_SHAPE"),
    ({"scale_row": 3, "scale_col": 1}, "BAD_SHAPE"), ({"scale_row": -1}, "BAD_SHAPE"),
    ({"scale_col": 1 << 33}, "BAD_SHAPE"), ({"rows": -1}, "BAD_SHAPE"),
    ({"rows": (1 << 24) + 1, "cols": 4}, "BAD_SHAPE"), ({"rows": 1 << 20, "cols": 1 << 15}, "BAD_SHAPE"),
])
def test_matrices_are_checked(lib, change, code):
    bad = fp8(**change)
    assert cast(lib, bad, rows=bad.rows, cols=bad.cols, row_stride=max(1, bad.cols)) == ERR[code]
    assert cast(lib, None, bad, rows=bad.cols, cols=bad.rows, row_stride=max(1, bad.rows)) == ERR[code]
    assert product(lib, bad, fp8(codes=D, scales=E)) == ERR[code]
    assert product(lib, fp8(codes=D, scales=E), bad) == ERR[code]
    assert lib.muon_last_error() != b""


def test_casts_are_checked(lib):
    ok = fp8()
    assert cast(lib, None) == ERR["NULL_POINTER"]
    assert cast(lib, ok, dtype=2) == ERR["BAD_ARG"]
    assert cast(lib, ok, x=None) == ERR["NULL_POINTER"]
    assert cast(lib, ok, x=C + 2) == ERR["MISALIGNED"]
    assert cast(lib, ok, x=C + 1, dtype=BF16) == ERR["MISALIGNED"]
    assert cast(lib, ok, row_stride=500) == ERR["BAD_SHAPE"]
    assert cast(lib, ok, rows=255) == ERR["BAD_SHAPE"]
    assert cast(lib, ok, cols=513, row_stride=513) == ERR["BAD_SHAPE"]
    assert cast(lib, ok, rows=-1) == ERR["BAD_SHAPE"]
    turned = dict(codes=D, scales=E, rows=512, cols=256)
    assert cast(lib, ok, fp8(**{**turned, "rows": 256})) == ERR["BAD_SHAPE"]
    assert cast(lib, ok, fp8(**turned, format=1)) == ERR["BAD_ARG"]
    assert cast(lib, ok, fp8(**turned, block_rows=128)) == ERR["BAD_ARG"]
    # x, codes and scales lie apart
    assert cast(lib, ok, x=A) == ERR["ALIAS"]
    assert cast(lib, ok, x=B) == ERR["ALIAS"]
    assert cast(lib, ok, fp8(**{**turned, "codes": A + 256 * 512 - 1})) == ERR["ALIAS"]
    assert cast(lib, ok, fp8(**{**turned, "scales": B})) == ERR["ALIAS"]
    assert cast(lib, fp8(scales=A)) == ERR["ALIAS"]
    # nothing to do
    assert cast(lib, fp8(rows=0, codes=None, scales=None), rows=0, x=None) == ERR["OK"]
    assert cast(lib, fp8(cols=0, codes=None, scales=None), cols=0, x=None) == ERR["OK"]


def test_products_are_checked(lib):
    a, b = fp8(), fp8(codes=C, scales=D, rows=384)
    assert product(lib, None, b) == ERR["NULL_POINTER"]
    assert product(lib, a, None) == ERR["NULL_POINTER"]
    assert product(lib, a, fp8(codes=C, scales=D, cols=511)) == ERR["BAD_SHAPE"]
    assert product(lib, a, b, dtype=2) == ERR["BAD_ARG"]
    assert product(lib, a, b, accumulate=1) == ERR["BAD_ARG"]
    assert product(lib, a, b, dtype=F32, accumulate=2) == ERR["BAD_ARG"]
    assert product(lib, a, b, out=None) == ERR["NULL_POINTER"]
    assert product(lib, a, b, out=G + 1) == ERR["MISALIGNED"]
    assert product(lib, a, b, dtype=F32, out=G + 2) == ERR["MISALIGNED"]
    assert product(lib, a, b, stride=383) == ERR["BAD_SHAPE"]
    for where in (A, B, C, D):
        assert product(lib, a, b, out=where) == ERR["ALIAS"]
    assert product(lib, a, b, out=C - 256 * 384 * 2 + 2) == ERR["ALIAS"]
    wide = dict(cols=1, row_stride=1, scale_row=1, scale_col=1)
    assert product(lib, fp8(rows=1 << 20, **wide), fp8(codes=C, scales=D, rows=(1 << 16) + 1, **wide),
                   stride=1 << 17) == ERR["BAD_SHAPE"]
    # nothing to do
    assert product(lib, fp8(rows=0, codes=None, scales=None), b, out=None) == ERR["OK"]
    assert product(lib, a, fp8(rows=0, codes=None, scales=None), out=None) == ERR["OK"]


def test_product_workspace(lib):
    out = ctypes.c_size_t(7)
    assert lib.muon_fp8_workspace_bytes(1, 4096, 4096, None) == ERR["NULL_POINTER"]
    for bad in ((-1, 1, 1), (1, 1 << 25, 1), (1, 1, -5), (1 << 20, 4, 1 << 20)):
        assert lib.muon_fp8_workspace_bytes(*bad, ctypes.byref(out)) == ERR["BAD_SHAPE"]
    sizes = [(m, n, k) for m in (1, 5, 16, 100, 300, 4096) for n in (1, 128, 1000, 4096) for k in
             (0, 1, 128, 7168, 100000)]
    needs = {}
    for size in sizes:
        assert lib.muon_fp8_workspace_bytes(*size, ctypes.byref(out)) == 0
        needs[size] = out.value
        assert out.value % 256 == 0
    for (m, n, k), need in needs.items():
        if need == 0 or m == 0:
            continue
        a, b = fp8(rows=m, cols=k), fp8(codes=C, scales=D, rows=n, cols=k)
        assert product(lib, a, b, ws_bytes=need - 1) == ERR["WORKSPACE_TOO_SMALL"]
        assert product(lib, a, b, ws=None) == ERR["NULL_POINTER"]
        assert product(lib, a, b, ws=W + 16) == ERR["MISALIGNED"]
        assert product(lib, a, b, ws=G) == ERR["ALIAS"]
        assert product(lib, a, b, ws=A) == ERR["ALIAS"]


@pytest.mark.parametrize("change,code", [
    ({"count": -1}, "BAD_ARG"), ({"count": (1 << 20) + 1}, "BAD_ARG"), ({"rows": 0}, "BAD_SHAPE"),
    ({"cols": 0}, "BAD_SHAPE"), ({"rows": (1 << 20) + 1}, "BAD_SHAPE"),
    ({"rows": 1 << 16, "cols": 1 << 16}, "BAD_SHAPE"), ({"in_dtype": 2}, "BAD_ARG"),
    ({"out_dtype": -1}, "BAD_ARG"), ({"in_row": 39}, "BAD_SHAPE"), ({"out_row": 39}, "BAD_SHAPE"),
    ({"in_row": -40}, "BAD_SHAPE"), ({"in_stride": -1}, "BAD_SHAPE"), ({"out_stride": -1}, "BAD_SHAPE"),
    ({"out_stride": (1 << 40) + 1}, "BAD_SHAPE"), ({"out_stride": 1199}, "OVERLAP"),
    ({"out_stride": 0}, "OVERLAP"), ({"out_stride": 39, "out_row": 400}, "OVERLAP"),
    ({"out_stride": 41, "out_row": 80}, "OVERLAP"), ({"src": None}, "NULL_POINTER"),
    ({"dst": None}, "NULL_POINTER"), ({"src": A + 2}, "MISALIGNED"), ({"dst": B + 1, "out_dtype": BF16},
                                                                      "MISALIGNED"),
    ({"dst": A}, "ALIAS"), ({"dst": A + 2399 * 4}, "ALIAS"), ({"src": W}, "ALIAS"), ({"dst": W + 4096}, "ALIAS"),
])
def test_stacks_are_checked(lib, change, code):
    assert ortho(lib, stack(**change)) == ERR[code]


def test_stack_arguments_are_checked(lib):
    s = stack()
    out = ctypes.c_size_t(0)
    assert lib.muon_stack_workspace_bytes(None, ctypes.byref(out)) == ERR["NULL_POINTER"]
    assert lib.muon_stack_workspace_bytes(ctypes.byref(s), None) == ERR["NULL_POINTER"]
    assert lib.muon_stack_workspace_bytes(ctypes.byref(s), ctypes.byref(out)) == 0
    two = out.value
    assert lib.muon_stack_workspace_bytes(ctypes.byref(stack(count=1)), ctypes.byref(out)) == 0
    assert two == 2 * out.value and out.value % 256 == 0
    assert ortho(lib, None) == ERR["NULL_POINTER"]
    assert ortho(lib, s, coefs=False) == ERR["NULL_POINTER"]
    assert ortho(lib, s, n=-1) == ERR["BAD_ARG"]
    assert ortho(lib, s, steps=[(1.0, 0.0, 0.0)] * 65) == ERR["BAD_ARG"]
    for bad in (float("nan"), float("inf")):
        assert ortho(lib, s, scale=bad) == ERR["BAD_ARG"]
        for k in range(3):
            c = [1.0, 0.0, 0.0]
            c[k] = bad
            assert ortho(lib, s, steps=[(1.0, 0.0, 0.0), tuple(c)]) == ERR["BAD_ARG"]
    # 9.9 a step: 9.9^7 is below 2^24, 9.9^8 is not
    assert ortho(lib, stack(count=0), steps=[(9.9, 0.0, 0.0)] * 7) == ERR["OK"]
    assert ortho(lib, stack(count=0), steps=[(9.9, 0.0, 0.0)] * 8) == ERR["BAD_ARG"]
    # between the ends: 30 x - 29 x^3 is 1 at x = 1 but 11.7 at x = 0.59
    grows = [(30.0, -29.0, 0.0), (1e6, 0.0, 0.0)]
    assert ortho(lib, stack(count=0), steps=grows + [(1.0, 0.0, 0.0)]) == ERR["OK"]
    assert ortho(lib, stack(count=0), steps=[(30.0, -29.0, 0.0), (1.5e6, 0.0, 0.0)]) == ERR["BAD_ARG"]
    assert ortho(lib, s, ws=None) == ERR["NULL_POINTER"]
    assert ortho(lib, s, ws=W + 8) == ERR["MISALIGNED"]
    assert ortho(lib, s, ws_bytes=out.value - 1) == ERR["WORKSPACE_TOO_SMALL"]
    assert ortho(lib, stack(count=0, src=None, dst=None), ws=None, ws_bytes=0) == ERR["OK"]


def test_binding_refuses_host_tensors_and_wrong_types():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 128)
    q, s = torch.zeros(4, 128, dtype=torch.float8_e4m3fn), torch.zeros(4, 1)
    with pytest.raises(ValueError, match="GPU tensor"):
        nsf.muon_fp8_cast(x, q, s)
    with pytest.raises(TypeError, match="must be a torch.Tensor"):
        nsf.muon_fp8_cast([1.0], q, s)
    with pytest.raises(ValueError, match="GPU tensor"):
        nsf.muon_fp8_matmul(q, s, q, s, x)
    with pytest.raises(ValueError, match="GPU tensor"):
        nsf.muon_orthogonalize_stack(x, x)
    with pytest.raises(ValueError, match="GPU tensor"):
        nsf.muon_stack_workspace_bytes(x)
    with pytest.raises(ValueError, match="'row' or 'square'"):
        nsf.fp8_scales(4, 4, "column", "cpu")


def test_scale_tensors_have_the_shape_and_order_of_blocks():
    assert nsf.fp8_scales(300, 1000, "row", "cpu").shape == (300, 8)
    assert nsf.fp8_scales(300, 1000, "row", "cpu").stride() == (1, 300)
    assert nsf.fp8_scales(300, 1000, "square", "cpu").shape == (3, 8)
    assert nsf.fp8_scales(0, 5, "square", "cpu").shape == (0, 1)


# ------------------------------------------------------------- the oracle's pins

@pytest.mark.parametrize("fmt,name", [("e4m3", "float8_e4m3fn"), ("e5m2", "float8_e5m2")])
def test_oracle_numbers_and_rounding(fmt, name):
    torch = pytest.importorskip("torch")
    v = fo.numbers(fmt)
    codes = np.arange(len(v), dtype=np.uint8)
    t = torch.from_numpy(codes).view(getattr(torch, name)).double().numpy()
    assert np.array_equal(v, t)
    assert v[1] == (2.0 ** -9 if fmt == "e4m3" else 2.0 ** -16) and v[-1] == (448 if fmt == "e4m3" else 57344)
    assert np.array_equal(fo.encode(v, fmt), codes) and np.array_equal(fo.encode(-v, fmt), codes | 0x80)
    # ties go to the even code, everything else to the nearest
    middle = (v[1:] + v[:-1]) / 2
    low = codes[:-1]
    assert np.array_equal(fo.encode(middle, fmt), np.where(low % 2 == 0, low, low + 1))
    assert np.array_equal(fo.encode(np.nextafter(middle, 0), fmt), low)
    assert np.array_equal(fo.encode(np.nextafter(middle, np.inf), fmt), low + 1)


def test_oracle_cast_by_hand():
    x = np.zeros((130, 129), np.float32)
    x[0, :3] = [448.0, 1.0, -17.0]       # scale 1: 17 lies between 16 and 18
    x[1, :2] = [896.0, 3.0]              # scale 2
    x[129, 128] = 2.0 ** -110            # below the floor 2^-100
    codes, scales = fo.cast(x, "e4m3", False)
    assert scales[0, 0] == 1 and scales[1, 0] == 2 and scales[129, 1] == np.float32(2.0 ** -100) / 448
    back = fo.widen(codes, scales, "e4m3")
    assert back[0, :3].tolist() == [448.0, 1.0, -16.0] and back[1, :2].tolist() == [896.0, 3.0]
    square, s2 = fo.cast(x, "e4m3", True)
    assert s2.shape == (2, 2) and s2[0, 0] == 2
    assert fo.widen(square, s2, "e4m3")[0, :3].tolist() == [448.0, 1.0, -16.0]


def test_oracle_iteration_against_singular_values():
    rng = np.random.default_rng(0)
    for rows, cols in ((6, 9), (9, 6), (5, 5), (1, 7)):
        u = rng.standard_normal((rows, cols))
        p, s, q = np.linalg.svd(u, full_matrices=False)
        s = s / (np.linalg.norm(s) + 1e-7)
        for a, b, c in nsf.QUINTIC:
            a, b, c = (float(np.float32(v)) for v in (a, b, c))
            s = a * s + b * s ** 3 + c * s ** 5
        want = (p * s) @ q
        got = fo.newton_schulz(u, nsf.QUINTIC)
        assert np.linalg.norm(got - want) <= 1e-13 * np.linalg.norm(want)
        # a planted mistake is seen
        wrong = fo.newton_schulz(u, [(3.4445, -4.7750, 2.0316)] * 5)
        assert np.linalg.norm(wrong - want) > 1e-6 * np.linalg.norm(want)


def test_oracle_product_bound_sees_a_lost_block():
    rng = np.random.default_rng(1)
    a, b = rng.standard_normal((3, 300)), rng.standard_normal((4, 300))
    cut = a.copy()
    cut[:, 256:] = 0
    assert (np.abs((a - cut) @ b.T) > fo.product_bound(a, b) + fo.cut_bound(a, b)).mean() > 0.8
