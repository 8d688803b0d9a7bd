"""GPU tests of the 8-bit casts and products.  Casts are held bit for bit against the float32
definition; products against float64 within the bound that counts their roundings."""

import numpy as np
import pytest

import newton_schulz_flat_amd as nsf
from oracle import fp8_oracle as fo
from tests.gpu_helpers import host, say

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

TYPES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def codes_of(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def values(rows, cols, dtype, seed, pad=0):
    """Numbers of very different sizes along rows and columns."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols + pad, generator=g)
    x *= torch.exp2(torch.randint(-12, 13, (rows, 1), generator=g).float())
    x *= torch.exp2(torch.randint(-4, 5, (1, cols + pad), generator=g).float())
    return x.to(DT[dtype]).cuda()[:, :cols]


def cast(x, fmt, block, both=True):
    rows, cols = x.shape
    out = [torch.zeros(a, b, dtype=TYPES[fmt], device="cuda") for a, b in ((rows, cols), (cols, rows))]
    sc = [nsf.fp8_scales(a, b, block, "cuda") for a, b in ((rows, cols), (cols, rows))]
    nsf.muon_fp8_cast(x, out[0], sc[0], *((out[1], sc[1]) if both else ()))
    return out, sc


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block", ["row", "square"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (1, 128, 0), (1, 4096, 0), (3, 127, 0), (128, 128, 0),
                                           (129, 257, 0), (7, 1000, 3), (300, 65, 1), (511, 384, 64)])
def test_cast_equals_the_definition(rows, cols, pad, dtype, block, fmt):
    say("cast", rows, cols, pad, dtype, block, fmt)
    x = values(rows, cols, dtype, rows * 1000 + cols, pad)
    (q, qt), (s, st) = cast(x, fmt, block)
    xh = x.float().cpu().numpy()
    for got, sc, want in ((q, s, fo.cast(xh, fmt, block == "square")),
                          (qt, st, fo.cast(xh.T, fmt, block == "square"))):
        assert np.array_equal(host(sc.contiguous()).view(np.uint32), want[1].view(np.uint32))
        assert np.array_equal(codes_of(got), want[0])
    # either side alone gives the same
    (q1, _), (s1, _) = cast(x, fmt, block, both=False)
    assert torch.equal(q1.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s1, s)
    only, sc = torch.zeros_like(qt), torch.zeros_like(st)
    nsf.muon_fp8_cast(x, codes_t=only, scales_t=sc)
    assert torch.equal(only.view(torch.uint8), qt.view(torch.uint8)) and torch.equal(sc, st)


@pytest.mark.parametrize("block", ["row", "square"])
def test_cast_ties_zeros_and_small_numbers(block):
    say("cast ties", block)
    v = fo.numbers("e4m3")
    x = np.zeros((128, 128), np.float32)
    middles = ((v[1:] + v[:-1]) / 2)[:120]
    x[0, :120] = middles           # every tie between neighbours
    x[0, 127] = 448.0              # a scale of one
    x[1, :] = 2.0 ** -120          # below the floor
    x[1, 0] = -2.0 ** -101
    x[2, :] = np.float32(1e-45)
    x[3, 5] = -0.0
    x[4, :] = np.float32(3.4028235e38)
    if block == "square":
        x[4, :] = 0.0
    t = torch.from_numpy(x).cuda()
    (q, qt), (s, st) = cast(t, "e4m3", block)
    for got, sc, m in ((q, s, x), (qt, st, x.T)):
        want = fo.cast(m, "e4m3", block == "square")
        assert np.array_equal(host(sc.contiguous()).view(np.uint32), want[1].view(np.uint32))
        assert np.array_equal(codes_of(got), want[0])


def test_cast_nan_and_infinity_stay_in_their_block():
    say("cast nan")
    x = values(200, 300, "f32", 5)
    clean, sc = cast(x, "e4m3", "row")
    x[7, 130] = float("nan")
    x[9, 3] = float("-inf")
    (q, _), (s, _) = cast(x, "e4m3", "row")
    assert torch.isnan(s[7, 1]) and torch.isinf(s[9, 0])
    keep = torch.ones_like(s, dtype=torch.bool)
    keep[7, 1] = keep[9, 0] = False
    assert torch.equal(s[keep], sc[0][keep])
    wide = keep.repeat_interleave(128, 1)[:, :300]
    assert torch.equal(q.view(torch.uint8)[wide], clean[0].view(torch.uint8)[wide])


def test_cast_writes_nothing_else():
    say("cast gaps")
    x = values(70, 90, "bf16", 8, pad=6)
    buf = torch.full((72, 128), 0x55, dtype=torch.uint8, device="cuda")
    q = buf.view(TYPES["e4m3"])[1:71, 5:95]
    held = torch.full((4, 100), -7.0, device="cuda")
    s = held[1:2, 3:73].t()
    nsf.muon_fp8_cast(x, q, s)
    want = fo.cast(x.float().cpu().numpy(), "e4m3", False)
    assert np.array_equal(codes_of(q), want[0]) and np.array_equal(host(s.contiguous()), want[1])
    buf[1:71, 5:95] = 0x55
    held[1:2, 3:73] = -7.0
    assert (buf == 0x55).all() and (held == -7.0).all()


def operand(rows, k, fmt, block, seed, pad=0):
    x = values(rows, k, "f32", seed)
    held = torch.full((rows, k + pad), 0x7F, dtype=torch.uint8, device="cuda").view(TYPES[fmt])[:, :k]
    s = nsf.fp8_scales(rows, k, block, "cuda")
    nsf.muon_fp8_cast(x, held, s)
    return held, s, fo.widen(codes_of(held), host(s.contiguous()), fmt)


def check_product(got, wa, wb, out, before=None):
    want = wa @ wb.T + (0 if before is None else before)
    bound = fo.product_bound(wa, wb)
    if before is not None:
        bound = bound + 2.0 ** -24 * np.abs(want) + 2.0 ** -24 * bound
    if out == "bf16":
        bound = bound + fo.cut_bound(wa, wb)
        bound = bound + 2.0 ** -8 * (np.abs(want) + bound)
        # as a whole the roundings of out stand above all else: half a step each, that is 2^-9
        # to 2^-8 of the value
        assert np.linalg.norm(got.double().cpu().numpy() - want) <= 2.0 ** -8 * np.linalg.norm(want)
    else:
        bound = bound + 2.0 ** -24 * np.abs(want)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= bound + 1e-300).all(), (err / (bound + 1e-300)).max()


SHAPES = [(1, 1, 1), (1, 64, 128), (1, 4096, 1000), (2, 130, 256), (16, 16, 16), (17, 33, 129),
          (64, 256, 512), (100, 300, 1999), (128, 128, 128), (129, 257, 384), (256, 512, 1024),
          (300, 1025, 272), (33, 2048, 7168), (513, 129, 96)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("blocks", [("row", "square"), ("row", "row"), ("square", "row"), ("square", "square")])
def test_product(m, n, k, blocks):
    for fa, fb, out, pad in (("e4m3", "e4m3", "bf16", 0), ("e5m2", "e4m3", "f32", 16),
                             ("e4m3", "e5m2", "f32", 5), ("e5m2", "e5m2", "bf16", 48)):
        say("product", m, n, k, blocks, fa, fb, out, pad)
        a, sa, wa = operand(m, k, fa, blocks[0], 1, pad)
        b, sb, wb = operand(n, k, fb, blocks[1], 2, pad)
        c = torch.zeros(m, n + pad, dtype=DT[out], device="cuda")
        c[:, n:] = 7.0
        nsf.muon_fp8_matmul(a, sa, b, sb, c[:, :n])
        check_product(c[:, :n], wa, wb, out)
        assert (c[:, n:] == 7.0).all()
        again = torch.zeros(m, n, dtype=DT[out], device="cuda")
        nsf.muon_fp8_matmul(a, sa, b, sb, again)
        assert torch.equal(again, c[:, :n])


@pytest.mark.parametrize("m,n,k", [(1, 300, 4096), (130, 257, 1000), (256, 256, 2048), (512, 384, 8192)])
def test_product_accumulates(m, n, k):
    say("accumulate", m, n, k)
    a, sa, wa = operand(m, k, "e5m2", "row", 3)
    b, sb, wb = operand(n, k, "e4m3", "row", 4)
    out = torch.randn(m, n, device="cuda") * float(np.abs(wa @ wb.T).mean())
    before = out.double().cpu().numpy()
    nsf.muon_fp8_matmul(a, sa, b, sb, out, accumulate=True)
    check_product(out, wa, wb, "f32", before)


def test_product_over_nothing():
    say("k = 0")
    a = torch.zeros(5, 0, dtype=TYPES["e4m3"], device="cuda")
    b = torch.zeros(7, 0, dtype=TYPES["e4m3"], device="cuda")
    out = torch.ones(5, 7, device="cuda")
    nsf.muon_fp8_matmul(a, nsf.fp8_scales(5, 0, "row", "cuda"), b, nsf.fp8_scales(7, 0, "row", "cuda"), out,
                        accumulate=True)
    assert (out == 1).all()
    nsf.muon_fp8_matmul(a, nsf.fp8_scales(5, 0, "row", "cuda"), b, nsf.fp8_scales(7, 0, "row", "cuda"), out)
    assert (out == 0).all()


@pytest.mark.parametrize("m,n,k", [(3, 140, 600), (300, 300, 512)])
def test_product_nan_stays_in_its_row(m, n, k):
    say("nan", m, n, k)
    a, sa, _ = operand(m, k, "e4m3", "row", 5)
    b, sb, _ = operand(n, k, "e4m3", "row", 6)
    clean, out = (torch.zeros(m, n, device="cuda") for _ in range(2))
    nsf.muon_fp8_matmul(a, sa, b, sb, clean)
    sa[2, 1] = float("nan")
    b.view(torch.uint8)[100, k - 1] = 0x7F
    nsf.muon_fp8_matmul(a, sa, b, sb, out)
    assert torch.isnan(out[2]).all() and torch.isnan(out[:, 100]).all()
    keep = torch.ones(m, n, dtype=torch.bool, device="cuda")
    keep[2], keep[:, 100] = False, False
    assert torch.equal(out[keep], clean[keep])


def test_cast_and_product_replayed():
    """Forward product, input gradient and weight gradient of a layer, captured at the first
    call and replayed with other inputs."""
    say("replay")
    m, n, k = 200, 384, 256
    x, w, dy = values(m, k, "bf16", 1), values(n, k, "f32", 2), values(m, n, "bf16", 3)
    grad = torch.zeros(n, k, device="cuda")
    y, dx = (torch.zeros(m, j, dtype=torch.bfloat16, device="cuda") for j in (n, k))
    q = {name: torch.zeros(*shape, dtype=TYPES[f], device="cuda") for name, shape, f in
         (("x", (m, k), "e4m3"), ("xt", (k, m), "e4m3"), ("w", (n, k), "e4m3"), ("wt", (k, n), "e4m3"),
          ("dy", (m, n), "e5m2"), ("dyt", (n, m), "e5m2"))}
    s = {name: nsf.fp8_scales(*q[name].shape, "square" if name[0] == "w" else "row", "cuda") for name in q}
    need = max(nsf.muon_fp8_workspace_bytes(*z) for z in ((m, n, k), (m, k, n), (n, k, m)))
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")

    def layer():
        nsf.muon_fp8_cast(w, q["w"], s["w"], q["wt"], s["wt"])
        nsf.muon_fp8_cast(x, q["x"], s["x"], q["xt"], s["xt"])
        nsf.muon_fp8_cast(dy, q["dy"], s["dy"], q["dyt"], s["dyt"])
        nsf.muon_fp8_matmul(q["x"], s["x"], q["w"], s["w"], y, workspace=ws)
        nsf.muon_fp8_matmul(q["dy"], s["dy"], q["wt"], s["wt"], dx, workspace=ws)
        nsf.muon_fp8_matmul(q["dyt"], s["dyt"], q["xt"], s["xt"], grad, accumulate=True, workspace=ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for seed in (11, 12, 13):
        x.copy_(values(m, k, "bf16", seed))
        w.copy_(values(n, k, "f32", seed + 100))
        dy.copy_(values(m, n, "bf16", seed + 200))
        grad.normal_()
        start = grad.clone()
        graph.replay()
        got = [t.clone() for t in (y, dx, grad)]
        torch.cuda.synchronize()
        grad.copy_(start)
        layer()
        for a, b in zip(got, (y, dx, grad)):
            assert torch.equal(a, b)
        # and against the formulas, through the numbers that the codes stand for
        wide = {name: fo.widen(codes_of(q[name]), host(s[name].contiguous()),
                               "e5m2" if name[:2] == "dy" else "e4m3") for name in q}
        check_product(y, wide["x"], wide["w"], "bf16")
        check_product(dx, wide["dy"], wide["wt"], "bf16")
        check_product(grad, wide["dyt"], wide["xt"], "f32", start.double().cpu().numpy())


def test_another_stream():
    say("stream")
    a, sa, wa = operand(300, 700, "e4m3", "row", 1)
    b, sb, wb = operand(200, 700, "e4m3", "square", 2)
    out = torch.zeros(300, 200, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        nsf.muon_fp8_matmul(a, sa, b, sb, out)
    torch.cuda.current_stream().wait_stream(stream)
    check_product(out, wa, wb, "f32")
