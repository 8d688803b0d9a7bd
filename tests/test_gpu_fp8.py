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


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block", ["row", "square"])
def test_cast_numbers_beside_the_middles(block, fmt):
    """The float32 numbers closest to every middle between two codes, their neighbours, and exact
    middles whose L / m is no float32: all lie nearer to it than a rounding of the quotient."""
    say("cast beside middles", block, fmt)
    rng = np.random.default_rng(3)
    v = fo.numbers(fmt)
    middles, top = (v[1:] + v[:-1]) / 2, v[-1]
    rows = 128 * 24
    m = np.exp2(rng.uniform(-99, 127.5, rows)).astype(np.float32)
    m[::3] = np.float32(7) * rng.integers(1, 100, rows)[::3].astype(np.float32)
    m[:4] = 3.4e38, 2.0 ** 101, 2.0 ** -100, 1.0
    if block == "square":
        m = m.reshape(-1, 128).max(axis=1).repeat(128)
    x = np.zeros((rows, 256), np.float32)
    near = (rng.choice(middles, x.shape) * m[:, None].astype(np.float64) / top).astype(np.float32)
    x[:] = np.nextafter(near, np.float32(np.inf) * rng.choice([-1, 1], x.shape).astype(np.float32))
    x = np.where(rng.integers(0, 3, x.shape) == 0, x, near) * rng.choice(np.float32([-1, 1, 1, 0]), x.shape)
    x[:, ::128] = m[:, None]
    for part in (x, np.ascontiguousarray(x.T)):
        t = torch.from_numpy(part).cuda()
        (q, qt), (s, st) = cast(t, fmt, block)
        for got, sc, w in ((q, s, part), (qt, st, part.T)):
            want = fo.cast(w, fmt, block == "square")
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


# --------------------------------------------------------------- larger shapes, against float64 on the GPU

def wide_gpu(codes, scales):
    s = scales.double()
    if s.shape[0] != codes.shape[0]:
        s = s.repeat_interleave(128, 0)[:codes.shape[0]]
    return codes.double() * s.repeat_interleave(128, 1)[:, :codes.shape[1]]


def check_on_gpu(got, a, sa, b, sb, before=None):
    """As check_product; what the 8-bit instruction cuts off, 7 of 8 products at 2^-13 of their
    group's largest, is below 7 x 2^-13 of the sum of magnitudes."""
    wa, wb = wide_gpu(a, sa), wide_gpu(b, sb)
    want, total = wa @ wb.t().contiguous(), wa.abs() @ wb.abs().t().contiguous()
    bound = (128 + fo.blocks(a.shape[1]) + 4) * 2.0 ** -24 * total
    if before is not None:
        want = want + before.double()
        bound += 2.0 ** -23 * want.abs()
    err = (got.double() - want).abs()
    if got.dtype == torch.bfloat16:
        bound = bound + 7 * 2.0 ** -13 * total
        bound = bound + 2.0 ** -8 * (want.abs() + bound)
        assert torch.linalg.norm(err) <= 2.0 ** -8 * torch.linalg.norm(want)
    else:
        bound = bound + 2.0 ** -24 * want.abs()
    assert (err <= bound + 1e-300).all(), (err / (bound + 1e-300)).max().item()


def big_operand(rows, k, fmt, block, seed, pad):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, k, generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-6, 7, (rows, 1), generator=g, device="cuda").float())
    held = torch.full((rows, k + pad), 0x7F, dtype=torch.uint8, device="cuda").view(TYPES[fmt])[:, :k]
    s = nsf.fp8_scales(rows, k, block, "cuda")
    nsf.muon_fp8_cast(x, held, s)
    return held, s


# tiles of 256 (whole and ragged), of 128, and of either with k's blocks shared by workgroups
BIG = [(2048, 8192, 1152), (2000, 8100, 1168), (1000, 4000, 512), (1024, 1024, 8192), (600, 2048, 7168),
       (4096, 1024, 8200)]


@pytest.mark.parametrize("m,n,k", BIG)
@pytest.mark.parametrize("blocks", ["square", "row"])
@pytest.mark.parametrize("pad", [0, 11])
def test_large_products(m, n, k, blocks, pad):
    for fa, fb, out, add in (("e4m3", "e4m3", "bf16", False), ("e5m2", "e4m3", "f32", True),
                             ("e4m3", "e5m2", "f32", False), ("e5m2", "e5m2", "bf16", False)):
        say("large product", m, n, k, blocks, fa, fb, out, add, pad)
        a, sa = big_operand(m, k, fa, "row", 1, pad)
        b, sb = big_operand(n, k, fb, blocks, 2, pad)
        c = torch.full((m, n), 0.5, dtype=DT[out], device="cuda")
        before = c.clone() if add else None
        nsf.muon_fp8_matmul(a, sa, b, sb, c, accumulate=add)
        check_on_gpu(c, a, sa, b, sb, before)


def test_products_past_2_31_elements():
    say("past 2^31")
    m, n, k = 50001, 50000, 144            # 2.5 G results
    a, sa = big_operand(m, k, "e4m3", "row", 1, 0)
    b, sb = big_operand(n, k, "e4m3", "square", 2, 0)
    c = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    nsf.muon_fp8_matmul(a, sa, b, sb, c)
    for at in (0, 25000, m - 70):
        check_on_gpu(c[at:at + 70], a[at:at + 70], sa[at:at + 70], b, sb)


def test_casts_past_2_31_elements():
    say("cast past 2^31")
    rows, cols = 70000, 32768              # 2.3 G elements
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.bfloat16)
    for block in ("row", "square"):
        q = torch.empty(rows, cols, dtype=TYPES["e4m3"], device="cuda")
        qt = torch.empty(cols, rows, dtype=TYPES["e4m3"], device="cuda")
        s, st = nsf.fp8_scales(rows, cols, block, "cuda"), nsf.fp8_scales(cols, rows, block, "cuda")
        nsf.muon_fp8_cast(x, q, s, qt, st)
        for at in (0, 128 * 300, rows - rows % 128 - 128):
            part = x[at:at + 128, cols - 300:].float().cpu().numpy()
            part = part[:, 300 % 128:]     # whole blocks
            want, ws = fo.cast(part, "e4m3", block == "square")
            got = q[at:at + 128, cols - 256:]
            assert np.array_equal(codes_of(got), want)
            sc = s[at // 128:at // 128 + 1] if block == "square" else s[at:at + 128]
            assert np.array_equal(host(sc[:, -2:].contiguous()), ws)
            want, ws = fo.cast(part.T, "e4m3", block == "square")
            assert np.array_equal(codes_of(qt[cols - 256:, at:at + 128]), want)
            sc = st[-2:] if block == "square" else st[cols - 256:]
            assert np.array_equal(host(sc[:, at // 128:at // 128 + 1].contiguous()), ws)
        del q, qt


def test_one_matrix_as_both_operands():
    say("a a^T")
    a, sa = big_operand(300, 700, "e4m3", "row", 1, 0)
    out = torch.empty(300, 300, device="cuda")
    nsf.muon_fp8_matmul(a, sa, a, sa, out)
    check_on_gpu(out, a, sa, a, sa)
    assert torch.equal(out, out.t())


def test_scales_in_either_order():
    """Scales that lie row after row give what block-major ones give."""
    say("scale order")
    a, sa = big_operand(300, 700, "e4m3", "row", 1, 0)
    b, sb = big_operand(200, 700, "e4m3", "square", 2, 0)
    one, two = (torch.empty(300, 200, device="cuda") for _ in range(2))
    nsf.muon_fp8_matmul(a, sa, b, sb, one)
    nsf.muon_fp8_matmul(a, sa.contiguous(), b, sb.contiguous(), two)
    assert sa.contiguous().stride() != sa.stride() and torch.equal(one, two)
    x = values(300, 700, "f32", 3)
    q, qs = torch.empty_like(a), torch.empty(300, 6, device="cuda")
    nsf.muon_fp8_cast(x, q, qs)
    want = fo.cast(x.cpu().numpy(), "e4m3", False)
    assert np.array_equal(codes_of(q), want[0]) and np.array_equal(host(qs), want[1])


# --------------------------------------------------------------- a layer's training step

def test_training_step_of_a_layer():
    """The 8-bit copy of the weight, the layer's three products with the weight's gradient added
    into the flat buffer, the norm, the clipped step and the refreshed copy: eager, then captured
    and replayed on other inputs."""
    say("layer")
    m, n, k = 96, 256, 384
    hyper = [(0.02, 0.01, 0.95, True)]
    descs = [(0, n, k)]
    state = {name: torch.zeros(n * k, device="cuda") for name in ("w", "grad", "mom")}
    x, dy = (torch.zeros(m, j, dtype=torch.bfloat16, device="cuda") for j in (k, n))
    y, dx = (torch.zeros(m, j, dtype=torch.bfloat16, device="cuda") for j in (n, k))
    shapes = {"w": (n, k), "wt": (k, n), "x": (m, k), "xt": (k, m), "dy": (m, n), "dyt": (n, m)}
    q = {name: torch.zeros(*z, dtype=TYPES["e5m2" if name[0] == "d" else "e4m3"], device="cuda")
         for name, z in shapes.items()}
    s = {name: nsf.fp8_scales(*z, "square" if name[0] == "w" else "row", "cuda")
         for name, z in shapes.items()}
    groups, clip = nsf.group_table(hyper, "cuda"), nsf.clip_state("cuda")
    tensors = nsf.tensor_list([state["grad"]])
    ws = torch.empty(max(nsf.muon_workspace_bytes(descs), 1 << 20), dtype=torch.uint8, device="cuda")
    need = max(nsf.muon_fp8_workspace_bytes(*z) for z in ((m, n, k), (m, k, n), (n, k, m)))
    ws8 = torch.empty(need, dtype=torch.uint8, device="cuda")

    def step():
        w = state["w"].view(n, k)
        state["grad"].zero_()
        nsf.muon_fp8_cast(x, q["x"], s["x"], q["xt"], s["xt"])
        nsf.muon_fp8_matmul(q["x"], s["x"], q["w"], s["w"], y, workspace=ws8)
        nsf.muon_fp8_cast(dy, q["dy"], s["dy"], q["dyt"], s["dyt"])
        nsf.muon_fp8_matmul(q["dy"], s["dy"], q["wt"], s["wt"], dx, workspace=ws8)
        nsf.muon_fp8_matmul(q["dyt"], s["dyt"], q["xt"], s["xt"], state["grad"].view(n, k),
                            accumulate=True, workspace=ws8)
        nsf.muon_grad_norm(tensors, 1.0, clip, workspace=ws)
        nsf.muon_step_clipped(state["w"], state["grad"], state["mom"], descs, groups, clip, workspace=ws)
        nsf.muon_fp8_cast(w, q["w"], s["w"], q["wt"], s["wt"])

    def fill(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        state["w"].normal_(0, 0.02, generator=g)
        state["mom"].normal_(0, 1e-3, generator=g)
        x.normal_(0, 1, generator=g)
        dy.normal_(0, 1e-2, generator=g)
        nsf.muon_fp8_cast(state["w"].view(n, k), q["w"], s["w"], q["wt"], s["wt"])

    fill(0)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2, 3):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        got = {name: t.clone() for name, t in (("y", y), ("dx", dx), *state.items())}
        copies = {name: q[name].view(torch.uint8).clone() for name in ("w", "wt")}
        fill(seed)
        old = {name: wide_gpu(q[name], s[name]) for name in ("w", "wt")}
        step()
        for name, t in (("y", y), ("dx", dx), *state.items()):
            assert torch.equal(got[name], t), name
        # the refreshed copies are the casts of the updated weight
        wn = state["w"].view(n, k).cpu().numpy()
        for name, m_ in (("w", wn), ("wt", wn.T)):
            want = fo.cast(m_, "e4m3", True)
            assert np.array_equal(copies[name].cpu().numpy(), want[0])
            assert np.array_equal(host(s[name].contiguous()), want[1])
        # gradients of L = sum(dy * y), y = x w^T, against its differences: L is linear in each of x and
        # w, so a difference quotient of any step is the gradient, up to float64 roundings
        wide = {name: wide_gpu(q[name], s[name]) for name in ("x", "dy", "dyt", "xt")}
        grad = got["grad"].view(n, k).double()
        for i, j in ((0, 0), (17, 300), (n - 1, k - 1)):
            loss = []
            for move in (-1.0, 1.0):
                w = old["w"].clone()
                w[i, j] += move
                loss.append((wide["dyt"].t() * (wide["xt"].t() @ w.t())).sum())
            size = (wide["dyt"][i].abs() * wide["xt"][j].abs()).sum()
            assert abs((loss[1] - loss[0]) / 2 - grad[i, j]) <= 200 * 2.0 ** -24 * size + 1e-12
            loss = []
            for move in (-1.0, 1.0):
                xs = wide["x"].clone()
                xs[i % m, j] += move
                loss.append((wide["dy"] * (xs @ old["wt"])).sum())
            size = (wide["dy"][i % m].abs() * old["wt"][j].abs()).sum()
            assert abs((loss[1] - loss[0]) / 2 - got["dx"][i % m, j]) <= (
                2.0 ** -8 * abs(got["dx"][i % m, j]) * 1.01 + (7 * 2.0 ** -13 + 200 * 2.0 ** -24) * size + 1e-12)


# --------------------------------------------------------------- scales of every size

# few rows, in one split and in several; tiles of 64 (direct and unaligned, in splits), 128 and 256
ANY_SCALE = [(3, 140, 600), (1, 1024, 14336), (100, 300, 1999), (300, 300, 512), (33, 2048, 7168),
             (1000, 4000, 512), (1000, 4000, 527), (2000, 8100, 1168)]


def check_any_scale(got, a, sa, b, sb):
    """As check_on_gpu, and what subnormal numbers add: half of 2^-149 for a block's product and for its
    addition, half of 2^-133 for a result in bfloat16."""
    wa, wb = wide_gpu(a, sa), wide_gpu(b, sb)
    want, total = wa @ wb.t().contiguous(), wa.abs() @ wb.abs().t().contiguous()
    bound = (128 + fo.blocks(a.shape[1]) + 4) * 2.0 ** -24 * total + fo.blocks(a.shape[1]) * 2.0 ** -149
    if got.dtype == torch.bfloat16:
        bound = bound + 7 * 2.0 ** -13 * total
        bound = bound + 2.0 ** -8 * (want.abs() + bound) + 2.0 ** -134
    else:
        bound = bound + 2.0 ** -24 * want.abs()
    err = (got.double() - want).abs()
    assert (err <= bound).all(), ((err / bound).max().item(), torch.isnan(got).sum().item())


@pytest.mark.parametrize("m,n,k", ANY_SCALE)
@pytest.mark.parametrize("blocks", ["square", "row"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_products_of_scales_of_every_size(m, n, k, blocks, out):
    """Both operands small or large, and rows and blocks of a that are, beside ordinary ones,
    whose results keep their bits."""
    fa, fb = ("e4m3", "e4m3") if out == "bf16" else ("e5m2", "e4m3")
    a, sa = big_operand(m, k, fa, "row", 1, 0)
    b, sb = big_operand(n, k, fb, blocks, 2, 0)
    plain = torch.zeros(m, n, dtype=DT[out], device="cuda")
    nsf.muon_fp8_matmul(a, sa, b, sb, plain)
    for ea, eb in ((-62, -62), (-58, -70), (-110, -10), (-10, -110), (-100, 30), (50, 45), (-126, 100)):
        say("scales", m, n, k, blocks, out, ea, eb)
        c = torch.full((m, n), 7.0, dtype=DT[out], device="cuda")
        ta, tb = sa * 2.0 ** ea, sb * 2.0 ** eb
        nsf.muon_fp8_matmul(a, ta, b, tb, c)
        check_any_scale(c, a, ta, b, tb)
    say("scales, one row", m, n, k, blocks, out)
    c = torch.full((m, n), 7.0, dtype=DT[out], device="cuda")
    ta, tb = sa.clone(), sb.clone()
    ta[m // 2] *= 2.0 ** -110
    tb[:, -1] *= 2.0 ** -24
    nsf.muon_fp8_matmul(a, sa, b, tb, plain)
    nsf.muon_fp8_matmul(a, ta, b, tb, c)
    check_any_scale(c, a, ta, b, tb)
    rest = [i for i in range(m) if i != m // 2]
    assert torch.equal(c[rest], plain[rest])


@pytest.mark.parametrize("m,n,k", ANY_SCALE)
@pytest.mark.parametrize("blocks", ["square", "row"])
def test_large_scales_of_blocks_that_do_not_meet(m, n, k, blocks):
    """Two scales whose product is infinite, of a block whose codes never meet: zero, not NaN."""
    say("large scales", m, n, k, blocks)
    a, sa = big_operand(m, k, "e4m3", "row", 1, 0)
    b, sb = big_operand(n, k, "e4m3", blocks, 2, 0)
    a.view(torch.uint8)[:, 128:192] = 0
    b.view(torch.uint8)[:, 192:256] = 0
    ta, tb = sa.clone(), sb.clone()
    ta[:, 1], tb[:, 1] = 2.0 ** 65, 2.0 ** 66
    for out in ("f32", "bf16"):
        want, c = (torch.full((m, n), 7.0, dtype=DT[out], device="cuda") for _ in range(2))
        nsf.muon_fp8_matmul(a, sa, b, sb, want)
        nsf.muon_fp8_matmul(a, ta, b, tb, c)
        assert torch.equal(c, want)


@pytest.mark.parametrize("m,n,k", ANY_SCALE)
@pytest.mark.parametrize("blocks", ["square", "row"])
def test_rows_of_zeros(m, n, k, blocks):
    """Padding of a and small blocks of b: products of their scales are subnormal, sums zero."""
    say("zero rows", m, n, k, blocks)
    for out in ("f32", "bf16"):
        x = torch.randn(m, k, device="cuda")
        x[m // 2:] = 0
        a = torch.empty(m, k, dtype=TYPES["e4m3"], device="cuda")
        sa = nsf.fp8_scales(m, k, "row", "cuda")
        nsf.muon_fp8_cast(x, a, sa)
        b, sb = big_operand(n, k, "e4m3", blocks, 2, 0)
        sb *= 2.0 ** -30
        c = torch.full((m, n), 7.0, dtype=DT[out], device="cuda")
        nsf.muon_fp8_matmul(a, sa, b, sb, c)
        check_any_scale(c, a, sa, b, sb)
        assert (c[m // 2:] == 0).all()


# up to 16 rows with k in several splits
FEW_SPLIT = [(1, 1024, 14336), (16, 2047, 7169), (5, 100, 20000)]


@pytest.mark.parametrize("m,n,k", FEW_SPLIT)
@pytest.mark.parametrize("blocks", ["square", "row"])
def test_few_rows_in_splits(m, n, k, blocks):
    assert nsf.muon_fp8_workspace_bytes(m, n, k) > 0
    for fa, fb, out, add in (("e4m3", "e4m3", "bf16", False), ("e5m2", "e4m3", "f32", True),
                             ("e4m3", "e5m2", "f32", False), ("e5m2", "e5m2", "bf16", False)):
        say("few rows in splits", m, n, k, blocks, fa, fb, out, add)
        a, sa = big_operand(m, k, fa, "row", 1, 0)
        b, sb = big_operand(n, k, fb, blocks, 2, 0)
        held = torch.full((m, n + 3), 0.5, dtype=DT[out], device="cuda")
        c = held[:, :n]
        before = c.clone() if add else None
        ws = torch.full((nsf.muon_fp8_workspace_bytes(m, n, k),), 0xFF, dtype=torch.uint8, device="cuda")
        nsf.muon_fp8_matmul(a, sa, b, sb, c, accumulate=add, workspace=ws)
        check_on_gpu(c, a, sa, b, sb, before)
        assert (held[:, n:] == 0.5).all()


@pytest.mark.parametrize("m,n,k", [(3, 140, 600), (1, 1024, 14336), (100, 300, 1999), (300, 300, 512),
                                   (512, 384, 8192), (1000, 4000, 512), (2000, 8100, 1168)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("fa,fb", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
def test_nan_and_infinities_of_either_kind(m, n, k, out, fa, fb):
    """A NaN code, an infinite one (5 exponent bits have them) and scales that are NaN or infinite
    reach the results of their row of a or of b and no others."""
    a, sa = big_operand(m, k, fa, "row", 5, 0)
    b, sb = big_operand(n, k, fb, "row", 6, 0)
    clean = torch.zeros(m, n, dtype=DT[out], device="cuda")
    nsf.muon_fp8_matmul(a, sa, b, sb, clean)
    i, j = m - 1, 100

    def run(what, change_a=None, change_b=None, scale_a=None, scale_b=None):
        say("nan and infinities", m, n, k, out, fa, fb, what)
        ta, tsa, tb, tsb = a.clone(), sa.clone(), b.clone(), sb.clone()
        if change_a is not None:
            ta.view(torch.uint8)[i, k // 2] = change_a
        if change_b is not None:
            tb.view(torch.uint8)[j, k - 1] = change_b
        if scale_a is not None:
            tsa[i, 1] = scale_a
        if scale_b is not None:
            tsb[j, 2] = scale_b
        c = torch.full((m, n), 7.0, dtype=DT[out], device="cuda")
        nsf.muon_fp8_matmul(ta, tsa, tb, tsb, c)
        of_a, of_b = change_a is not None or scale_a is not None, change_b is not None or scale_b is not None
        rest = torch.ones(m, n, dtype=torch.bool, device="cuda")
        if of_a:
            rest[i] = False
        if of_b:
            rest[:, j] = False
        assert torch.equal(c[rest], clean[rest])
        assert not torch.isfinite(c[~rest]).any()
        return c, ta, tb

    for nan in (0x7F, 0xFF):
        c, _, _ = run("codes %x" % nan, nan, nan)
        assert torch.isnan(c[i]).all() and torch.isnan(c[:, j]).all()
    c, _, _ = run("scales", scale_a=float("nan"), scale_b=float("nan"))
    assert torch.isnan(c[i]).all() and torch.isnan(c[:, j]).all()
    run("infinite scales", scale_a=float("inf"))
    run("infinite scales", scale_b=float("-inf"))
    for code, sign in ((0x7C, 1.0), (0xFC, -1.0)):
        if fa == "e5m2":
            # infinity times a code: of its sign, and no number where that is zero
            c, _, _ = run("a %x" % code, change_a=code)
            assert torch.equal(torch.nan_to_num(c[i].float(), nan=0.0),
                               torch.nan_to_num(sign * float("inf") * b[:, k // 2].float(), nan=0.0))
        if fb == "e5m2":
            c, _, _ = run("b %x" % code, change_b=code)
            assert torch.equal(torch.nan_to_num(c[:, j].float(), nan=0.0),
                               torch.nan_to_num(sign * float("inf") * a[:, k - 1].float(), nan=0.0))


@pytest.mark.parametrize("m,n,k", [(3, 140, 600), (100, 300, 1999), (512, 384, 8192), (2000, 8100, 1168)])
def test_scales_of_every_size_accumulated_and_replayed(m, n, k):
    """One captured call, replayed with ordinary, small and subnormal scales and NaN among them,
    each added into out."""
    say("scales replayed", m, n, k)
    a, sa = big_operand(m, k, "e5m2", "row", 1, 0)
    b, sb = big_operand(n, k, "e4m3", "row", 2, 0)
    ta, tb, out = sa.clone(), sb.clone(), torch.zeros(m, n, device="cuda")
    ws = torch.empty(max(256, nsf.muon_fp8_workspace_bytes(m, n, k)), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nsf.muon_fp8_matmul(a, ta, b, tb, out, accumulate=True, workspace=ws)
    before = torch.randn(m, n, device="cuda")
    for ea, eb in ((0, 0), (-62, -55), (-128, 10), (-128, -3), (0, 0)):
        ta.copy_(sa * 2.0 ** ea)
        tb.copy_(sb * 2.0 ** eb)
        start = before * 2.0 ** (ea + eb)
        out.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        wa, wb = wide_gpu(a, ta), wide_gpu(b, tb)
        want = wa @ wb.t().contiguous() + start.double()
        total = wa.abs() @ wb.abs().t().contiguous()
        bound = (128 + fo.blocks(k) + 4) * 2.0 ** -24 * total + fo.blocks(k) * 2.0 ** -149 + 2.0 ** -23 * want.abs()
        assert ((got.double() - want).abs() <= bound).all()
        out.copy_(start)
        nsf.muon_fp8_matmul(a, ta, b, tb, out, accumulate=True, workspace=ws)
        assert torch.equal(out, got)
    # a NaN beside small scales: in its row, the others as without it
    ta.copy_(sa * 2.0 ** -62)
    tb.copy_(sb * 2.0 ** -62)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    got = out.clone()
    ta[m // 2, 1] = float("nan")
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.isnan(out[m // 2]).all()
    rest = torch.arange(m, device="cuda") != m // 2
    assert torch.equal(out[rest], got[rest])
