"""GPU tests of the orthogonalization of stacks, against float64.

The tolerance of a case comes from the arithmetic itself: the same iteration in
float64 with every X, A and B rounded to the pairs' 22 digits deviates from the
exact one by some amount; the kernels drop one product of halves (as much again),
sum in float32 (2^-24 a step of up to 3 K / 32 of them, growing as their square root) and
round the scaled input, so eight times that deviation is allowed, and 2e-6 for
matrices that it leaves nearly exact."""

import numpy as np
import pytest

import newton_schulz_flat_amd as nsf
from oracle import fp8_oracle as fo
from tests.gpu_helpers import rel_fro, say

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
POLISHED = [nsf.QUINTIC[0]] * 3 + [(1.875, -1.25, 0.375)] * 2


def tolerance(u, steps, want, out):
    tol = 2e-6 + 8 * rel_fro(fo.newton_schulz(u, steps, digits=22), want)
    return tol + (2.0 ** -8 if out == "bf16" else 0.0)


def check(x, out, steps=nsf.QUINTIC, scale=None):
    kind = "bf16" if out.dtype == torch.bfloat16 else "f32"
    xs = x.double().cpu().numpy().reshape(-1, *x.shape[-2:])
    os = out.double().cpu().numpy().reshape(-1, *x.shape[-2:])
    s = max(1.0, x.shape[-2] / x.shape[-1]) ** 0.5 if scale is None else scale
    for u, o in zip(xs, os):
        want = fo.newton_schulz(u, steps)
        tol = tolerance(u, steps, want, kind)
        err = rel_fro(o, s * want)
        assert err <= tol, (x.shape, err, tol)


def stack(count, rows, cols, dtype="f32", seed=0, std=1e-3, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = std * torch.randn(count, rows, cols + pad, generator=g)
    return x.to(DT[dtype]).cuda()[:, :, :cols]


@pytest.mark.parametrize("count,rows,cols", [(1, 1, 1), (3, 1, 70), (2, 5, 3), (7, 16, 16), (4, 33, 65),
                                             (16, 48, 64), (2, 64, 64), (3, 64, 200), (2, 65, 64),
                                             (5, 100, 129), (2, 128, 513), (3, 300, 77), (1, 257, 255),
                                             (2, 320, 640), (300, 20, 24), (1, 700, 900)])
@pytest.mark.parametrize("dtype,out,pad", [("f32", "f32", 0), ("bf16", "bf16", 0), ("f32", "bf16", 5),
                                           ("bf16", "f32", 23)])
def test_stack(count, rows, cols, dtype, out, pad):
    say("stack", count, rows, cols, dtype, out, pad)
    x = stack(count, rows, cols, dtype, seed=rows + cols, pad=pad)
    held = torch.full((count, rows, cols + pad), 3.0, dtype=DT[out], device="cuda")
    nsf.muon_orthogonalize_stack(x, held[:, :, :cols])
    check(x[:4], held[:4, :, :cols])
    assert (held[:, :, cols:] == 3.0).all()
    # each matrix depends on itself alone
    one = torch.empty(rows, cols, dtype=DT[out], device="cuda")
    nsf.muon_orthogonalize_stack(x[count - 1], one)
    assert rel_fro(one.double().cpu().numpy(), held[-1, :, :cols].double().cpu().numpy()) <= 1e-5 + (
        2.0 ** -8 if out == "bf16" else 0)


@pytest.mark.parametrize("rows,cols", [(40, 90), (130, 70), (512, 512)])
def test_coefficients_and_scale(rows, cols):
    x = stack(2, rows, cols, seed=9)
    for steps in ([], [nsf.QUINTIC[0]], POLISHED, [(2.0, -1.5, 0.5)] * 12,
                  [(8.0, -22.0, 15.0), (1.0, -0.2, 0.0)] + POLISHED, [(0.01, 0.0, 0.0)] * 3):
        for scale in (None, 1.0, -0.25):
            say("coefficients", rows, cols, steps, scale)
            out = torch.empty_like(x)
            nsf.muon_orthogonalize_stack(x, out, coefficients=steps, scale=scale)
            check(x, out, steps, scale)


def test_coefficients_that_let_values_grow_are_refused():
    x = stack(1, 40, 90)
    out = torch.zeros_like(x)
    # |8 x - 22 x^3 + 16 x^5| reaches 2 at x = 1, and 4 x - 3 x^3 + 0.6 x^5 3.2 there
    steps = [(8.0, -22.0, 16.0), (4.0, -3.0, 0.6)] + POLISHED
    with pytest.raises(nsf.MuonError, match="BAD_ARG.*grow"):
        nsf.muon_orthogonalize_stack(x, out, coefficients=steps)
    assert (out == 0).all()


@pytest.mark.parametrize("std", [1e-30, 1e-12, 1.0, 1e15, 1e30])
@pytest.mark.parametrize("rows,cols", [(24, 60), (200, 150)])
def test_sizes_of_numbers(rows, cols, std):
    say("std", rows, cols, std)
    x = stack(1, rows, cols, seed=3, std=std)
    out = torch.empty_like(x)
    nsf.muon_orthogonalize_stack(x, out)
    check(x, out)


@pytest.mark.parametrize("rows,cols", [(24, 60), (200, 150)])
def test_zero_matrices_and_low_rank(rows, cols):
    say("zero, low rank", rows, cols)
    x = stack(3, rows, cols, seed=4)
    x[0] = 0
    x[1] = x[1, :, :1] @ x[1, :1, :]
    x[2, 3:] = 0
    out = torch.empty_like(x)
    nsf.muon_orthogonalize_stack(x, out)
    assert (out[0] == 0).all()
    for k in (1, 2):
        u = x[k].double().cpu().numpy()
        want = fo.newton_schulz(u, nsf.QUINTIC) * max(1.0, rows / cols) ** 0.5
        # roundings in the null space grow by the first coefficient a step: 482 times 2^-22 of
        # an iterate's norm at each of five steps
        err = np.linalg.norm(out[k].double().cpu().numpy() - want)
        assert err <= 5 * 482 * 2.0 ** -22 * np.linalg.norm(want) * 2


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("rows,cols", [(24, 60), (200, 150)])
@pytest.mark.parametrize("steps", [0, 2])
def test_nan_and_infinity_stay_in_their_matrix(rows, cols, bad, steps):
    say("nan", rows, cols, bad, steps)
    x = stack(3, rows, cols, seed=6)
    clean, out = torch.empty_like(x), torch.empty_like(x)
    nsf.muon_orthogonalize_stack(x, clean, coefficients=nsf.QUINTIC[:steps])
    x[1, 5, 7] = bad
    nsf.muon_orthogonalize_stack(x, out, coefficients=nsf.QUINTIC[:steps])
    assert torch.isnan(out[1]).all()
    assert torch.equal(out[0], clean[0]) and torch.equal(out[2], clean[2])


def test_strides_and_overlapping_inputs():
    """Matrices side by side in longer rows, one matrix for all, windows that overlap."""
    say("strides")
    base = stack(1, 90, 400, seed=2)[0]
    side = base.view(90, 4, 100).transpose(0, 1)            # four 90 x 100, 100 apart
    out = torch.empty(90, 4, 100, device="cuda").transpose(0, 1)
    nsf.muon_orthogonalize_stack(side, out)
    check(side, out)
    same = base[:, :100].unsqueeze(0).expand(3, 90, 100)
    got = torch.empty(3, 90, 100, device="cuda")
    nsf.muon_orthogonalize_stack(same, got)
    assert torch.equal(got[0], out[0]) and torch.equal(got[1], got[2])
    windows = base.as_strided((5, 40, 64), (7, 400, 1))
    got = torch.empty(5, 40, 64, device="cuda")
    nsf.muon_orthogonalize_stack(windows, got)
    check(windows, got)


@pytest.mark.parametrize("rows,cols", [(24, 60), (200, 150)])
def test_groups_that_fit_the_workspace(rows, cols):
    say("groups", rows, cols)
    x = stack(5, rows, cols, seed=8)
    one, two = torch.empty_like(x), torch.empty_like(x)
    nsf.muon_orthogonalize_stack(x, one)
    for fit in (1, 2):
        ws = torch.empty(nsf.muon_stack_workspace_bytes(x[:fit]), dtype=torch.uint8, device="cuda")
        nsf.muon_orthogonalize_stack(x, two, workspace=ws)
        assert torch.equal(one, two)
    with pytest.raises(nsf.MuonError, match="WORKSPACE"):
        nsf.muon_orthogonalize_stack(x, two, workspace=ws[:256])


@pytest.mark.parametrize("rows,cols", [(24, 60), (200, 150), (512, 768)])
def test_replayed(rows, cols):
    say("replay", rows, cols)
    x = stack(3, rows, cols, seed=1)
    out, want = torch.empty_like(x), torch.empty_like(x)
    ws = torch.empty(nsf.muon_stack_workspace_bytes(x), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nsf.muon_orthogonalize_stack(x, out, workspace=ws)
    for seed in (2, 3, 4):
        x.copy_(stack(3, rows, cols, seed=seed))
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        nsf.muon_orthogonalize_stack(x, want)
        assert torch.equal(out, want)
        check(x, out)


def test_same_update_as_the_flat_entry_point():
    """The float32 mode of muon_orthogonalize on a flat buffer and the stack agree."""
    say("flat")
    x = stack(3, 256, 192, seed=7)
    descs = [(k * 256 * 192, 256, 192) for k in range(3)]
    flat, out = torch.empty(3 * 256 * 192, device="cuda"), torch.empty_like(x)
    nsf.muon_orthogonalize(x.reshape(-1), flat, descs, mode="f32")
    nsf.muon_orthogonalize_stack(x, out)
    for k in range(3):
        assert rel_fro(out[k].double().cpu().numpy(),
                       flat.view_as(x)[k].double().cpu().numpy()) <= 2e-5


# --------------------------------------------------------------- larger matrices, against float64 on the GPU

def reference(u, steps, digits=None):
    """fo.newton_schulz on the GPU."""
    def held(m):
        if digits is None:
            return m
        step = torch.exp2(torch.ceil(torch.log2(m.abs().clamp(min=1e-30))) - digits)
        return torch.round(m / step) * step

    x = u.double()
    x = x / (torch.linalg.norm(x) + 1e-7)
    tall = x.shape[0] > x.shape[1]
    x = held(x.t().contiguous() if tall else x)
    for a, b, c in steps:
        a, b, c = (float(np.float32(v)) for v in (a, b, c))
        g = held(x @ x.t().contiguous())
        x = held(a * x + held(b * g + c * (g @ g)) @ x)
    return x.t() if tall else x


# one workgroup a matrix with more than 64 KB of LDS; strips with B made beside them and apart; tiles
# of 64, 128 and 256, a workgroup a tile and shared
@pytest.mark.parametrize("count,rows,cols", [(2, 64, 400), (1, 1000, 30), (3, 64, 900), (1, 5000, 60),
                                             (1, 128, 8000), (40, 100, 700), (1, 1024, 1024),
                                             (1, 1500, 2100), (1, 2048, 2048), (8, 1024, 1000),
                                             (1, 256, 8192), (1, 4096, 4096), (1, 4100, 2000)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_larger_matrices(count, rows, cols, out):
    say("larger", count, rows, cols, out)
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = 1e-3 * torch.randn(count, rows, cols, generator=g, device="cuda")
    o = torch.empty(count, rows, cols, dtype=DT[out], device="cuda")
    nsf.muon_orthogonalize_stack(x, o)
    again = torch.empty_like(o)
    nsf.muon_orthogonalize_stack(x, again)
    assert torch.equal(o, again)
    for k in {0, count - 1}:
        want = reference(x[k], nsf.QUINTIC)
        tol = 2e-6 + 8 * torch.linalg.norm(reference(x[k], nsf.QUINTIC, 22) - want) / torch.linalg.norm(want)
        tol += 2.0 ** -8 if out == "bf16" else 0
        want = want * max(1.0, rows / cols) ** 0.5
        assert torch.linalg.norm(o[k].double() - want) <= tol * torch.linalg.norm(want)


@pytest.mark.parametrize("rows,cols", [(64, 400), (60, 2000), (128, 128), (1100, 900), (2048, 2048)])
def test_larger_replayed(rows, cols):
    say("larger replay", rows, cols)
    x = stack(2, rows, cols, seed=1)
    out, want = torch.empty_like(x), torch.empty_like(x)
    ws = torch.empty(nsf.muon_stack_workspace_bytes(x), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nsf.muon_orthogonalize_stack(x, out, workspace=ws)
    for seed in (2, 3, 4):
        x.copy_(stack(2, rows, cols, seed=seed))
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        nsf.muon_orthogonalize_stack(x, want)
        assert torch.equal(out, want)


@pytest.mark.parametrize("count,rows,cols", [(5, 100, 700), (40, 100, 400), (3, 700, 900), (2, 2048, 1024)])
def test_larger_groups_that_fit(count, rows, cols):
    say("larger groups", count, rows, cols)
    x = stack(count, rows, cols, seed=8)
    one, two = torch.empty_like(x), torch.empty_like(x)
    nsf.muon_orthogonalize_stack(x, one)
    ws = torch.full((nsf.muon_stack_workspace_bytes(x) // count,), 0xFF, dtype=torch.uint8, device="cuda")
    nsf.muon_orthogonalize_stack(x, two, workspace=ws)
    assert torch.equal(one, two)
    with pytest.raises(nsf.MuonError, match="WORKSPACE"):
        nsf.muon_orthogonalize_stack(x, two, workspace=ws[:-256])


def test_offsets_past_2_31():
    """Three matrices of 1.05 G elements: one step, checked on some columns of the last one."""
    say("past 2^31")
    rows, cols = 1000, 1 << 20
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(3, rows, cols, dtype=torch.bfloat16, device="cuda")
    for k in range(3):
        x[k].normal_(0, 1e-3 * (k + 1), generator=g)
    out = torch.empty_like(x)
    nsf.muon_orthogonalize_stack(x, out, coefficients=nsf.QUINTIC[:1], scale=1.0)
    for k in (0, 2):
        gram = torch.zeros(rows, rows, dtype=torch.float64, device="cuda")
        for at in range(0, cols, 1 << 17):
            part = x[k, :, at:at + (1 << 17)].double()
            gram += part @ part.t().contiguous()
        norm = torch.sqrt(torch.trace(gram)) + 1e-7
        gram /= norm * norm
        a, b, c = (float(np.float32(v)) for v in nsf.QUINTIC[0])
        poly = b * gram + c * gram @ gram
        for at in (0, cols // 2 + 5, cols - 100):
            u = x[k, :, at:at + 100].double() / norm
            want = a * u + poly @ u
            err = torch.linalg.norm(out[k, :, at:at + 100].double() - want)
            assert err <= (2.0 ** -8 + 1e-5) * torch.linalg.norm(want)


def test_another_stream_and_default_workspaces():
    say("stream")
    x, z = stack(2, 200, 150, seed=1), stack(2, 150, 300, seed=2)
    want = [torch.empty_like(x), torch.empty_like(z)]
    nsf.muon_orthogonalize_stack(x, want[0])
    nsf.muon_orthogonalize_stack(z, want[1])
    got = [torch.empty_like(x), torch.empty_like(z)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s, u, o in zip(streams, (x, z), got):
            with torch.cuda.stream(s):
                nsf.muon_orthogonalize_stack(u, o)
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# shorter side above 64 or too long for a workgroup's LDS, up to 128: strips; one and several parts
SHORT = [(100, 700), (900, 40), (128, 128), (20, 5000)]


@pytest.mark.parametrize("rows,cols", SHORT)
@pytest.mark.parametrize("std", [1e-30, 1e-12, 1e15, 1e30])
def test_short_sides_sizes_of_numbers(rows, cols, std):
    test_sizes_of_numbers(rows, cols, std)


@pytest.mark.parametrize("rows,cols", SHORT)
def test_short_sides(rows, cols):
    test_zero_matrices_and_low_rank(rows, cols)
    for steps in (1, 2):
        for bad in (float("nan"), float("inf")):
            test_nan_and_infinity_stay_in_their_matrix(rows, cols, bad, steps)
    test_groups_that_fit_the_workspace(rows, cols)
    test_replayed(rows, cols)
    test_coefficients_and_scale(rows, cols)


@pytest.mark.parametrize("rows,cols", SHORT)
def test_short_sides_within_larger_matrices(rows, cols):
    """Views that start and step at odd elements of a bfloat16 tensor full of NaN elsewhere."""
    say("short views", rows, cols)
    base = torch.full((3, rows + 3, cols + 9), float("nan"), dtype=torch.bfloat16, device="cuda")
    x = base[:, 1:-2, 5:-4]
    x.copy_(stack(3, rows, cols, seed=5))
    held = torch.full((3, rows + 2, cols + 5), 7.0, dtype=torch.bfloat16, device="cuda")
    nsf.muon_orthogonalize_stack(x, held[:, 1:-1, 3:-2])
    check(x, held[:, 1:-1, 3:-2])
    held[:, 1:-1, 3:-2] = 7.0
    assert (held == 7.0).all()


# --------------------------------------------------------------- numbers at the ends of float32

# one workgroup a matrix, strips, tiles of 64 with shared K steps
@pytest.mark.parametrize("rows,cols", [(24, 60), (100, 700), (700, 90), (200, 150)])
@pytest.mark.parametrize("norm", [1.4e-45, 1e-44, 1e-42, 7e-42, 1e-41, 1e-38])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_subnormal_matrices(rows, cols, norm, out):
    """Matrices whose norm is far below 1e-7: every step multiplies by its first coefficient
    (b X^3 is 2^-200 of that).  Roundings, half steps of 2^-24: the norm's reciprocal, its product with U,
    a float16 pair (2), for each of five steps a product and, but for the last, a pair, the scale, its product.
    A pair is also off by half of the smallest float16, 2^-25, where the norm's bound, at most 1.01 times the norm,
    lies between 2^14 and 2^15: 2^-39 of the norm for each of five pairs (where the bound is below 2^-112 and
    the norm therefore stored below 2^14, no number but 0 is below 2, and 2^-25 is less than the first kind)."""
    say("subnormal", rows, cols, norm, out)
    g = torch.Generator().manual_seed(rows)
    u = torch.randn(2, rows, cols, generator=g, dtype=torch.float64)
    if norm < 1e-42:
        u[:, 3:], u[:, :, 4:] = 0, 0
    if norm < 1e-44:
        u[:, :, 1:], u[:, 1:] = 0, 0
    u *= norm / torch.linalg.norm(u, dim=(1, 2), keepdim=True)
    x = u.float().cuda()
    assert (x != 0).any()
    u = x.double().cpu().numpy()
    inverse = 1 / (np.sqrt((u * u).sum(axis=(1, 2), keepdims=True)) + 1e-7)
    for steps, scale in ((nsf.QUINTIC, None), (POLISHED, -0.25), ([], 3.0)):
        o = torch.empty(2, rows, cols, dtype=DT[out], device="cuda")
        nsf.muon_orthogonalize_stack(x, o, coefficients=steps, scale=scale)
        want = u * inverse * (max(1.0, rows / cols) ** 0.5 if scale is None else scale)
        for a, _, _ in steps:
            want = want * float(np.float32(a))
        tol = 20 * 2.0 ** -24 + (2.0 ** -8 if out == "bf16" else 0)
        err = np.abs(o.double().cpu().numpy() - want)
        pairs = 5 * 1.01 * 2.0 ** -39 * np.sqrt((want * want).sum(axis=(1, 2), keepdims=True))
        # (a bfloat16 result below 2^-126 is off by half of 2^-133)
        assert (err <= tol * np.abs(want) + pairs + 2.0 ** -134).all(), (err / (np.abs(want) + 1e-300)).max()


@pytest.mark.parametrize("rows,cols", [(24, 60), (100, 700), (200, 150)])
def test_coefficients_of_unlike_sizes(rows, cols):
    """Polynomials that are nearly zero at the end of their interval, with a last coefficient far
    below the others, and coefficients for an iterate that was shrunk before."""
    x = stack(2, rows, cols, seed=12)
    for steps in ([(2.598, -2.598, 1e-8), (1.5, -0.5, 0.0)], [(2.598, -2.598, -1e-8)] + POLISHED,
                  [(1e-9, 0.0, 0.0), (5.0, -20e18, 16e36)] + POLISHED):
        say("unlike", rows, cols, steps)
        out = torch.empty_like(x)
        nsf.muon_orthogonalize_stack(x, out, coefficients=steps)
        check(x, out, steps)


@pytest.mark.parametrize("count,rows,cols", [(2, 64, 400), (2, 128, 2000), (1, 3000, 100), (1, 1024, 1000)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_largest_finite_matrices(count, rows, cols, dtype):
    """Entries near float32's largest number: a norm whose reciprocal is no normal float32.
    Without steps an element takes four roundings: the reciprocal, two products, the scale."""
    say("largest", count, rows, cols, dtype)
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = 3.3e38 * (0.5 + 0.5 * torch.rand(count, rows, cols, generator=g, device="cuda"))
    x = (x * (torch.randint(0, 2, x.shape, generator=g, device="cuda") * 2 - 1)).to(DT[dtype])
    assert torch.isfinite(x).all()
    scale = max(1.0, rows / cols) ** 0.5
    o = torch.empty(count, rows, cols, device="cuda")
    for steps in ((), nsf.QUINTIC):
        nsf.muon_orthogonalize_stack(x, o, coefficients=steps)
        for k in range(count):
            want = reference(x[k], steps) * scale
            err = (o[k].double() - want).abs()
            if not steps:
                assert (err <= 4 * 2.0 ** -24 * want.abs()).all()
            else:
                tol = 2e-6 + 8 * torch.linalg.norm(reference(x[k], steps, 22) * scale - want) / torch.linalg.norm(want)
                assert torch.linalg.norm(err) <= tol * torch.linalg.norm(want)


# Every way in which a stage is divided among workgroups: tiles of 64, 128 and 256, a workgroup a tile, and K
# steps shared by more or by fewer workgroups than there are tiles (test_stack_scale.py holds the list
# to that); ragged sides, tall and wide
EVERY_TILING = [(1, 131, 132), (84, 237, 201), (39, 989, 648), (1, 2832, 2940), (1, 2026, 2321), (1, 5034, 3274),
                (1, 3274, 5034), (2, 129, 2756), (3, 3231, 3201), (1, 3396, 2414)]


@pytest.mark.parametrize("count,rows,cols", EVERY_TILING)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_every_tiling(count, rows, cols, out):
    say("tiling", count, rows, cols, out)
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = 1e-3 * torch.randn(count, rows, cols, generator=g, device="cuda")
    o, again = (torch.full((count, rows, cols), 7.0, dtype=DT[out], device="cuda") for _ in range(2))
    ws = torch.full((nsf.muon_stack_workspace_bytes(x),), 0xFF, dtype=torch.uint8, device="cuda")
    nsf.muon_orthogonalize_stack(x, o, workspace=ws)
    nsf.muon_orthogonalize_stack(x, again, workspace=ws)
    assert torch.equal(o, again)
    for k in {0, count - 1}:
        want = reference(x[k], nsf.QUINTIC)
        tol = 2e-6 + 8 * torch.linalg.norm(reference(x[k], nsf.QUINTIC, 22) - want) / torch.linalg.norm(want)
        tol += 2.0 ** -8 if out == "bf16" else 0
        want = want * max(1.0, rows / cols) ** 0.5
        assert torch.linalg.norm(o[k].double() - want) <= tol * torch.linalg.norm(want)


@pytest.mark.parametrize("rows,cols", [(24, 60), (100, 700), (200, 150)])
def test_large_coefficients_for_small_matrices(rows, cols):
    """c x^5 is nothing beside a x for an iterate of 1e-27, though c alone is large: what the
    first coefficients leave, within the roundings counted in test_subnormal_matrices."""
    say("large coefficients", rows, cols)
    x = stack(2, rows, cols, seed=13, std=1e-27)
    steps = [(1e-9, 0.0, 0.0), (5.0, 0.0, 1e38), (3.0, -1.0, 0.5)]
    out = torch.empty_like(x)
    nsf.muon_orthogonalize_stack(x, out, coefficients=steps, scale=1.0)
    u = x.double().cpu().numpy()
    want = u / (np.sqrt((u * u).sum(axis=(1, 2), keepdims=True)) + 1e-7)
    for a, _, _ in steps:
        want = want * float(np.float32(a))
    size = np.sqrt((want * want).sum(axis=(1, 2), keepdims=True))
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= 20 * 2.0 ** -24 * np.abs(want) + 3 * 1.01 * 2.0 ** -39 * size).all()
