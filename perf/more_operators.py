"""8-bit products with a scale for each block of 128, the casts that feed them, and
orthogonalisation of stacks of matrices in float32 accuracy, as cases to be measured.

Three operators around the training step of linear layers:

``cast``     a matrix (float32 master weights, bfloat16 activations or gradients)
             into 8-bit floats with one scale for each 1 x 128 or 128 x 128
             block, and the same of its transpose
``product``  out (+)= A B^T of two such matrices, along their blocks: a layer's
             forward product, the gradient of its input, and the gradient of its
             weight, added into the optimizer's float32 gradient buffer
``ortho``    the Newton-Schulz orthogonalisation of a stack of equal matrices,
             float32 or bfloat16, with strides, with coefficients for each step

With ``own`` false ``run`` computes them in elementary torch operations; with
``own`` true it calls the framework.
"""

import math

import torch

own = False

BLOCK = 128
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
FORMATS = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
#: Blocks whose largest magnitude is below this take the scale of this.
FLOOR = 2.0 ** -100

QUINTIC = (3.4445, -4.7750, 2.0315)
#: Step coefficients: five equal steps, or three of them and two of the polynomial
#: (15 x - 10 x^3 + 3 x^5) / 8, which has 1 as a fixed point.
SCHEDULES = {"quintic": [QUINTIC] * 5, "polished": [QUINTIC] * 3 + [(1.875, -1.25, 0.375)] * 2}


def blocks(n):
    return -(-n // BLOCK)


def listed():
    return [
        # one token's activations on the way into a product: nothing but latency
        {"name": "cast_token", "op": "cast", "rows": 1, "cols": 4096, "dtype": "bf16", "square": False,
         "format": "e4m3", "both": False, "pad": 0},
        # a batch of activations, by rows for the product and transposed for the weight's gradient
        {"name": "cast_activations", "op": "cast", "rows": 8192, "cols": 4096, "dtype": "bf16",
         "square": False, "format": "e4m3", "both": True, "pad": 0},
        # a layer's float32 master weight in 128 x 128 blocks, with its transpose for the backward pass
        {"name": "cast_weight", "op": "cast", "rows": 14336, "cols": 4096, "dtype": "f32",
         "square": True, "format": "e4m3", "both": True, "pad": 0},
        # one token through a layer
        {"name": "product_token", "op": "product", "m": 1, "n": 4096, "k": 14336, "a_square": False,
         "b_square": True, "a_format": "e4m3", "out": "bf16", "add": False, "pad": 0},
        # an odd number of tokens and odd sides
        {"name": "product_odd", "op": "product", "m": 333, "n": 1025, "k": 1999, "a_square": False,
         "b_square": True, "a_format": "e4m3", "out": "f32", "add": False, "pad": 0},
        # the tokens of one expert, 7168 wide
        {"name": "product_expert", "op": "product", "m": 600, "n": 2048, "k": 7168, "a_square": False,
         "b_square": True, "a_format": "e4m3", "out": "bf16", "add": False, "pad": 0},
        # the forward product of a layer's largest matrix
        {"name": "product_forward", "op": "product", "m": 8192, "n": 14336, "k": 4096,
         "a_square": False, "b_square": True, "a_format": "e4m3", "out": "bf16", "add": False, "pad": 0},
        # its weight's gradient over 8192 tokens (gradients in e5m2), added to the flat float32 buffer
        {"name": "product_weight_gradient", "op": "product", "m": 14336, "n": 4096, "k": 8192,
         "a_square": False, "b_square": False, "a_format": "e5m2", "out": "f32", "add": True, "pad": 0},
        # small matrices, one launch
        {"name": "ortho_small", "op": "ortho", "count": 16, "rows": 48, "cols": 64, "dtype": "f32",
         "out": "f32", "steps": "quintic", "pad": 0},
        # the heads of a query projection, each orthogonalised on its own
        {"name": "ortho_heads", "op": "ortho", "count": 32, "rows": 128, "cols": 4096, "dtype": "bf16",
         "out": "bf16", "steps": "quintic", "pad": 0},
        # odd tall matrices in rows longer than they are
        {"name": "ortho_odd", "op": "ortho", "count": 6, "rows": 1111, "cols": 777, "dtype": "f32",
         "out": "f32", "steps": "polished", "pad": 23},
        # a layer's largest matrix
        {"name": "ortho_layer", "op": "ortho", "count": 1, "rows": 14336, "cols": 4096, "dtype": "f32",
         "out": "bf16", "steps": "quintic", "pad": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _side(rng, lo, hi):
    """A side of a matrix: any, or (as most models have them) a multiple of 64."""
    n = _log(rng, lo, hi)
    return max(64, n // 64 * 64) if rng.random() < 0.5 else n


def _products(rows, cols):
    """Operations of one step of an orthogonalisation, its two symmetric products by one
    triangle each."""
    r, c = sorted((rows, cols))
    return r * (r + 1) * (c + r) + 2 * r * r * c


def draw(rng):
    op = rng.choice(["cast", "product", "ortho"])
    if op == "cast":
        rows, cols = _log(rng, 1, 16384), _side(rng, 64, 16384)
        while rows * cols > 14336 * 4096:
            rows, cols = max(1, rows // 2), max(64, cols * 3 // 4)
        return {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(["f32", "bf16"]),
                "square": rng.random() < 0.5, "format": rng.choice(["e4m3", "e4m3", "e5m2"]),
                "both": rng.random() < 0.5, "pad": rng.choice([0, 0, 5, 64])}
    if op == "product":
        m, n, k = _log(rng, 1, 16384), _side(rng, 64, 16384), _side(rng, 64, 16384)
        while m * n * k > 8192 * 14336 * 4096:
            m, n, k = max(1, m * 2 // 3), max(64, n * 3 // 4), max(64, k * 3 // 4)
        add = rng.random() < 0.3
        return {"op": op, "m": m, "n": n, "k": k, "a_square": rng.random() < 0.2,
                "b_square": rng.random() < 0.6, "a_format": rng.choice(["e4m3", "e4m3", "e5m2"]),
                "out": "f32" if add else rng.choice(["f32", "bf16"]), "add": add,
                "pad": rng.choice([0, 0, 16, 37])}
    rows, cols = _side(rng, 1, 8192), _side(rng, 1, 8192)
    while _products(rows, cols) > _products(14336, 4096):
        rows, cols = rows * 3 // 4, cols * 3 // 4
    count = _log(rng, 1, max(1.0, min(512.0, _products(14336, 4096) / 3 / _products(rows, cols))))
    return {"op": op, "count": count, "rows": rows, "cols": cols, "dtype": rng.choice(["f32", "bf16"]),
            "out": rng.choice(["f32", "bf16"]), "steps": rng.choice(["quintic", "polished"]),
            "pad": rng.choice([0, 0, 23])}


def matrix(rows, cols, dtype, gen, kind, pad=0):
    """Values as they are met: weights of one size, activations with channels of very
    different sizes, gradients with rows (tokens) of different sizes."""
    x = torch.randn(rows, cols + pad, generator=gen, device="cuda")
    if kind == "weight":
        x *= 0.02
    elif kind == "activation":
        x *= torch.randn(cols + pad, generator=gen, device="cuda").exp()
    else:
        x *= 1e-4 * torch.randn(rows, 1, generator=gen, device="cuda").exp()
    return x.to(dtype)[:, :cols]


def block_view(x, square):
    """x, padded with zeros to whole blocks, as (row blocks, rows of one, column blocks, 128)."""
    rows, cols = x.shape
    high = BLOCK if square else 1
    x = torch.nn.functional.pad(x, (0, blocks(cols) * BLOCK - cols, 0, -rows % high))
    return x.reshape(-1, high, blocks(cols), BLOCK)


def quantise(x, fmt, square):
    """Codes and scales: a block's scale is its largest magnitude over the format's largest
    number, a code the number nearest to the value times the scale's reciprocal."""
    rows, cols = x.shape
    v = block_view(x.float(), square)
    scales = v.abs().amax(dim=(1, 3)).clamp(min=FLOOR) / LARGEST[fmt]
    q = (v * (1.0 / scales)[:, None, :, None]).clamp(-LARGEST[fmt], LARGEST[fmt])
    return q.reshape(-1, blocks(cols) * BLOCK)[:rows, :cols].to(FORMATS[fmt]), scales


def widen(codes, scales, square, dtype):
    """The numbers that codes and scales stand for."""
    rows, cols = codes.shape
    s = scales.to(dtype)
    if square:
        s = s.repeat_interleave(BLOCK, 0)[:rows]
    return codes.to(dtype) * s.repeat_interleave(BLOCK, 1)[:, :cols]


def operand(rows, cols, fmt, square, gen, kind, pad):
    """An operand of a product: codes (in rows that may be longer) and scales, block-major."""
    codes, scales = quantise(matrix(rows, cols, torch.float32, gen, kind), fmt, square)
    held = torch.zeros(rows, cols + pad, dtype=codes.dtype, device="cuda")[:, :cols]
    held.copy_(codes)
    return held, scales.t().contiguous().t()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if own:
        import newton_schulz_flat_amd as nsf
        s["nsf"] = nsf
    if case["op"] == "cast":
        rows, cols = case["rows"], case["cols"]
        kind = "weight" if case["square"] else "activation" if case["format"] == "e4m3" else "gradient"
        s["x"] = matrix(rows, cols, TYPES[case["dtype"]], gen, kind, case["pad"])
        if own:
            s["out"] = [(torch.empty(a, b, dtype=FORMATS[case["format"]], device="cuda"),
                         nsf.fp8_scales(a, b, "square" if case["square"] else "row", "cuda"))
                        for a, b in [(rows, cols)] + [(cols, rows)] * case["both"]]
    elif case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], s["a_scales"] = operand(m, k, case["a_format"], case["a_square"], gen,
                                        "gradient" if case["add"] else "activation", case["pad"])
        s["b"], s["b_scales"] = operand(n, k, "e4m3", case["b_square"], gen,
                                        "weight" if case["b_square"] else "activation", case["pad"])
        s["out"] = torch.zeros(m, n, dtype=TYPES[case["out"]], device="cuda")
        if case["add"]:
            s["out"].normal_(0.0, 1e-3, generator=gen)
        if own:
            s["workspace"] = torch.empty(nsf.muon_fp8_workspace_bytes(m, n, k), dtype=torch.uint8,
                                         device="cuda")
    else:
        count, rows, cols = case["count"], case["rows"], case["cols"]
        wide = cols + case["pad"]
        # noise, and a few directions that stand out of it
        x = torch.randn(count, rows, wide, generator=gen, device="cuda")
        left = torch.randn(count, rows, 4, generator=gen, device="cuda")
        right = torch.randn(count, 4, wide, generator=gen, device="cuda")
        x += left @ right
        s["x"] = (1e-3 * x).to(TYPES[case["dtype"]])[:, :, :cols]
        s["out"] = torch.empty(count, rows, cols, dtype=TYPES[case["out"]], device="cuda")
        if own:
            s["workspace"] = torch.empty(nsf.muon_stack_workspace_bytes(s["x"]), dtype=torch.uint8,
                                         device="cuda")
    return s


def shape_scale(case):
    return math.sqrt(max(1.0, case["rows"] / case["cols"]))


def plain_ortho(s):
    case = s["case"]
    x = s["x"].float()
    if case["rows"] > case["cols"]:
        x = x.transpose(1, 2).contiguous()
    norm = x.square().sum(dim=(1, 2), dtype=torch.float64, keepdim=True).sqrt()
    x = x * (1.0 / (norm + 1e-7)).float()
    for a, b, c in SCHEDULES[case["steps"]]:
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    x = x * shape_scale(case)
    if case["rows"] > case["cols"]:
        x = x.transpose(1, 2)
    s["out"].copy_(x)
    return s["out"]


def run(s):
    case = s["case"]
    if case["op"] == "cast":
        if not own:
            result = quantise(s["x"], case["format"], case["square"])
            if case["both"]:
                result += quantise(s["x"].t(), case["format"], case["square"])
            return result
        out = s["out"]
        s["nsf"].muon_fp8_cast(s["x"], *out[0], *(out[1] if case["both"] else ()))
        return tuple(t for pair in out for t in pair)
    if case["op"] == "product":
        if not own:
            a = widen(s["a"], s["a_scales"], case["a_square"], torch.float32)
            b = widen(s["b"], s["b_scales"], case["b_square"], torch.float32)
            if case["add"]:
                s["out"] += a @ b.t()
            else:
                s["out"].copy_(a @ b.t())
            return s["out"]
        s["nsf"].muon_fp8_matmul(s["a"], s["a_scales"], s["b"], s["b_scales"], s["out"],
                                 accumulate=case["add"], workspace=s["workspace"])
        return s["out"]
    if not own:
        return plain_ortho(s)
    s["nsf"].muon_orthogonalize_stack(s["x"], s["out"], coefficients=SCHEDULES[case["steps"]],
                                      workspace=s["workspace"])
    return s["out"]


def work(case):
    if case["op"] == "cast":
        n, sides = case["rows"] * case["cols"], 1 + case["both"]
        if case["square"]:
            scales = sides * blocks(case["rows"]) * blocks(case["cols"])
        else:
            scales = case["rows"] * blocks(case["cols"])
            scales += case["both"] * case["cols"] * blocks(case["rows"])
        return {"bytes": n * (SIZE[case["dtype"]] + sides) + 4 * scales, "flops": 3 * n}
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        scales = sum((blocks(r) if sq else r) * blocks(k)
                     for r, sq in ((m, case["a_square"]), (n, case["b_square"])))
        return {"bytes": (m + n) * k + 4 * scales + m * n * SIZE[case["out"]] * (1 + case["add"]),
                "flops": 2 * m * n * k}
    n = case["count"] * case["rows"] * case["cols"]
    return {"bytes": n * (SIZE[case["dtype"]] + SIZE[case["out"]]),
            "flops": case["count"] * len(SCHEDULES[case["steps"]]) * _products(case["rows"], case["cols"])}


def exact_cast(x, fmt, square):
    """Block by block along the columns, in float64; the nearest 8-bit number is looked up
    in the sorted list of them."""
    numbers = torch.arange(256, dtype=torch.uint8, device="cuda").view(FORMATS[fmt]).double()
    numbers = torch.unique(numbers[numbers.isfinite()])
    middles = (numbers[1:] + numbers[:-1]) / 2
    rows, cols = x.shape
    codes, scales = [], []
    for at in range(0, cols, BLOCK):
        part = x[:, at:at + BLOCK].double()
        top = part.abs().max(dim=1).values
        if square:
            top = torch.cat([t.max().expand(t.numel()) for t in top.split(BLOCK)])
        scale = torch.maximum(top, top.new_tensor(FLOOR)) / numbers[-1]
        codes.append(numbers[torch.bucketize(part / scale[:, None], middles)])
        scales.append(scale[::BLOCK] if square else scale)
    return torch.cat(codes, dim=1), torch.stack(scales, dim=1)


def exact(case, seed):
    """The operators from their definitions, in float64."""
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    if case["op"] == "cast":
        result = exact_cast(s["x"], case["format"], case["square"])
        if case["both"]:
            result += exact_cast(s["x"].t(), case["format"], case["square"])
        return result
    if case["op"] == "product":
        total = s["out"].double() if case["add"] else torch.zeros(case["m"], case["n"],
                                                                  dtype=torch.float64, device="cuda")
        row_a = torch.arange(case["m"], device="cuda") // (BLOCK if case["a_square"] else 1)
        row_b = torch.arange(case["n"], device="cuda") // (BLOCK if case["b_square"] else 1)
        for j in range(blocks(case["k"])):
            at = slice(j * BLOCK, (j + 1) * BLOCK)
            part = torch.mm(s["a"][:, at].double(), s["b"][:, at].double().t().contiguous())
            part *= s["a_scales"][row_a, j].double()[:, None]
            total += part.mul_(s["b_scales"][row_b, j].double())
        return total
    # through the singular values of a few small matrices, else by the iteration itself
    out = []
    for m in s["x"]:
        m = m.double()
        m = m / (torch.linalg.matrix_norm(m) + 1e-7)
        tall = m.shape[0] > m.shape[1]
        w = m.mT.contiguous() if tall else m
        if w.shape[0] <= 64 and case["count"] <= 16:
            u, t, v = torch.linalg.svd(w, full_matrices=False)
            for a, b, c in SCHEDULES[case["steps"]]:
                t = t * (a + t * t * (b + c * t * t))
            w = (u * t) @ v
        else:
            eye = torch.eye(w.shape[0], dtype=torch.float64, device="cuda")
            for a, b, c in SCHEDULES[case["steps"]]:
                g = torch.mm(w, w.mT.contiguous())
                w = torch.mm(torch.addmm(a * eye, b * eye + c * g, g), w)
        out.append((w.mT if tall else w) * shape_scale(case))
    return torch.stack(out)
