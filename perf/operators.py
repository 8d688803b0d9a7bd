"""The gradient-norm, clipping and AdamW operators, as cases to be measured.

Three operators over flat optimizer buffers:

``norm``   the global 2-norm of many gradient tensors, with the clipping
           coefficient min(1, max_norm / (norm + 1e-6)) (and, on demand, the
           norm of each tensor)
``clip``   the same norm, then every gradient times the coefficient, written
           to another buffer (float32 gradients for the optimizer)
``adamw``  one AdamW step on flat buffers in ranges, the gradient multiplied
           by the clipping coefficient as it is read

With ``own`` false ``run`` computes them in elementary torch operations; with
``own`` true it calls the framework.
"""

import math
import random

import numpy as np
import torch

own = False

#: The seven matrices of one 4096-hidden decoder layer, by number of elements.
LAYER = [4096 * 4096, 1024 * 4096, 1024 * 4096, 4096 * 4096, 14336 * 4096, 14336 * 4096,
         4096 * 14336]
#: 128 expert matrices and two dense ones.
EXPERTS = [2048 * 7168] * 128 + [7168 * 18432] * 2

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


def f32(x):
    """A hyperparameter as the device holds it: rounded to float32."""
    return float(np.float32(x))


def sizes(case):
    """Numbers of elements of the case's tensors."""
    if case["set"] == "layers":
        return LAYER * case["count"]
    if case["set"] == "experts":
        return EXPERTS
    if case["set"] == "equal":
        return [case["hi"]] * case["count"]
    r = random.Random(case["mix"])
    lo, hi = math.log(case["lo"]), math.log(case["hi"])
    return [int(round(math.exp(r.uniform(lo, hi)))) for _ in range(case["count"])]


def layout(case):
    """(offset, size) of every tensor in the flat buffer, and the buffer's
    length.  "pad" is the alignment in elements: 64 as in the optimizer's flat
    buffers, 1 where tensors are packed one behind the other."""
    at, off, pad = [], 0, case["pad"]
    for n in sizes(case):
        at.append((off, n))
        off = -(-(off + n) // pad) * pad
    return at, off


def listed():
    return [
        # the norm weights and biases of a few small layers: nothing but latency
        {"name": "norm_vectors", "op": "norm", "set": "range", "count": 9, "lo": 64, "hi": 1024,
         "mix": 1, "pad": 64, "dtype": "f32", "std": 0.05, "each": False},
        # one decoder layer's bfloat16 gradients, with the norm of each matrix for the log
        {"name": "norm_layer_bf16", "op": "norm", "set": "layers", "count": 1, "pad": 64,
         "dtype": "bf16", "std": 1e-3, "each": True},
        # a bucket of 512 odd-sized tensors packed without padding (odd addresses)
        {"name": "norm_packed_512", "op": "norm", "set": "range", "count": 512, "lo": 16384,
         "hi": 1048576, "mix": 9, "pad": 1, "dtype": "f32", "std": 1e-3, "each": False},
        # the whole owner share of a 32-layer model: 7 G float32 gradients
        {"name": "norm_owner_share", "op": "norm", "set": "layers", "count": 32, "pad": 64,
         "dtype": "f32", "std": 1e-3, "each": False},
        # the small vectors again, clipped
        {"name": "clip_vectors", "op": "clip", "set": "range", "count": 9, "lo": 64, "hi": 1024,
         "mix": 2, "pad": 64, "dtype": "f32", "out": "f32", "std": 0.05},
        # one layer's bfloat16 gradients, clipped into the float32 buffer that the step reads
        {"name": "clip_layer_bf16", "op": "clip", "set": "layers", "count": 1, "pad": 64,
         "dtype": "bf16", "out": "f32", "std": 1e-3},
        # the packed bucket, odd addresses on both sides
        {"name": "clip_packed_512", "op": "clip", "set": "range", "count": 512, "lo": 16384,
         "hi": 1048576, "mix": 9, "pad": 1, "dtype": "f32", "out": "f32", "std": 1e-3},
        # the expert matrices' float32 gradients: 2.1 G elements
        {"name": "clip_experts", "op": "clip", "set": "experts", "pad": 64, "dtype": "f32",
         "out": "f32", "std": 1e-3},
        # 65 norm weights of width 4096, float32: latency
        {"name": "adamw_vectors", "op": "adamw", "set": "equal", "count": 65, "hi": 4096, "pad": 64,
         "dtype": "f32", "weights": "f32", "copy": False, "groups": 1, "std": 1e-2},
        # odd-sized tensors in three groups, bfloat16 weights and gradients
        {"name": "adamw_ragged_groups", "op": "adamw", "set": "range", "count": 200, "lo": 100,
         "hi": 400000, "mix": 5, "pad": 64, "dtype": "bf16", "weights": "bf16", "copy": False,
         "groups": 3, "std": 1e-3},
        # an embedding of 32000 x 4096, bfloat16 weights, float32 gradients
        {"name": "adamw_embedding", "op": "adamw", "set": "equal", "count": 1, "hi": 32000 * 4096,
         "pad": 64, "dtype": "f32", "weights": "bf16", "copy": False, "groups": 1, "std": 1e-3},
        # embedding and head of 128000 x 4096: float32 weights with the model's bfloat16 copy
        {"name": "adamw_master_copy", "op": "adamw", "set": "equal", "count": 2,
         "hi": 128000 * 4096, "pad": 64, "dtype": "f32", "weights": "f32", "copy": True,
         "groups": 2, "std": 1e-3},
    ]


def draw(rng):
    op = rng.choice(["norm", "clip", "adamw"])
    most = {"norm": 1 << 31, "clip": 1 << 30, "adamw": 1 << 29}[op]
    total = int(math.exp(rng.uniform(math.log(2000), math.log(most))))
    count = max(1, min(int(math.exp(rng.uniform(0, math.log(700)))), total // 16))
    mean = max(2, total // count)
    case = {"op": op, "set": "range", "count": count, "lo": max(1, mean // 8), "hi": 2 * mean,
            "mix": rng.randrange(1 << 20), "dtype": rng.choice(["f32", "bf16"]),
            # clipped as a rule, now and then below the largest norm
            "std": float("%.3g" % (rng.uniform(0.5, 12.0) / math.sqrt(total)))}
    if op == "adamw":
        case["pad"] = rng.choice([8, 64])
        case["weights"] = rng.choice(["f32", "bf16"])
        case["copy"] = case["weights"] == "f32" and rng.random() < 0.5
        case["groups"] = rng.randint(1, min(4, count))
    else:
        case["pad"] = rng.choice([1, 4, 64])
        if op == "norm":
            case["each"] = count <= 16 and rng.random() < 0.5
        else:
            case["out"] = rng.choice(["f32", "bf16"])
    return case


MAX_NORM = 1.0


def hyper(k):
    """(lr, weight_decay, beta1, beta2, eps, step) of group k, as float32 values."""
    return (f32(1e-3 / (k + 1)), f32(0.1 if k % 2 == 0 else 0.0), f32(0.9), f32(0.95 if k % 2 else 0.999),
            f32(1e-8), 100 + k)


def group_of(i, case):
    """Tensors of a group lie together: the first share of them is group 0, and so on."""
    return i * case["groups"] // case["count"]


def gradients(case, at, length, gen):
    flat = torch.zeros(length, dtype=TYPES[case["dtype"]], device="cuda")
    for off, n in at:
        flat[off:off + n].normal_(0.0, case["std"], generator=gen)
    return flat


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    at, length = layout(case)
    s = {"case": case, "at": at, "grads": gradients(case, at, length, gen)}
    views = [s["grads"][o:o + n] for o, n in at]
    if case["op"] == "adamw":
        std = 0.02
        w = torch.zeros(length, dtype=TYPES[case["weights"]], device="cuda")
        m = torch.zeros(length, dtype=torch.float32, device="cuda")
        v = torch.zeros(length, dtype=torch.float32, device="cuda")
        for o, n in at:
            w[o:o + n].normal_(0.0, std, generator=gen)
            m[o:o + n].normal_(0.0, 0.3 * case["std"], generator=gen)
            # a second moment near the gradients' own square, never below it by much
            v[o:o + n].normal_(0.0, 0.2, generator=gen).add_(1.0).abs_().add_(0.05).mul_(case["std"] ** 2)
        s.update(weights=w, m=m, v=v, coef=torch.rand((), generator=gen, device="cuda") * 0.8 + 0.1)
        s["copy"] = torch.zeros(length, dtype=torch.bfloat16, device="cuda") if case["copy"] else None
        # one slice of the flat buffers per group
        s["slices"] = []
        for k in range(case["groups"]):
            mine = [i for i in range(case["count"]) if group_of(i, case) == k]
            s["slices"].append((at[mine[0]][0], at[mine[-1]][0] + at[mine[-1]][1]))
    elif case["op"] == "clip":
        s["out"] = torch.zeros(length, dtype=TYPES[case["out"]], device="cuda")
    if own:
        import newton_schulz_flat_amd as nsf
        s["nsf"] = nsf
        s["record"] = nsf.clip_state("cuda")
        if case["op"] == "adamw":
            nsf.clip_coef(s["record"]).copy_(s["coef"])
            s["table"] = nsf.adamw_group_table([hyper(k) for k in range(case["groups"])], "cuda")
            s["ranges"] = nsf.ranges_array([(o, n, o, group_of(i, case)) for i, (o, n) in enumerate(at)])
        else:
            s["tensors"] = nsf.tensor_list(views)
            s["norms"] = torch.zeros(len(at), device="cuda") if case.get("each") else None
            if case["op"] == "clip":
                s["out_tensors"] = nsf.tensor_list([s["out"][o:o + n] for o, n in at])
            s["workspace"] = torch.empty(nsf.muon_clip_workspace_bytes(s["tensors"]),
                                         dtype=torch.uint8, device="cuda")
    return s


def plain_norm(s):
    # the flat buffer is zero between tensors, so its norm is theirs; sums of
    # billions of squares are taken in 64 bits
    total = s["grads"].float().square().sum(dtype=torch.float64)
    norm = total.sqrt()
    coef = torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0)
    return norm.float(), coef.float()


def plain_adamw(s):
    w, g, m, v = s["weights"], s["grads"], s["m"], s["v"]
    for k, (a, b) in enumerate(s["slices"]):
        lr, decay, b1, b2, eps, t = hyper(k)
        gk = g[a:b].float() * s["coef"]
        m[a:b] = b1 * m[a:b] + (1 - b1) * gk
        v[a:b] = b2 * v[a:b] + (1 - b2) * gk * gk
        root = v[a:b].sqrt() / math.sqrt(1 - b2 ** t) + eps
        new = w[a:b].float() * (1 - lr * decay) - lr / (1 - b1 ** t) * m[a:b] / root
        w[a:b] = new
        if s["copy"] is not None:
            s["copy"][a:b] = new
    return [x for x in (w, m, v, s["copy"]) if x is not None]


def run(s):
    op = s["case"]["op"]
    if not own:
        if op == "adamw":
            return plain_adamw(s)
        norm, coef = plain_norm(s)
        if op == "clip":
            s["out"].copy_(s["grads"].float() * coef)
            return norm, coef, s["out"]
        if s["case"]["each"]:
            each = torch.stack([s["grads"][o:o + n].float().square().sum(dtype=torch.float64)
                                for o, n in s["at"]]).sqrt().float()
            return norm, coef, each
        return norm, coef
    nsf = s["nsf"]
    if op == "adamw":
        nsf.muon_adamw(s["weights"], s["grads"], s["m"], s["v"], s["ranges"], s["table"],
                       clip=s["record"], model_copy=s["copy"])
        return [x for x in (s["weights"], s["m"], s["v"], s["copy"]) if x is not None]
    nsf.muon_grad_norm(s["tensors"], MAX_NORM, s["record"], tensor_norms=s["norms"],
                       workspace=s["workspace"])
    result = (nsf.clip_norm(s["record"]), nsf.clip_coef(s["record"]))
    if op == "clip":
        nsf.muon_clip_grads(s["tensors"], s["record"], out=s["out_tensors"])
        return result + (s["out"],)
    return result + ((s["norms"],) if s["norms"] is not None else ())


def work(case):
    n = sum(sizes(case))
    g = SIZE[case["dtype"]]
    if case["op"] == "norm":
        return {"bytes": n * g, "flops": 2 * n}
    if case["op"] == "clip":
        return {"bytes": n * (g + SIZE[case["out"]]), "flops": 3 * n}
    per = g + 2 * SIZE[case["weights"]] + 16 + (2 if case["copy"] else 0)
    return {"bytes": n * per, "flops": 16 * n}


def exact(case, seed):
    """The operators from their definitions, in float64, tensor by tensor."""
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    wide = {i: s["grads"].narrow(0, o, n) for i, (o, n) in enumerate(s["at"])}
    if case["op"] == "adamw":
        w, m, v = (torch.zeros(x.numel(), dtype=torch.float64, device="cuda")
                   for x in (s["weights"], s["m"], s["v"]))
        for i, (o, n) in enumerate(s["at"]):
            lr, decay, b1, b2, eps, t = hyper(group_of(i, case))
            g = torch.mul(wide[i].double(), s["coef"].double())
            m[o:o + n] = torch.lerp(g, s["m"][o:o + n].double(), b1)
            v[o:o + n] = torch.lerp(torch.pow(g, 2), s["v"][o:o + n].double(), b2)
            mhat = m[o:o + n] / -math.expm1(t * math.log(b1))
            vhat = v[o:o + n] / -math.expm1(t * math.log(b2))
            old = s["weights"][o:o + n].double()
            w[o:o + n] = old - lr * decay * old - lr * (mhat / (torch.sqrt(vhat) + eps))
        return [w, m, v] + ([w] if case["copy"] else [])
    each = torch.stack([torch.linalg.vector_norm(wide[i].double()) for i in sorted(wide)])
    norm = torch.linalg.vector_norm(each)
    coef = torch.minimum(torch.ones_like(norm), MAX_NORM / (norm + 1e-6))
    if case["op"] == "clip":
        out = torch.zeros(s["out"].numel(), dtype=torch.float64, device="cuda")
        for i, (o, n) in enumerate(s["at"]):
            torch.mul(wide[i].double(), coef, out=out[o:o + n])
        return norm, coef, out
    return (norm, coef, each) if case["each"] else (norm, coef)
