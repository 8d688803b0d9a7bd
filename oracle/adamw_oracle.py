"""Oracles of the gradient norm, clipping and AdamW (test infrastructure only).

float64 definitions, in exact or compensated sums:

* ``sumsq``: sum of the squares of all elements.  Squares of float32 values are
  exact in float64; ``math.fsum`` rounds their sum once.
* ``coefficient``: ``min(1, max_norm / (sqrt(sumsq) + 1e-6))``, NaN for NaN.
* ``adamw``: the AdamW step (decoupled weight decay, bias-corrected moments)
  from its textbook form, m_hat and v_hat written out.

Same-order float32 chains, against which the device is held bit for bit: each
line is one IEEE-754 binary32 operation rounded to nearest even (NumPy never
fuses a multiply and an add; its float32 division and square root are
correctly rounded).

* ``clip_same_order``:   ``fl(coef * g)``, rounded once more for bfloat16
* ``adamw_same_order``:  ``g' = fl(coef*g)``, ``m = fl(fl(b1*m) + fl(c1*g'))``,
  ``v = fl(fl(b2*v) + fl(fl(c2*g')*g'))``, ``d = fl(fl(sqrt(v)*r) + eps)``,
  ``w = fl(fl(w*f) - fl(a*fl(m/d)))`` with ``c = fl(1 - b)``,
  ``f = fl(1 - fl(lr*wd))``, ``a = fl(lr / (1 - b1^t))`` and
  ``r = fl(1 / sqrt(1 - b2^t))`` in float64, the powers by repeated squaring.

Hyperparameters are float32 values, as the device holds them.
"""

from __future__ import annotations

import math

import numpy as np

from oracle import same_order as so

F32 = np.float32


def sumsq(arrays) -> float:
    """Sum of squares of float32 (or wider) arrays, rounded once."""
    wide = [np.asarray(a, dtype=np.float64).ravel() for a in arrays]
    if any(np.isnan(a).any() for a in wide):
        return math.nan
    if any(np.isinf(a).any() for a in wide):
        return math.inf
    return math.fsum(x for a in wide for x in (a * a).tolist())


def coefficient(s: float, max_norm: float) -> float:
    """min(1, max_norm / (sqrt(s) + 1e-6)); max_norm as a float32 value."""
    m = float(F32(max_norm))
    if math.isnan(s):
        return math.nan
    norm = math.sqrt(s)
    if math.isinf(norm):
        return math.nan if math.isinf(m) else 0.0
    return min(1.0, m / (norm + 1e-6))


def widen(a: np.ndarray) -> np.ndarray:
    """float32 values of a float32 array or of bfloat16 bits (uint16)."""
    return so.bf16_bits_to_f32(a) if a.dtype == np.uint16 else a.astype(np.float32, copy=False)


def clip_same_order(src: np.ndarray, coef, out_dtype: str) -> np.ndarray:
    with np.errstate(all="ignore"):
        v = (F32(coef) * widen(src)).astype(np.float32)
    return so.f32_to_bf16_bits(v) if out_dtype == "bf16" else v


def power(b: float, t: int) -> float:
    p = 1.0
    while t:
        if t & 1:
            p *= b
        b *= b
        t >>= 1
    return p


def adamw_same_order(w, g, m, v, group, coef=None):
    """New (w, m, v); w and g are float32 or bfloat16 bits, group is (lr, wd, beta1,
    beta2, eps, step).  w comes back in its own representation."""
    lr, wd, b1, b2, eps = (F32(x) for x in group[:5])
    t = int(group[5])
    gc = (F32(1.0) if coef is None else F32(coef)) * widen(g)
    one = F32(1.0)
    c1, c2 = one - b1, one - b2
    f = one - F32(lr * wd)
    a = F32(float(lr) / (1.0 - power(float(b1), t)))
    r = F32(1.0 / math.sqrt(1.0 - power(float(b2), t)))
    with np.errstate(all="ignore"):
        m1 = b1 * m + c1 * gc
        v1 = b2 * v + (c2 * gc) * gc
        d = np.sqrt(v1) * r + eps
        wn = widen(w) * f - a * (m1 / d)
    out = so.f32_to_bf16_bits(wn) if w.dtype == np.uint16 else wn
    return out, m1, v1


def adamw(w, g, m, v, group, coef: float = 1.0):
    """New (w, m, v) in float64."""
    lr, wd, b1, b2, eps = (float(F32(x)) for x in group[:5])
    t = int(group[5])
    w, g, m, v = (np.asarray(widen(x) if x.dtype == np.uint16 else x, dtype=np.float64)
                  for x in (w, g, m, v))
    g = g * float(coef)
    m = b1 * m + (1.0 - b1) * g
    v = b2 * v + (1.0 - b2) * g * g
    m_hat = m / (1.0 - b1 ** t)
    v_hat = v / (1.0 - b2 ** t)
    w = w - lr * wd * w - lr * m_hat / (np.sqrt(v_hat) + eps)
    return w, m, v
