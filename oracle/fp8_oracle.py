"""8-bit casts and products, and the pairs of float16, in plain NumPy: test infrastructure only.

The 8-bit numbers are worked out from the formats' definition (sign, exponent,
mantissa), codes by comparison with the middles between them, ties to the even
code."""

import numpy as np

BLOCK = 128
FLOOR = np.float32(2.0 ** -100)
#: (exponent bits, mantissa bits, bias, largest code of a finite number)
FORMATS = {"e4m3": (4, 3, 7, 0x7E), "e5m2": (5, 2, 15, 0x7B)}


def numbers(fmt):
    """The number of every code 0 .. largest (positive ones), in float64."""
    _, man, bias, last = FORMATS[fmt]
    code = np.arange(last + 1)
    e, m = code >> man, code & ((1 << man) - 1)
    return np.where(e == 0, m * 2.0 ** (1 - bias - man),
                    (1 + m / 2.0 ** man) * 2.0 ** (e.astype(float) - bias))


def decode(codes, fmt):
    """Values of uint8 codes of finite numbers, in float64."""
    codes = np.asarray(codes, np.uint8)
    return np.where(codes & 0x80, -1.0, 1.0) * numbers(fmt)[codes & 0x7F]


def encode(x, fmt):
    """Codes of float values no larger than the format's largest (up to half a step)."""
    v = numbers(fmt)
    mag = np.abs(np.asarray(x, np.float64))
    middle = (v[1:] + v[:-1]) / 2
    low = np.searchsorted(middle, mag, side="left")   # middle[low - 1] < mag <= middle[low]
    tie = (low < len(middle)) & (mag == middle[np.minimum(low, len(middle) - 1)])
    code = np.where(tie & (low % 2 == 1), low + 1, low).astype(np.uint8)
    return code | (np.signbit(x).astype(np.uint8) << 7)


def blocks(n):
    return -(-n // BLOCK)


def cast(x, fmt, square):
    """(codes, scales) of a float32 matrix: scales in float32, codes of x top / m itself.  (In
    float64 x top is exact, and where the quotient is the middle of two codes, so is it; others
    lie 2^-29 beside one at least.)"""
    x = np.asarray(x, np.float32)
    rows, cols = x.shape
    high = BLOCK if square else 1
    codes = np.zeros((rows, cols), np.uint8)
    scales = np.zeros((-(-rows // high), blocks(cols)), np.float32)
    top = np.float32(numbers(fmt)[-1])
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            part = x[i * high:(i + 1) * high, j * BLOCK:(j + 1) * BLOCK]
            m = np.float32(max(np.max(np.abs(part)), FLOOR))
            scales[i, j] = m / top
            codes[i * high:(i + 1) * high, j * BLOCK:(j + 1) * BLOCK] = encode(
                part.astype(np.float64) * np.float64(top) / np.float64(m), fmt)
    return codes, scales


def widen(codes, scales, fmt):
    """The float64 numbers that codes and scales stand for."""
    v = decode(codes, fmt)
    s = np.asarray(scales, np.float64)
    if s.shape[0] != v.shape[0]:
        s = np.repeat(s, BLOCK, axis=0)[:v.shape[0]]
    return v * np.repeat(s, BLOCK, axis=1)[:, :v.shape[1]]


def product_bound(a, b):
    """Bound on the float32 roundings of one product element: a block's sum takes 128
    additions at most, the outer sum two multiplications and one addition a block, each off by
    2^-24 of a partial sum that is no larger than the sum of magnitudes."""
    steps = BLOCK + blocks(a.shape[1]) + 4
    return steps * 2.0 ** -24 * (np.abs(a) @ np.abs(b).T)


def cut_bound(a, b):
    """Bound on what the 8-bit matrix instruction cuts off: each of the 7 other products of a
    group of 8 (however the instruction groups a block's 128) loses at most 2^-13 of the
    group's largest, and no group's largest exceeds its block's."""
    total = 0.0
    for at in range(0, a.shape[1], BLOCK):
        x, y = np.abs(a[:, at:at + BLOCK]), np.abs(b[:, at:at + BLOCK])
        top = np.zeros((x.shape[0], y.shape[0]))
        for k in range(x.shape[1]):
            np.maximum(top, np.outer(x[:, k], y[:, k]), out=top)
        total = total + top
    return 16 * 7 * 2.0 ** -13 * total


def newton_schulz(u, steps, digits=None):
    """Orthogonalisation in float64, of a matrix in its own orientation, without a shape scale.
    With ``digits`` every iterate, A and B is rounded to so many binary digits relative to
    its own largest entry's power of two or, for smaller entries, their own (the pairs of
    float16), so that the deviation from the exact iteration shows what they cost."""
    def held(m):
        if digits is None:
            return m
        step = 2.0 ** (np.ceil(np.log2(np.maximum(np.abs(m), 1e-30))) - digits)
        return np.round(m / step) * step

    u = np.asarray(u, np.float64)
    x = u / (np.linalg.norm(u) + 1e-7)
    tall = x.shape[0] > x.shape[1]
    x = held(x.T if tall else x)
    for a, b, c in steps:
        a, b, c = (float(np.float32(v)) for v in (a, b, c))
        g = held(x @ x.T)
        p = held(b * g + c * (g @ g))
        x = held(a * x + p @ x)
    return x.T if tall else x
