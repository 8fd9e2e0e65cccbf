"""fp64 oracle of 4-bit rows: 32 values share a factor of five significant
bits, each value is a whole number from -7 to 7 times its factor.

TEST INFRASTRUCTURE ONLY (like the rest of ``oracle/``); it shares no code with
the CUDA path.  Exact rational arithmetic (``fractions``) decides every tie.
"""

from __future__ import annotations

from fractions import Fraction

import numpy as np

from . import _f64

GROUP = 32


def nearest_even(x: Fraction) -> int:
    """The nearest whole number, ties to the even one."""
    return round(x)  # Python's rule for fractions


def factor(values) -> float:
    """The factor of one group of bf16 values: amax / 7 in five significant
    bits, at least 2^-120; 1 for zeros; NaN with a NaN among them."""
    values = [float(v) for v in values]
    if any(np.isnan(v) for v in values):
        return float("nan")
    amax = max([abs(v) for v in values if np.isfinite(v)] + [0.0])
    if amax == 0:
        return 1.0
    q = Fraction(amax) / 7
    e = 0
    while q >= Fraction(2) ** (e + 1):
        e += 1
    while q < Fraction(2) ** e:
        e -= 1
    step = Fraction(2) ** (e - 4)
    return float(max(nearest_even(q / step) * step, Fraction(2) ** -120))


def quantise(x):
    """(codes int [..., d] from -7 to 7, factors [..., d / 32]) of rows x; the
    codes of a group with a NaN say nothing (0 here)."""
    x = _f64(x)
    g = x.reshape(-1, GROUP)
    f = np.array([factor(row) for row in g])
    c = np.zeros(g.shape, dtype=np.int64)
    for i, row in enumerate(g):
        if np.isnan(f[i]):
            continue
        F = Fraction(f[i])
        for j, v in enumerate(row):
            c[i, j] = 7 * int(np.sign(v)) if np.isinf(v) \
                else max(-7, min(7, nearest_even(Fraction(float(v)) / F)))
    return c.reshape(x.shape), f.reshape(x.shape[:-1] + (-1,))


def pack(codes) -> np.ndarray:
    """Bytes [..., d / 2]: element 2i in the low half of byte i."""
    u = (np.asarray(codes) + 8).astype(np.uint8)
    return u[..., 0::2] | (u[..., 1::2] << 4)


def unpack(b) -> np.ndarray:
    if hasattr(b, "detach"):
        b = b.detach().cpu().numpy()
    b = np.asarray(b, dtype=np.uint8)
    out = np.empty(b.shape[:-1] + (2 * b.shape[-1],), dtype=np.int64)
    out[..., 0::2], out[..., 1::2] = (b & 15).astype(np.int64) - 8, (b >> 4).astype(np.int64) - 8
    return out


def values(b, factors) -> np.ndarray:
    """What packed bytes and their factors stand for, float64 [..., d]."""
    return unpack(b) * np.repeat(_f64(factors), GROUP, axis=-1)
