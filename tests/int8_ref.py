"""Plain 64-bit forms of the int8 operators for their tests (numpy, from the definitions)."""
from __future__ import annotations

from fractions import Fraction

import numpy as np


def codes(p: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """Codes and row maxima of rows p: nearest integer to 127 p / max|p|, ties to even."""
    p = np.asarray(p, np.float64)
    top = np.abs(p).max(axis=1, initial=0.0)
    bad = ~np.isfinite(p).all(axis=1)
    safe = np.where(bad | (top == 0), 1.0, top)
    with np.errstate(invalid="ignore", over="ignore"):
        q = np.rint(np.where(bad[:, None], 0.0, p) * 127.0 / safe[:, None])
    q[top == 0] = 0
    return q.astype(np.int8), np.where(bad, np.nan, top)


def code_fraction(p: float, top: float) -> int:
    """The same for one element in exact arithmetic."""
    f = Fraction(127) * Fraction(p) / Fraction(top)
    lo = f.numerator // f.denominator
    rest = f - lo
    if rest * 2 == 1:
        return lo if lo % 2 == 0 else lo + 1
    return lo + (rest * 2 > 1)


def quantize(x: np.ndarray):
    q, top = codes(x)
    return q, top / 127.0


def rmsnorm(x: np.ndarray, w: np.ndarray, eps: float, residual: np.ndarray | None = None):
    """x, w, residual fp32 arrays (the values of their type): (codes, scale, h fp32)."""
    with np.errstate(over="ignore", invalid="ignore"):
        h = x.astype(np.float32) if residual is None else (x + residual).astype(np.float32)
        q, top = codes((h * w).astype(np.float32))
        mean = (h.astype(np.float64) ** 2).mean(axis=1)
        with np.errstate(divide="ignore"):
            scale = top / (127.0 * np.sqrt(mean + np.float64(np.float32(eps))))
    scale = np.where(top == 0, 0.0, scale)
    return q, scale, h


def silu_mul(gate_up: np.ndarray):
    g, u = np.split(np.asarray(gate_up, np.float64), 2, axis=1)
    with np.errstate(over="ignore", invalid="ignore"):
        p = g / (1.0 + np.exp(-g)) * u
    q, top = codes(p)
    return q, top / 127.0


def gemm(x: np.ndarray, xs: np.ndarray, w: np.ndarray, ws: np.ndarray, bias: np.ndarray | None = None):
    """(y, the magnitude of the product part, in 64 bits): the sums of int8 products are exact in float64."""
    acc = x.astype(np.float64) @ w.astype(np.float64).T
    y = acc * xs.astype(np.float64)[:, None] * ws.astype(np.float64)[None, :]
    return (y if bias is None else y + bias.astype(np.float64)), np.abs(y)
