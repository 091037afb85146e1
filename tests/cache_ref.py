"""Plain 64-bit forms of the attention cache's operators for their tests (numpy, from the definitions)."""
from __future__ import annotations

import numpy as np

MAGS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
U_BF16 = 2.0**-8    # half a step of bf16, relative
U_F32 = 2.0**-24


def exponent(amax: np.ndarray) -> np.ndarray:
    """The scale byte of blocks with these largest magnitudes."""
    amax = np.asarray(amax, np.float64)
    bad = ~np.isfinite(amax)
    _, p = np.frexp(np.where(bad, 1.0, amax))
    e = np.maximum(np.where(amax == 0, 0, p - 3 + 127), 0)
    return np.where(bad, 255, e).astype(np.uint8)


def nearest(a: np.ndarray) -> np.ndarray:
    """Index of the magnitude nearest to a >= 0, ties to the even index."""
    a = np.asarray(a, np.float64)
    code = np.zeros(a.shape, np.uint8)
    for i in range(7):
        mid = (MAGS[i] + MAGS[i + 1]) / 2
        code += (a >= mid) if i % 2 == 1 else (a > mid)
    return code


def encode(x: np.ndarray):
    """Rows [..., d] -> (codes [..., d/2], scales [..., d/32]), both uint8."""
    x = np.asarray(x, np.float64)
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    with np.errstate(invalid="ignore"):
        amax = np.where(np.isfinite(b).all(-1), np.abs(b).max(-1, initial=0.0), np.nan)
    e = exponent(amax)
    bad = e == 255
    unit = np.ldexp(1.0, np.where(bad, 127, e).astype(int) - 127)
    with np.errstate(invalid="ignore"):
        c = nearest(np.where(bad[..., None], 0.0, np.abs(b) / unit[..., None]))
    c = np.where(bad[..., None], 0, c | (np.signbit(b).astype(np.uint8) << 3)).astype(np.uint8)
    c = c.reshape(*x.shape[:-1], x.shape[-1] // 2, 2)
    return c[..., 0] | (c[..., 1] << 4), e


def decode(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """Values in 64 bits; NaN for blocks with scale byte 255."""
    n = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    v = np.where(n & 8, -1.0, 1.0) * MAGS[n & 7]
    e = np.repeat(scales, 32, -1).astype(int)
    return np.where(e == 255, np.nan, v * np.ldexp(1.0, np.where(e == 255, 127, e) - 127)) + 0.0


def norm(x: np.ndarray, w: np.ndarray | None, eps: float) -> np.ndarray:
    x = np.asarray(x, np.float64)
    if w is None:
        return x
    with np.errstate(divide="ignore", invalid="ignore"):
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + np.float64(np.float32(eps))) * np.asarray(w, np.float64)
    return np.where((x == 0).all(-1, keepdims=True), 0.0, y)


def rotate(x: np.ndarray, cos: np.ndarray, sin: np.ndarray, interleaved: bool):
    """x [tokens, heads, d], cos and sin [tokens, rot / 2] -> (rotated, |a| + |b| of each channel's pair)."""
    half = cos.shape[1]
    y, size = np.array(x, np.float64), np.abs(x)
    first = np.arange(0, 2 * half, 2) if interleaved else np.arange(half)
    second = first + 1 if interleaved else first + half
    a, b = x[..., first], x[..., second]
    c, s = cos[:, None].astype(np.float64), sin[:, None].astype(np.float64)
    y[..., first] = a * c - b * s
    y[..., second] = b * c + a * s
    size[..., first] = size[..., second] = np.abs(a) + np.abs(b)
    return y, size


def attention(q, keys, values, scale: float, causal: bool, window: int, sinks=None):
    """One sequence: q [n, heads, d], keys and values [l, kv, d] in 64 bits -> (out, bound of what rounding may add).

    The bound counts: the weights' rounding to bf16 (half a step u of each, relative, in the product and in the sum: with
    weights p (1 + e) the result moves by sum p e (v - out) / sum p (1 + e), at most u (sum p |v| / sum p + |out|) /
    (1 - u)), the result's own, and the scores' errors, which enter the weights and the sum (twice). A score's: a query times
    the scale is taken as sums of parts that leave at most 2^-13 of its block's largest magnitude (or 2^-130), products add in
    fp32 (d terms and the accumulator's roundings), with the maximum taken off, and the exponential itself (2 steps).
    A weight below the smallest normal number counts as zero. The maximum in use is never above the row's, so the
    largest weight, and the sum with it, is at least 1, and what is lost of the result is at most 2^-126 |v| a token."""
    n, heads, d = q.shape
    length, kv = keys.shape[:2]
    out = np.zeros((n, heads, d))
    bound = np.zeros((n, heads, d))
    pos = np.arange(length - n, length)[:, None]
    j = np.arange(length)[None, :]
    seen = np.ones((n, length), bool)
    if causal:
        seen = j <= pos
        if window:
            seen &= j > pos - window
    for h in range(heads):
        k, v = keys[:, h // (heads // kv)], values[:, h // (heads // kv)]
        bad_k, bad_v = np.isnan(k).any(-1), np.isnan(v)
        k, v = np.where(bad_k[:, None], 0.0, k), np.where(bad_v, 0.0, v)
        x = np.asarray(q[:, h], np.float64)
        s = scale * (x @ k.T)
        size = scale * (np.abs(x) @ np.abs(k).T)
        blocks = np.maximum(2.0**-13 * scale * np.abs(x).reshape(n, d // 32, 32).max(-1), 2.0**-130)
        parts = (blocks @ np.abs(k).reshape(length, d // 32, 32).sum(-1).T)
        delta = np.where(seen, parts + (d + 8) * U_F32 * size + 4 * U_F32 * np.abs(s), 0.0).max(1, initial=0.0)
        delta = np.expm1(2 * delta + 8 * U_F32)
        s = np.where(seen, s, -np.inf)
        top = s.max(1, initial=-np.inf)
        if sinks is not None:
            top = np.maximum(top, float(sinks[h]))
        top = np.where(np.isfinite(top), top, 0.0)
        p = np.exp(s - top[:, None])
        total = p.sum(1) + (0.0 if sinks is None else np.exp(float(sinks[h]) - top))
        total = np.where(total > 0, total, 1.0)
        o = (p @ v) / total[:, None]
        mag = (p @ np.abs(v)) / total[:, None]
        # sums of `length` terms in fp32, in any order
        bound[:, h] = (mag + np.abs(o)) * U_BF16 * (1 + delta[:, None]) / (1 - U_BF16)
        bound[:, h] += mag * (2 * delta[:, None] + 2 * (length + 8) * U_F32)
        bound[:, h] += 2.0**-126 * (seen.astype(np.float64) @ np.abs(v))
        bound[:, h] += U_BF16 * (np.abs(o) + bound[:, h]) + 2.0**-134
        o[(seen & bad_k[None, :]).any(1)] = np.nan
        o[(seen.astype(np.float64) @ bad_v.astype(np.float64)) > 0] = np.nan
        out[:, h] = o
    return out, bound
