"""Rotary positions in float64 (TEST INFRASTRUCTURE).

A pair (a, b) at position p turns by t = p w_i:
    factor (a cos t - b sin t, b cos t + a sin t),   w_i = theta^(-2 i / rot),
with the frequencies optionally scaled for long contexts: by one factor, by
bands of wavelengths, or by the ramp over the pair index of arXiv 2309.00071.
"""
from __future__ import annotations

import math

import numpy as np


def frequencies(theta: float, rot: int, scaling: str = "plain", params=()) -> tuple:
    """(w_i in radians per position, factor)."""
    w = np.array([theta ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "plain":
        return w, 1.0
    if scaling == "linear":
        return w / params[0], 1.0
    if scaling == "bands":
        f, low, high, length = params
        out = []
        for x in w:
            turns = length * x / (2 * math.pi)
            if turns <= low:
                out.append(x / f)
            elif turns >= high:
                out.append(x)
            else:
                k = (turns - low) / (high - low)
                out.append((1 - k) * x / f + k * x)
        return np.array(out), 1.0
    f, fast, slow, length = params
    pair = lambda turns: rot * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
    low, high = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rot - 1)
    k = np.clip((np.arange(rot // 2) - low) / (high - low if high > low else 0.001), 0, 1)
    return w / f * k + w * (1 - k), (0.1 * math.log(f) + 1.0 if f > 1 else 1.0)


def rotate(x: np.ndarray, positions, w: np.ndarray, factor: float, layout: str) -> np.ndarray:
    """x (rows, heads, dim) float64, positions (rows)."""
    rot = 2 * len(w)
    t = np.asarray(positions, dtype=np.float64)[:, None] * w
    c, s = factor * np.cos(t)[:, None], factor * np.sin(t)[:, None]
    y = np.array(x, dtype=np.float64)
    ia, ib = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


U32 = 2.0 ** -24


def f32_error(x: np.ndarray, rot: int, factor: float, layout: str) -> np.ndarray:
    """Bound on |fp32 rotation - rotate(x)| per value: sine and cosine within
    3 u, their product with the factor 1 u, the two products and the sum 1 u
    each of (|a| + |b|) factor, u = 2^-24: 6 u, and one more for the second
    order. Values behind the rotated part are copies."""
    e = np.zeros(x.shape)
    ia, ib = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    e[..., ia] = e[..., ib] = 7 * U32 * abs(factor) * (np.abs(x[..., ia]) + np.abs(x[..., ib]))
    return e
