"""The 8-bit key/value cache and attention over it (TEST INFRASTRUCTURE).

The cache of one sequence, head by head, as codes and one scale per page:
value = scale * code. Writing follows the cache's fp32 contract (each operation
rounded to binary32 by numpy's float32 arithmetic); attention is float64.
"""
from __future__ import annotations

import math

import numpy as np

F = np.float32


def write(codes: np.ndarray, scales: np.ndarray, x: np.ndarray, start: int, page: int) -> None:
    """Adds tokens x (n, dim) float32 behind `start` held ones of one head.
    codes (tokens, dim) int, scales (pages) float32, both updated in place."""
    end = start + len(x)
    for p in range(start // page, -(-end // page)):
        lo, hi = max(start, p * page), min(end, (p + 1) * page)
        new = x[lo - start:hi - start].astype(F)
        scale = F(np.max(np.abs(new))) / F(127)
        if lo > p * page:
            old = scales[p]
            scale = max(old, scale)
            if scale > old:
                held = codes[p * page:lo].astype(F) * old
                codes[p * page:lo] = np.rint(held / scale).astype(np.int64)
        codes[lo:hi] = np.clip(np.rint(new / scale), -127, 127).astype(np.int64) if scale > 0 else 0
        scales[p] = scale


def values(codes: np.ndarray, scales: np.ndarray, page: int) -> np.ndarray:
    """float64 values of codes (tokens, dim)."""
    return codes.astype(np.float64) * np.repeat(scales.astype(np.float64), page)[:len(codes), None]


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, places, scale: float, softcap: float = 0.0, window: int = 0):
    """One head: q (rows, dim) at `places`, k and v (tokens, dim), float64.
    Returns (out, lse, weight of |v|): the last is sum_j p_j |v_j|, for the
    tolerances."""
    s = q @ k.T * scale
    if softcap:
        s = softcap * np.tanh(s / softcap)
    j = np.arange(len(k))
    at = np.asarray(places)[:, None]
    seen = (j <= at) & ((j > at - window) if window else True)
    out, mass = np.zeros((len(q), v.shape[1])), np.zeros((len(q), v.shape[1]))
    lse = np.full(len(q), -math.inf)
    for r in range(len(q)):
        if seen[r].any():
            x = s[r][seen[r]]
            top = x.max()
            e = np.exp(x - top)
            p = e / e.sum()
            out[r], mass[r] = p @ v[seen[r]], p @ np.abs(v[seen[r]])
            lse[r] = top + math.log(e.sum())
    return out, lse, mass


def score_error(q: np.ndarray, k: np.ndarray, scale: float, softcap: float) -> np.ndarray:
    """Bound per row on the error of any score computed in fp32 from exact q
    and k: the products' sum (a tensor core may cut each of its dim / 16 + 16
    steps by 2 u of the magnitudes), the three scalings 3 u, and for the cap
    4 u of its range. u = 2^-24. A query's values below 2^-25 of its largest are
    lost: 2^-25 dim |k|max |q|max."""
    u, dim = 2.0 ** -24, q.shape[1]
    big = np.max(np.abs(q) @ np.abs(k).T, axis=1) if len(k) else np.zeros(len(q))
    lost = 2.0 ** -25 * dim * np.max(np.abs(q), axis=1) * (np.max(np.abs(k)) if len(k) else 0.0)
    return abs(scale) * (big * (2 * (dim / 16 + 16) + 6) * u + lost) + (8 * u * softcap)


def out_error(out: np.ndarray, mass: np.ndarray, v: np.ndarray, delta: np.ndarray, tokens: int) -> np.ndarray:
    """Bound on the bf16 output's error: its own rounding 2^-8 |o|; each
    probability off by e^delta twice (itself and the sum), its exponential
    2^-21, its fp16 rounding 2^-11; the running sums (2 u a step of 16 tokens
    and of every rescaling, at most one a step); probabilities below 2^-29 of the
    largest lose 2^-39 of it absolutely, a token each."""
    u = 2.0 ** -24
    rel = 2 * np.expm1(delta)[:, None] + 2.0 ** -20 + 2.0 ** -11 + 8 * u * (tokens / 16 + 8)
    under = tokens * 2.0 ** -39 * (np.max(np.abs(v)) if len(v) else 0.0)
    return (2.0 ** -8 * np.abs(out) + rel * mass + under) * (1 + 2.0 ** -8)


def lse_error(lse: np.ndarray, delta: np.ndarray, tokens: int) -> np.ndarray:
    """Bound on the fp32 lse's error: the scores', exponentials' 2^-21, sums of
    `tokens` terms (2 u a step of 8), and 6 u of its size."""
    u = 2.0 ** -24
    size = np.where(np.isfinite(lse), np.abs(lse), 0.0)
    return delta + 2.0 ** -20 + 2 * u * (tokens / 8 + 16) + 6 * u * (size + 32)
