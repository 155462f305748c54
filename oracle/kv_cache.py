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


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, v_scales, places, scale: float, softcap: float = 0.0,
           window: int = 0):
    """One head: q (rows, dim) at `places`, k and v (tokens, dim), float64.
    Returns (out, lse, sum_j p_j |v_j|, sum_j p_j 383 s_j): the last two, with s
    the tokens' V scales, for the tolerances."""
    s = q @ k.T * scale
    if softcap:
        s = softcap * np.tanh(s / softcap)
    j = np.arange(len(k))
    at = np.asarray(places)[:, None]
    seen = (j <= at) & ((j > at - window) if window else True)
    out, mass = np.zeros((len(q), v.shape[1])), np.zeros((len(q), v.shape[1]))
    lse, gross = np.full(len(q), -math.inf), np.zeros(len(q))
    for r in range(len(q)):
        if seen[r].any():
            x = s[r][seen[r]]
            top = x.max()
            e = np.exp(x - top)
            p = e / e.sum()
            out[r], mass[r] = p @ v[seen[r]], p @ np.abs(v[seen[r]])
            lse[r] = top + math.log(e.sum())
            gross[r] = 383 * (p @ v_scales[seen[r]])
    return out, lse, mass, gross


def score_error(q: np.ndarray, unit: float, scale: float, softcap: float) -> np.ndarray:
    """Bound per row on the error of any score computed in fp32 from exact q and
    codes of a scale of at most `unit`. The sums run over q (code + 128), from
    -128 sum(q): no partial sum exceeds 255 unit |q|_1, and each of the dim / 16
    + 16 steps (a tensor core may cut a step by 2 u of that) and of the dim / 4 + 4
    additions of sum(q) costs of it; the scalings 6 u. For the cap 4 u of its range,
    twice, or, of scores below a sixteenth of it where it is wide (above 64), 8 u of
    themselves, so never more than 8 u 16 |score|. u = 2^-24. A query's values below
    2^-25 of its largest are lost: 2^-25 dim 127 unit |q|max."""
    u, dim = 2.0 ** -24, q.shape[1]
    big = 255 * unit * np.sum(np.abs(q), axis=1)
    lost = 2.0 ** -25 * dim * np.max(np.abs(q), axis=1) * 127 * unit
    cap = np.minimum(softcap, 16 * abs(scale) * big) if softcap > 64 else softcap
    return abs(scale) * (big * (2 * (dim / 16 + 16) + dim / 4 + 4 + 6) * u + lost) + 8 * u * cap


def out_error(out: np.ndarray, mass: np.ndarray, gross: np.ndarray, unit: float, delta: np.ndarray, tokens: int) -> np.ndarray:
    """Bound on the bf16 output's error: its own rounding 2^-8 |o|; each
    probability off by e^delta twice (itself and the sum), its exponential
    2^-21, its fp16 rounding 2^-11: of `mass`, the sum of p |v|. The running sums
    take 128 times a step's probabilities away and add the bytes, code + 128: 8 u a
    step of 16 tokens and of the joining, of `gross`, the sum of p (255 + 128) s with s
    the scale of the value's page, which no partial sum exceeds. Probabilities below 2^-22 of the running maximum,
    which is at most the largest or the integer (base 2) above it, are fp16 subnormals:
    half a step there is 2^-25 of the factor 2^-8 they stand high, 2^-33 of twice the
    largest, a token each, times its code and twice `unit`, the largest scale of V (their
    ratio is taken to it, or to the power of two above it)."""
    u = 2.0 ** -24
    rel = 2 * np.expm1(delta)[:, None] + 2.0 ** -20 + 2.0 ** -11
    under = tokens * 2.0 ** -33 * 127 * 4 * unit
    return (2.0 ** -8 * np.abs(out) + rel * mass + 8 * u * (tokens / 16 + 32) * gross[:, None] + under) * (1 + 2.0 ** -8)


def lse_error(lse: np.ndarray, delta: np.ndarray, tokens: int) -> np.ndarray:
    """Bound on the fp32 lse's error: the scores', exponentials' 2^-21, sums of
    `tokens` terms (2 u a step of 8), and 6 u of its size."""
    u = 2.0 ** -24
    size = np.where(np.isfinite(lse), np.abs(lse), 0.0)
    return delta + 2.0 ** -20 + 2 * u * (tokens / 8 + 16) + 6 * u * (size + 32)
