"""The paged key/value cache and attention over it (oracle, fp64).

A sequence with n tokens, the last m of them new, attends from each new token
at position p = n - m + i to the tokens j in [0, n) with j <= p (causal) and
j > p - window (window > 0):

    out = sum_j softmax_j(scale q.k_j) v_j,    lse = log sum_j exp(scale q.k_j);

a row at a negative position sees nothing; a row that sees nothing, or only
scores of -inf, gives zeros and lse -inf.

The quantised cache holds, per token and head, e4m3 codes of x / 2^k with the
smallest k >= -110 such that max|x| <= 448 * 2^k (448: the largest e4m3
value), rounded to nearest even and, at k = 120, held to 240 so that the value
is a finite bf16 one; the byte k + 127 goes with it.  A vector that is not
finite throughout is stored as byte 255 (NaN) and codes 0.
"""
from __future__ import annotations

import math

import numpy as np


def scale_exponent(amax: float) -> int:
    """Smallest k >= -110 with amax <= 448 * 2^k."""
    if amax == 0.0:
        return -110
    k = math.frexp(amax)[1] - 12  # 448 * 2^k is below amax here
    while amax > 448.0 * 2.0 ** k:
        k += 1
    return max(k, -110)


def e4m3_round(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 values (ties to even) of |x| <= 448: 4 significant bits,
    steps of 2^-9 below 2^-6."""
    _, e = np.frexp(np.maximum(np.abs(x), 2.0 ** -6))
    step = np.ldexp(1.0, e - 4)
    return np.rint(x / step) * step


def quantise(x: np.ndarray):
    """x [..., D] float64 -> (codes' values [..., D], exponent bytes [...])."""
    x = np.asarray(x, dtype=np.float64)
    codes = np.zeros_like(x)
    e = np.full(x.shape[:-1], 255, dtype=np.uint8)
    for i in np.ndindex(*x.shape[:-1]):
        if not np.isfinite(x[i]).all():
            continue
        k = scale_exponent(float(np.abs(x[i]).max()))
        lim = 240.0 if k == 120 else 448.0
        codes[i] = e4m3_round(np.clip(x[i] / 2.0 ** k, -lim, lim))
        e[i] = k + 127
    return codes, e


def dequantise(codes: np.ndarray, e: np.ndarray) -> np.ndarray:
    s = np.where(e == 255, np.nan, np.exp2(e.astype(np.float64) - 127.0))
    return np.asarray(codes, dtype=np.float64) * s[..., None]


def visible(n: int, m: int, causal: bool, window: int) -> np.ndarray:
    """[m, n] mask of what each new token sees."""
    p = np.arange(n - m, n)[:, None]
    j = np.arange(n)[None, :]
    see = np.broadcast_to(p >= 0, (m, n)).copy()  # a negative position (m > n) sees nothing, causal or not
    if causal:
        see &= j <= p
        if window:
            see &= j > p - window
    return see


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, causal: bool = True, window: int = 0):
    """One sequence: q [m, Hq, D], k and v [n, H, D] float64.  Returns out
    [m, Hq, D], lse [m, Hq] and, for error bounds, the softmax-weighted |v|
    [m, Hq, D] and the largest sum_d |q_d k_jd| * scale of each row [m, Hq]."""
    m, Hq, D = q.shape
    n, H = k.shape[0], k.shape[1]
    out, bulk = np.zeros((m, Hq, D)), np.zeros((m, Hq, D))
    lse, reach = np.full((m, Hq), -np.inf), np.zeros((m, Hq))
    see = visible(n, m, causal, window)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        for h in range(Hq):
            kh, vh = k[:, h // (Hq // H)], v[:, h // (Hq // H)]
            for i in range(m):
                at = np.flatnonzero(see[i])
                if not at.size:
                    continue
                s = (kh[at] @ q[i, h]) * scale
                top = s.max()
                if top == -np.inf:
                    continue
                w = np.exp(s - top)
                out[i, h] = (w @ vh[at]) / w.sum()
                bulk[i, h] = (w @ np.abs(vh[at])) / w.sum()
                lse[i, h] = top + np.log(w.sum())
                reach[i, h] = (np.abs(kh[at]) @ np.abs(q[i, h])).max() * abs(scale)
    return out, lse, bulk, reach
