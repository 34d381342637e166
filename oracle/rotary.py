"""Rotary positions (oracle, fp64).

Pair i of a head's first d values, (i, i + d/2) or (2i, 2i + 1), is the complex
number a + ib times scale * e^(i position f_i); the rest stays.  Frequencies:
f_i = base^(-2i/d), for longer contexts divided by a factor throughout (linear)
or, "yarn" (Peng et al., "YaRN: Efficient Context Window Extension of Large
Language Models", 2023), only for pairs that turn seldom over the length of the
first training, with a linear transition over the pairs' index.
"""
from __future__ import annotations

import numpy as np


def rotate(x, positions, freq, interleaved=False, scale=1.0):
    """x [tokens, heads, dim] float64, positions [tokens], freq [d / 2]."""
    x = np.array(x, dtype=np.float64)
    d = 2 * len(freq)
    turn = scale * np.exp(1j * np.asarray(positions, dtype=np.float64)[:, None, None] * np.asarray(freq)[None, None, :])
    re, im = (slice(0, d, 2), slice(1, d, 2)) if interleaved else (slice(0, d // 2), slice(d // 2, d))
    with np.errstate(invalid="ignore", over="ignore"):
        z = (x[..., re] + 1j * x[..., im]) * turn
        x[..., re], x[..., im] = z.real, z.imag
    return x


def reach(x, freq, interleaved=False, scale=1.0):
    """|scale| (|a| + |b|) of each value's pair, for error bounds; 0 where nothing turns."""
    x, d, out = np.abs(np.asarray(x, dtype=np.float64)), 2 * len(freq), np.zeros(np.shape(x))
    re, im = (slice(0, d, 2), slice(1, d, 2)) if interleaved else (slice(0, d // 2), slice(d // 2, d))
    out[..., re] = out[..., im] = abs(scale) * (x[..., re] + x[..., im])
    return out


def yarn(d, base, factor, original, beta_fast=32.0, beta_slow=1.0):
    """A pair that turns n times over the original length has the index that solves original base^(-2i/d) = 2 pi n."""
    i = np.arange(d // 2, dtype=np.float64)
    f = np.power(base, -2.0 * i / d)
    where = [d / 2 * np.log(original / (2 * np.pi * n)) / np.log(base) for n in (beta_fast, beta_slow)]
    lo, hi = max(np.floor(where[0]), 0.0), min(np.ceil(where[1]), d - 1.0)
    slow = np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
    return (1.0 - slow) * f + slow * f / factor
