"""The residual's addition and the root-mean-square norm (oracle, fp64).

    r = x + delta,  y = r w / sqrt(mean r^2 + eps)

and, for an 8-bit output, per group of channels s = max|y| / 448 (448: the
largest e4m3 value) with codes y / s rounded to the nearest e4m3 value.
"""
from __future__ import annotations

import numpy as np

from .kv import e4m3_round


def add_norm(x, delta=None, weight=None, eps=1e-6):
    """x, delta [rows, hidden], weight [hidden], float64.  Returns r and y."""
    r = np.asarray(x, dtype=np.float64)
    if delta is not None:
        r = r + np.asarray(delta, dtype=np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        y = r / np.sqrt((r * r).mean(axis=1, keepdims=True) + eps)
        return r, y if weight is None else y * np.asarray(weight, dtype=np.float64)


def groups(hidden: int, group: int):
    """Slices of the channels that share a scale."""
    wide = group or hidden
    return [slice(i, min(hidden, i + wide)) for i in range(0, hidden, wide)]


def quantise(y, group=0):
    """Codes' values [rows, hidden] and scales [rows, groups] of finite y."""
    codes, scales = np.zeros_like(y), []
    for g in groups(y.shape[1], group):
        s = np.abs(y[:, g]).max(axis=1, keepdims=True) / 448.0
        codes[:, g] = e4m3_round(np.divide(y[:, g], s, out=np.zeros_like(y[:, g]), where=s > 0))
        scales.append(s)
    return codes, np.concatenate(scales, axis=1)
