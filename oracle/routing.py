"""Router top-k and gate weights (oracle).

The pages state only that the model has 256 routed experts and that the
router selects eight per token ("FreeToken vs vLLM on one RTX 3090", section
"Why the performance differs", FreeToken exploits MoE sparsity).  Readings
taken where they are silent:

* Selection is by logit, descending; equal logits are ordered by the lower
  expert index first.  -0.0 and +0.0 compare equal (float comparison).  NaN
  logits are ordered as -inf.  The output order of the k picks is this order.
* Gates are the softmax restricted to the k selected logits,
  w_j = exp(l_j - m) / sum_{i in top-k} exp(l_i - m), m = the largest selected
  logit.  This equals "softmax over all experts, then renormalise the selected
  k", the convention of the Qwen3-MoE family whose shape the decode workload
  uses.
"""
from __future__ import annotations

import dataclasses

import numpy as np


def selection_order(logits: np.ndarray) -> np.ndarray:
    """Per row, all expert indices sorted by (logit descending, index ascending)."""
    x = np.asarray(logits, dtype=np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    x = x + 0.0                                     # -0.0 -> +0.0
    idx = np.broadcast_to(np.arange(x.shape[-1]), x.shape)
    # lexsort: last key is primary -> primary -logit, secondary index
    return np.lexsort((idx, -x), axis=-1)


def topk(logits: np.ndarray, k: int) -> np.ndarray:
    """Top-k expert indices per token, int32 [T, k], in selection order."""
    return selection_order(logits)[..., :k].astype(np.int32)


def gates(logits: np.ndarray, topk_idx: np.ndarray) -> np.ndarray:
    """Gate weights float64 [T, k]: softmax over the selected logits only."""
    x = np.asarray(logits, dtype=np.float64)
    sel = np.take_along_axis(x, np.asarray(topk_idx, dtype=np.int64), axis=-1)
    m = sel.max(axis=-1, keepdims=True)
    p = np.exp(sel - m)
    return p / p.sum(axis=-1, keepdims=True)


def route(logits: np.ndarray, k: int):
    """(topk_idx int32 [T,k], gates float64 [T,k]) for router logits [T,E]."""
    idx = topk(logits, k)
    return idx, gates(logits, idx)


@dataclasses.dataclass
class Rule:
    """A routing rule: scores s = softmax or sigmoid of the logits, the choice by v = s + bias (with groups: among the
    top_groups groups of consecutive experts whose best v, or sum of the best two, is largest), gates s of the picks,
    renormalised over them or not, times scale.  Without a bias v has the logits' order.  Values that fp64 cannot tell
    apart have the order of their logits (that of exact arithmetic where the biases are equal), equal ones go to the lower
    index; a NaN logit or v is -inf, an infinite one the largest fp32 number; without any score the gates are 0."""
    score: str = "softmax"
    bias: np.ndarray | None = None
    groups: int = 1
    top_groups: int = 1
    group_top: int = 1
    renormalise: bool = True
    scale: float = 1.0


def clean(x):
    x = np.asarray(x, dtype=np.float64)
    return np.minimum(np.where(np.isnan(x), -np.inf, x), float(np.finfo(np.float32).max)) + 0.0


def route_by(rule: Rule, logits: np.ndarray, k: int):
    """(topk_idx int32 [T, k], gates float64 [T, k]) by a rule."""
    x = clean(logits)
    T, E = x.shape
    with np.errstate(over="ignore"):
        if rule.score == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-x))
        else:
            e = np.exp(x - np.maximum(x.max(axis=1, keepdims=True), -1e300))
            s = np.divide(e, e.sum(axis=1, keepdims=True), out=np.zeros_like(e), where=e.sum(axis=1, keepdims=True) > 0)
    v = x if rule.bias is None else clean(s + np.asarray(rule.bias, dtype=np.float64))
    tie = np.where(v > -np.inf, x, 0.0)
    if rule.groups > 1 and rule.top_groups < rule.groups:
        of = (v if rule.bias is not None or rule.group_top == 1 else s).reshape(T, rule.groups, -1)
        best = np.sort(of, axis=2)[:, :, ::-1][:, :, :rule.group_top].sum(axis=2)
        by = np.zeros_like(best)  # a group's best expert's logit
        if rule.group_top == 1:
            by = np.where(of == best[:, :, None], tie.reshape(of.shape), -np.inf).max(axis=2)
        take = np.array([np.lexsort((np.arange(rule.groups), -by[t], -best[t])) for t in range(T)]).reshape(T, rule.groups)[:, :rule.top_groups]
        part = np.zeros((T, rule.groups), dtype=bool)
        np.put_along_axis(part, take, True, axis=1)
        part = np.repeat(part, E // rule.groups, axis=1)
    else:
        part = np.ones((T, E), dtype=bool)
    idx = np.empty((T, k), dtype=np.int32)
    for t in range(T):  # those that take part, by (v descending, logit descending, index ascending)
        at = np.flatnonzero(part[t])
        idx[t] = at[np.lexsort((at, -tie[t, at], -v[t, at]))[:k]]
    w = np.take_along_axis(s, idx.astype(np.int64), axis=1)
    if rule.renormalise:
        l = np.take_along_axis(x, idx.astype(np.int64), axis=1)
        if rule.score == "softmax":  # the row's denominator cancels, and so may its underflow
            w = np.exp(l - np.maximum(l.max(axis=1, keepdims=True), -1e300))
        total = w.sum(axis=1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    return idx, w * rule.scale
