"""Oracle: a router's choice by values, and its bias's balancing step -- TEST INFRASTRUCTURE ONLY.

Values v = score + bias (fp64); groups of consecutive experts ranked by their best or the sum of their two
best; the k largest values of the open groups in descending order, the lower index among equals.  Gates,
counts and losses as in oracle.router, with this choice."""
from __future__ import annotations

import numpy as np

from oracle.router import _live, _log_sum_exp, _scores


def choose(row, k, sigmoid, bias=None, groups=1, top_groups=1, two=True):
    """Experts of one row of logits that is routed."""
    E = len(row)
    with np.errstate(over="ignore"):
        v = 1 / (1 + np.exp(-row)) if sigmoid else np.exp(row - row.max()) / np.exp(row - row.max()).sum()
    can = row > -np.inf
    if bias is not None:
        can = can & (bias > -np.inf)
        v = v + bias
    worth = []
    size = E // groups
    for g in range(groups):
        members = sorted((v[e] for e in range(g * size, (g + 1) * size) if can[e]), reverse=True)
        worth.append(-np.inf if not members else sum(members[:2]) if two else members[0])
    open_ = sorted(range(groups), key=lambda g: (-worth[g], g))[:top_groups]
    left = [e for e in range(E) if can[e] and e // size in open_]
    return sorted(left, key=lambda e: (-v[e], e))[:k]


def forward(logits, k, sigmoid=False, renorm=True, scale=1.0, mask=None, **choice):
    l = np.asarray(logits, dtype=np.float64)
    T, E = l.shape
    ids, gates = np.full((T, k), -1, dtype=np.int32), np.zeros((T, k))
    counts, prob = np.zeros(E, dtype=np.int64), np.zeros(E)
    n, z, bad = 0, 0.0, False
    for t in range(T):
        on = mask is None or mask[t]
        if not _live(l[t], on):
            bad |= bool(on) and bool(np.isnan(l[t]).any() or np.isposinf(l[t]).any())
            continue
        n += 1
        s = _scores(l[t], sigmoid)
        P = np.exp(s - _log_sum_exp(s))
        order = choose(l[t], k, sigmoid, **choice)
        if order:
            c = s[order]
            if renorm:                        # by the largest: c - log(sum) loses the sum next to 1e38
                e = np.exp(c - c.max())
                g = e / e.sum()
            else:
                g = np.exp(c) if sigmoid else P[order]
            ids[t, :len(order)] = order
            gates[t, :len(order)] = scale * g
            counts[order] += 1
        prob += P
        z += _log_sum_exp(l[t]) ** 2
    balance = E / k * float(counts @ prob) / n / n if n else 0.0
    return {"topk_ids": ids, "gates": gates, "counts": counts, "prob_sum": prob, "live": n,
            "losses": np.array([balance, z / n if n else 0.0]), "bad": bad}


def bias_update(bias, counts, rate):
    """fp32, as stored."""
    c = np.asarray(counts, dtype=np.int64)
    return (bias + np.float32(rate) * np.sign(c.sum() - c * len(c)).astype(np.float32)).astype(np.float32)
