"""Oracle: top-k router, its balance losses and their gradient -- TEST INFRASTRUCTURE ONLY.

With s = l (softmax scores) or log sigmoid(l) (sigmoid scores) and
P_te = exp(s_te) / sum_i exp(s_ti), token t goes to its k largest logits (the
lower index among equals) with gates scale * P / (sum of P over the chosen)
(renorm), scale * P (softmax) or scale * sigmoid(l) (sigmoid);
    balance = E / (k n^2) sum_e c_e sum_t P_te,   z = 1/n sum_t lse(l_t)^2
over the n rows that are routed.  Rows that are not: padding, nothing above
-infinity, NaN or +infinity.  Everything in fp64.
"""
from __future__ import annotations

import numpy as np


def _log_sum_exp(s):
    m = s.max()
    return m + np.log(np.exp(s - m).sum())


def _scores(l, sigmoid):
    with np.errstate(over="ignore"):
        return -np.logaddexp(0.0, -l) if sigmoid else l


def _live(row, on):
    return bool(on) and not np.isnan(row).any() and not np.isposinf(row).any() and np.isfinite(row).any()


def forward(logits, k, sigmoid=False, renorm=True, scale=1.0, mask=None):
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
        order = [e for e in sorted(range(E), key=lambda e: (-l[t, e], e))[:k] if l[t, e] > -np.inf]
        chosen = s[order]
        if renorm:
            g = np.exp(chosen - _log_sum_exp(chosen))
        else:
            g = np.exp(chosen) if sigmoid else P[order]
        ids[t, :len(order)] = order
        gates[t, :len(order)] = scale * g
        counts[order] += 1
        prob += P
        z += _log_sum_exp(l[t]) ** 2
    balance = E / k * float(counts @ prob) / n / n if n else 0.0
    return {"topk_ids": ids, "gates": gates, "counts": counts, "prob_sum": prob, "live": n,
            "losses": np.array([balance, z / n if n else 0.0]), "bad": bad}


def objective(logits, ids, dlogp, counts, n, db, dz, sigmoid=False, renorm=True, mask=None):
    """The scalar whose gradient `backward` gives: sum dlogp log p + db balance + dz z, with the
    choice (ids, counts, n) held fixed."""
    l = np.asarray(logits, dtype=np.float64)
    T, E = l.shape
    k = ids.shape[1]
    total = 0.0
    for t in range(T):
        if not _live(l[t], mask is None or mask[t]):
            continue
        s = _scores(l[t], sigmoid)
        logP = s - _log_sum_exp(s)
        sel = [j for j in range(k) if 0 <= ids[t, j] < E]
        if sel:
            c = s[ids[t, sel]]
            logp = c - _log_sum_exp(s[sorted(set(ids[t, sel]))]) if renorm else \
                (c if sigmoid else logP[ids[t, sel]])
            total += float(dlogp[t, sel] @ logp)
        total += db * E / k / n / n * float(counts @ np.exp(logP))
        total += dz / n * _log_sum_exp(l[t]) ** 2
    return total


def backward(logits, ids, dlogp, counts, n, db, dz, sigmoid=False, renorm=True, mask=None):
    l = np.asarray(logits, dtype=np.float64)
    T, E = l.shape
    k = ids.shape[1]
    out = np.zeros((T, E))
    g = db * E / k / max(n, 1) / max(n, 1) * np.asarray(counts, dtype=np.float64)
    for t in range(T):
        if not _live(l[t], mask is None or mask[t]):
            continue
        s = _scores(l[t], sigmoid)
        P = np.exp(s - _log_sum_exp(s))
        h = np.zeros(E)
        for j in range(k):
            if 0 <= ids[t, j] < E:
                h[ids[t, j]] += dlogp[t, j]
        if renorm:
            q = np.zeros(E)
            sel = sorted({int(e) for e in ids[t] if 0 <= e < E})
            if sel:
                q[sel] = np.exp(s[sel] - _log_sum_exp(s[sel]))
        else:
            q = np.zeros(E) if sigmoid else P
        ds = h - h.sum() * q + P * (g - float(P @ g))
        lse = _log_sum_exp(l[t])
        with np.errstate(over="ignore"):
            slope = np.exp(-np.logaddexp(0.0, l[t])) if sigmoid else 1.0     # sigmoid(-l)
        out[t] = ds * slope + dz * 2.0 / n * lse * np.exp(l[t] - lse)
    return out
