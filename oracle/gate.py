"""Router gate in fp64: the top-k experts of every token, their weights and
the logits' gradient.  TEST INFRASTRUCTURE ONLY (see the package docstring).

Per token with logits l (NaN sorts first, then larger first, equal values by
lower expert; -inf is never selected, the rest of a short row is id -1 and
weight 0), for the selected i:

    softmax           w_i = scale e^l_i / sum_e e^l_e
    softmax, renorm   w_i = scale e^l_i / sum_selected e^l_j
    sigmoid           w_i = scale s(l_i),  s(v) = 1 / (1 + e^-v)
    sigmoid, renorm   w_i = scale s(l_i) / sum_selected s(l_j)

The gradient treats the selection as a constant; the Jacobian-vector products
are written out per row.
"""

from __future__ import annotations

import numpy as np

SOFTMAX, SIGMOID = 0, 1


def select(logits: np.ndarray, k: int) -> np.ndarray:
    """ids int32 [T, k]."""
    l = np.asarray(logits, dtype=np.float64)
    T, E = l.shape
    ids = np.full((T, k), -1, np.int32)
    for t in range(T):
        row = sorted((e for e in range(E) if l[t, e] != -np.inf),
                     key=lambda e: (0, 0.0, e) if np.isnan(l[t, e]) else (1, -l[t, e], e))
        ids[t, :min(k, len(row))] = row[:k]
    return ids


def _log_sigmoid(v):
    return np.minimum(v, 0.0) - np.log1p(np.exp(-np.abs(v)))


def weights(logits, ids, score: int, renorm: bool, scale: float = 1.0) -> np.ndarray:
    """fp64 [T, k] weights of the given selection (0 where ids is -1)."""
    l = np.asarray(logits, dtype=np.float64)
    ids = np.asarray(ids)
    w = np.zeros(ids.shape)
    with np.errstate(invalid="ignore", over="ignore"):
        for t in range(l.shape[0]):
            ok = ids[t] >= 0
            if not ok.any():
                continue
            v = l[t, ids[t][ok]]
            a = v if score == SOFTMAX else _log_sigmoid(v)
            if renorm:
                r = np.exp(a - a.max())
                w[t, ok] = r / r.sum()
            elif score == SOFTMAX:
                m = l[t].max()
                w[t, ok] = np.exp(v - m) / np.exp(l[t] - m).sum()
            else:
                w[t, ok] = np.exp(a)
    return w * scale


def topk_gate_f64(logits, k: int, score: int, renorm: bool, scale: float = 1.0):
    ids = select(logits, k)
    return ids, weights(logits, ids, score, renorm, scale)


def topk_gate_backward_f64(logits, ids, dweights, score: int, renorm: bool, scale: float = 1.0) -> np.ndarray:
    """fp64 [T, E]."""
    l = np.asarray(logits, dtype=np.float64)
    d = np.zeros(l.shape)
    for t in range(l.shape[0]):
        ok = (ids[t] >= 0) & (ids[t] < l.shape[1])
        if not ok.any():
            continue
        i = ids[t][ok]
        g = scale * np.asarray(dweights[t], dtype=np.float64)[ok]
        u = weights(l[t:t + 1], i[None], score, renorm)[0]
        if score == SOFTMAX and not renorm:
            p = np.exp(l[t] - l[t].max())
            p /= p.sum()
            d[t] -= p * (g * u).sum()
            np.add.at(d[t], i, u * g)
        else:
            s1 = np.exp(_log_sigmoid(-l[t, i])) if score == SIGMOID else 1.0       # 1 - s
            np.add.at(d[t], i, u * (g - (g * u).sum()) * s1 if renorm else g * u * s1)
    return d
