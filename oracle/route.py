"""Routing to experts and its gradient, written out from their definitions in fp64.

Test infrastructure (see the package docstring); never used by the product path.
"""
import math

import numpy as np


def scores(row, sigmoid):
    """Scores of one token's logits (fp64)."""
    x = np.asarray(row, np.float64)
    with np.errstate(all="ignore"):
        if sigmoid:
            return 1.0 / (1.0 + np.exp(-x))
        if not (x > -math.inf).any() and not np.isnan(x).any():
            return np.zeros_like(x)
        if np.isnan(x).any() or (x == math.inf).any():
            return np.full_like(x, np.nan)
        e = np.exp(x - x.max())
        return e / e.sum()


def route(logits, k, bias=None, sigmoid=False, groups=1, topk_groups=1, group_top=1, renorm=True, scale=1.0, live=None):
    """(ids int [T, k], weights fp64 [T, k]); one token after the other, choices by
    sorting (value, index)."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    ids, weights = np.full((T, k), -1), np.zeros((T, k))
    size = E // groups
    for t in range(T if live is None else min(max(live, 0), T)):
        s = scores(logits[t], sigmoid)
        def order(v):
            return [-math.inf if logits[t, e] == -math.inf else (-1e300 if math.isnan(v[e]) else float(v[e])) for e in range(E)]
        # without a bias experts go by their logits, and groups too where one expert stands for each
        v = order(logits[t] if bias is None else s + np.asarray(bias, np.float64))
        of_group = order(s) if bias is None and group_top > 1 else v
        on = list(range(E))
        if groups > 1:
            count = []
            for g in range(groups):
                best = sorted(of_group[g * size:(g + 1) * size], reverse=True)[:group_top]
                c = sum(best)
                count.append(-1e300 if math.isnan(c) else c)
            kept = sorted(range(groups), key=lambda g: (-count[g], g))[:topk_groups]
            on = [e for e in on if e // size in kept]
        on = sorted((e for e in on if v[e] > -math.inf), key=lambda e: (-v[e], e))[:k]
        w = np.array([s[e] for e in on])
        if renorm and len(on):
            w = w / w.sum() if w.sum() != 0 else 0.0 * w
        ids[t, :len(on)] = on
        weights[t, :len(on)] = scale * w
    return ids, weights


def weights_of(row, ids, sigmoid, renorm, scale):
    """The weights of one token as a function of its logits, the choice held fixed."""
    s = scores(row, sigmoid)
    w = np.array([s[e] if 0 <= e < len(row) else 0.0 for e in ids])
    if renorm:
        w = w / w.sum() if w.sum() != 0 else 0.0 * w
    return scale * w


def route_backward(dweights, logits, ids, sigmoid=False, renorm=True, scale=1.0):
    """(dlogits fp64 [T, E], the sum of the magnitudes of its terms) from the
    Jacobian of each token's weights."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        s = scores(logits[t], sigmoid)
        there = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
        ds = np.zeros((E, E))              # d s[i] / d l[e]
        if sigmoid:
            np.fill_diagonal(ds, s * (1.0 - s))
        else:
            ds = np.diag(s) - np.outer(s, s)
        rows = np.array([ds[ids[t, j]] for j in there]).reshape(len(there), E)
        w = np.array([s[ids[t, j]] for j in there])
        if renorm and len(there):
            tot = w.sum()
            rows = rows * 0.0 if tot == 0 else rows / tot - np.outer(w, rows.sum(0)) / tot ** 2
            m = 0.0 * rows if tot == 0 else np.abs(np.array([ds[ids[t, j]] for j in there])) / tot + \
                np.outer(w, np.abs(np.array([ds[ids[t, j]] for j in there])).sum(0)) / tot ** 2
        else:
            m = np.abs(rows)
        g = np.array([float(dweights[t, j]) for j in there])
        if len(there):
            out[t] = scale * (g @ rows)
            mag[t] = abs(scale) * (np.abs(g) @ m)
    return out, mag
