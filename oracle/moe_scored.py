"""The float64 statement of routing by scores and of its gradient, and of the
combine's gradient, on the CPU in numpy, from their definitions.

Beside each gradient stands the sum of the absolute values of its terms, from
which the tests derive how far float32 arithmetic may be off.
"""
from __future__ import annotations

import numpy as np


def scores(logits, score):
    """s [T, E]; a row of minus infinities has zeros."""
    l = np.asarray(logits, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        top = np.max(l, axis=1, keepdims=True)
        e = np.where(np.isneginf(top), 0.0, np.exp(l - top))
        z = np.sum(e, axis=1, keepdims=True)
        return np.where(z == 0, 0.0, e / np.where(z == 0, 1.0, z))


def route(logits, k, score="softmax", bias=None, groups=1, groups_kept=None, group_top=2, renormalise=True, scale=1.0):
    """dict: ids [T, k], gates [T, k], scores and order (c) [T, E], stay [T, E]
    (experts of the groups kept).  One token, one choice at a time."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    kept = groups if groups_kept is None else groups_kept
    size = E // groups
    s = scores(l, score)
    if bias is None and (kept == groups or group_top == 1):
        c = l.copy()                       # (the scores' order, where the scores are equal too)
    else:
        c = s + (0.0 if bias is None else np.asarray(bias, np.float64))
    c = np.where(np.isnan(c), -np.inf, c)
    stay = np.ones((T, E), bool)
    ids = np.zeros((T, k), np.int32)
    for t in range(T):
        if kept < groups:
            value = np.array([np.sum(np.sort(c[t, q * size:(q + 1) * size])[::-1][:group_top]) for q in range(groups)])
            value = np.where(np.isnan(value), -np.inf, value)
            best = sorted(range(groups), key=lambda q: (-value[q], q))[:kept]
            stay[t] = [e // size in best for e in range(E)]
        live = [e for e in range(E) if stay[t, e]]
        ids[t] = sorted(live, key=lambda e: (-c[t, e], e))[:k]
    chosen = np.take_along_axis(s, ids.astype(np.int64), 1)
    gates = chosen
    if renormalise:
        total = chosen.sum(1, keepdims=True)
        gates = np.where(total == 0, 0.0, chosen / np.where(total == 0, 1.0, total))
    return dict(ids=ids, gates=scale * gates, scores=s, order=c, stay=stay, sums=s.sum(0))


def route_backward(logits, ids, dgates, score="softmax", renormalise=True, scale=1.0, dscore_sums=None):
    """(dlogits [T, E], sum of |terms|)."""
    s = scores(logits, score)
    T, E = s.shape
    dg = np.asarray(dgates, np.float64) * scale
    ids = np.asarray(ids, np.int64)
    ds = np.zeros((T, E)) if dscore_sums is None else np.tile(np.asarray(dscore_sums, np.float64), (T, 1))
    mag = np.abs(ds)
    rows = np.arange(T)[:, None]
    chosen = s[rows, ids]
    add, size = dg, np.abs(dg)
    if renormalise:
        total = chosen.sum(1, keepdims=True)
        ok = total != 0
        total = np.where(ok, total, 1.0)
        mean = np.sum(chosen * dg, 1, keepdims=True) / total
        add = np.where(ok, (dg - mean) / total, 0.0)
        size = np.where(ok, (np.abs(dg) + np.sum(chosen * np.abs(dg), 1, keepdims=True) / total) / total, 0.0)
    np.add.at(ds, (rows, ids), add)
    np.add.at(mag, (rows, ids), size)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            rest = 1.0 / (1.0 + np.exp(np.asarray(logits, np.float64)))
        return ds * s * rest, mag * s * rest
    return s * (ds - np.sum(s * ds, 1, keepdims=True)), s * (mag + np.sum(s * mag, 1, keepdims=True))


def combine_backward(dy, y_perm, assign_pos, gates):
    """(dy_perm [T*k, d], NaN where no position points; dgates [T, k], sum of
    |terms| [T, k])."""
    dy, y_perm, gates = (np.asarray(v, np.float64) for v in (dy, y_perm, gates))
    T, k = gates.shape
    dy_perm = np.full(y_perm.shape, np.nan)
    dgates, terms = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            p = int(assign_pos[t * k + j])
            if p < 0:
                continue
            dy_perm[p] = gates[t, j] * dy[t]
            dgates[t, j] = np.dot(dy[t], y_perm[p])
            terms[t, j] = np.dot(np.abs(dy[t]), np.abs(y_perm[p]))
    return dy_perm, dgates, terms
